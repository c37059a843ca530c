"""The gradient of H alone where the vocabulary takes more than one piece, with and without splits of
the sum over it, with dropped rows, and with a row that needs the second method (needs a B200)."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import lm  # noqa: E402


@pytest.mark.parametrize("far", [False, True])
@pytest.mark.parametrize("N,d,V,masked", [(8100, 256, 32000, 0.0), (8100, 256, 32000, 0.3), (8190, 1024, 20000, 0.1)])
def test_input_gradient_in_several_pieces(N, d, V, masked, far):
    g = torch.Generator(device="cuda")
    g.manual_seed(N + d)
    W = torch.randn(V, d, generator=g, device="cuda") * (2.5 / math.sqrt(d))
    labels = torch.randint(V, (N,), generator=g, device="cuda")
    labels[torch.rand(N, generator=g, device="cuda") < masked] = -1
    H = torch.randn(N, d, generator=g, device="cuda")
    labels[7] = V - 2                                  # in the last piece
    H[7] = (-60.0 if far else 1.0) * W[V - 2]          # a loss of some hundreds, or a sure row
    H[labels < 0] = math.nan
    w = 0.1 + torch.rand(N, generator=g, device="cuda")
    H, W = H.bfloat16(), W.bfloat16()
    got = lm.head_loss(H, W, labels, weights=w)
    for a in range(0, N, 2048):
        part = slice(a, a + 2048)
        r = ref.head(H[part], W, labels[part], w[part])
        bl, bH, _ = ref.head_bounds(r, H.dtype)
        ref.check(got.loss[part], r["loss"], bl, "loss"), ref.check(got.dH[part], r["dH"], bH, "dH")
    assert (float(got.loss[7]) > 60.0) == far
