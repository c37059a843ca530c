"""Samples of weight 0 in the table's clipped sum (needs a B200)."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import lm  # noqa: E402


@pytest.mark.parametrize("B,T,V,d,dt", [
    (6, 40, 30, 64, torch.bfloat16), (6, 40, 30, 31, torch.float32), (5, 2100, 7, 264, torch.bfloat16),
    (40, 3, 5, 8, torch.float32), (3, 900, 1, 40, torch.bfloat16)])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_sample_of_weight_zero_adds_nothing_whatever_it_holds(B, T, V, d, dt, bad):
    g = torch.Generator(device="cuda")
    g.manual_seed(B * T)
    ids = torch.randint(-1, V, (B, T), generator=g, device="cuda")
    G = torch.randn(B, T, d, generator=g, device="cuda").to(dt)
    w = 0.1 + torch.rand(B, generator=g, device="cuda")
    w[1::3] = 0.0
    clean = torch.where((w == 0)[:, None, None], torch.zeros_like(G), G)
    G[w == 0] = bad
    order = lm.embed_order(ids, V)
    got = lm.embed_grad(order, G, weights=w, scale=2.5)
    assert torch.equal(got, lm.embed_grad(order, clean, weights=w, scale=2.5))
    _, grad, _, bound = ref.embed_sums(ids, clean, V, 2.5, w)
    ref.check(got, grad, bound, "grad")
