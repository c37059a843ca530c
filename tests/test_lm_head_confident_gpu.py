"""Head loss and its gradients where a row is sure of its label (needs a B200).

There 1 - p is small and everything is made of it: the loss, the label's entry of the logits'
gradient and the sum of all others.  The bounds are relative to each entry of that gradient, so they do
not grow with p or with the logits.  Per entry g_v: every exponent is a difference of two logits, each
off by `top` (the products' accumulation), and its scaling to base 2 by 4 u of the gap to the row's
maximum; the exponential, the sum and the division by at most 2^-20 together.  The label's entry is the
negative sum of the others, so the largest of their relative errors bounds it."""
import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import lm  # noqa: E402

U16, U32, STEP, UNIT = ref.U16, ref.U32, ref.STEP, ref.UNIT
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def sure_rows(N, d, V, dt, seed, height):
    """Rows along their label's weights: 1 - p from about 1e-6 on, every logit lifted by `height`."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    W = torch.randn(V, d, generator=g, device="cuda") / d ** 0.5
    labels = torch.randperm(V, generator=g, device="cuda")[:N] if N <= V else torch.arange(N, device="cuda") % V
    # the first column lifts every logit of a row alike, the label's direction its own
    W[:, 0] = 1.0
    H = torch.zeros(N, d, device="cuda")
    lift = 5.0 + 14.0 * torch.rand(N, generator=g, device="cuda")
    H[:, 1:] = W[labels, 1:] * (lift / W[labels, 1:].square().sum(1))[:, None]
    H[:, 0] = height
    w = 0.1 + torch.rand(N, generator=g, device="cuda")
    return H.to(DT[dt]), W.to(DT[dt]), labels, w


def definition(H, W, labels, w):
    """loss, dH, dW and their bounds in 64 bits; the label's gradient from the others' sum."""
    planes = 6 if H.dtype == torch.float32 else 1
    h, W, f = H.double(), W.double(), w.double()
    z = h @ W.T
    rows = torch.arange(h.shape[0], device=h.device)
    logp = torch.log_softmax(z, 1)
    g = logp.exp()
    g[rows, labels] = 0.0
    rest = g.sum(1)
    g[rows, labels] = -rest
    loss = f * -torch.log1p(-rest)
    g = f[:, None] * g
    steps = lambda k: STEP * planes * (k / 16 + 1)  # noqa: E731
    dz = (steps(h.shape[1]) + (4 * U32 if planes == 6 else 0)) * (h.abs() @ W.abs().T)
    gap = (z.amax(1) - z.min(1).values) * 1.5
    rel = 2 * dz.amax(1) + 4 * U32 * gap + UNIT
    dg = (rel[:, None] + (U16 if planes == 1 else 4 * U32) + 4 * U32) * g.abs() + 2.0 ** -126
    bl = (f * rest * rel + UNIT * loss) * 1.01 + 1e-37   # d loss = rest times the relative error of (1 - p) / p
    ga, uo = g.abs() + dg, ref.half_step(H.dtype)
    dH, dW = g @ W, g.T @ h
    bH = dg @ W.abs() + steps(W.shape[0]) * (ga @ W.abs()) + uo * dH.abs() * 1.01 + 1e-37
    bW = dg.T @ h.abs() + steps(h.shape[0]) * (ga.T @ h.abs()) + uo * dW.abs() * 1.01 + 1e-37
    return loss, dH, dW, bl, bH, bW


CASES = [(200, 64, 1000), (77, 40, 333), (300, 264, 2049), (1200, 64, 700)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V", CASES)
@pytest.mark.parametrize("height", [0.0, 100.0, -300.0])
def test_gradients_of_sure_rows(N, d, V, dt, height):
    H, W, labels, w = sure_rows(N, d, V, dt, N + V, height)
    got = lm.head_loss(H, W, labels, weights=w, weight_grad=True)
    loss, dH, dW, bl, bH, bW = definition(H, W, labels, w)
    print("of the bounds:", ref.check(got.loss, loss, bl, "loss"), ref.check(got.dH, dH, bH, "dH"),
          ref.check(got.dW, dW, bW, "dW"))
    # a row's loss and gradient do not depend on what else was asked for
    assert torch.equal(lm.head_loss(H, W, labels, weights=w, grad=False).loss, got.loss)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_one_pass_and_two_passes_agree_on_sure_rows(dt):
    """dH alone of this size is summed in one pass; with dW, and where a row's loss is too large for
    that, in two."""
    H, W, labels, w = sure_rows(256, 512, 40001, dt, 9, 80.0)
    loss, dH, _, bl, bH, _ = definition(H, W, labels, w)
    alone, both = lm.head_loss(H, W, labels, weights=w), lm.head_loss(H, W, labels, weights=w, weight_grad=True)
    H2 = H.clone()
    H2[255] = H2[255] * -20.0            # far from its label: every row is computed again
    again = lm.head_loss(H2, W, labels, weights=w)
    for got in (alone, both):
        ref.check(got.loss, loss, bl, "loss"), ref.check(got.dH, dH, bH, "dH")
    ref.check(again.loss[:255], loss[:255], bl[:255], "loss"), ref.check(again.dH[:255], dH[:255], bH[:255], "dH")
