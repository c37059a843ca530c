"""Distillation on logits of any finite size (needs a B200).

A row's probabilities depend on differences of its logits alone, and fp32 forms the difference to
the row's maximum to half a last place, so the bounds here grow with the distance from the
maximum and never with the logits themselves.  With gap_j = (max z - z_j) / tau, in units of u = 2^-24:
the difference, its product with the rounded factor log2(e) / tau and that factor are off by at most
4 u gap_j together; the exponential and logarithm units, the sum of up to 2^17 terms (a few hundred a
thread, then a tree) and the roundings around them by at most 2^-20 relative (absolute for a logarithm).
"""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

from random_gradient_projection_b200 import lm  # noqa: E402

U, UNIT = 2.0 ** -24, 2.0 ** -20


def definition(z, idx, val, tau):
    """loss, Gout in 64 bits and their bounds (every entry valid, no weights)."""
    dtype = z.dtype
    z, val, i = z.double() / tau, val.double() / tau, idx.long()
    q, logp = torch.softmax(val, 1), torch.log_softmax(z, 1)
    at = logp.gather(1, i)
    lq = torch.log_softmax(val, 1)
    held = q > 0
    terms = torch.where(held, q * (lq - at), torch.zeros_like(q))
    p, mass = logp.exp(), torch.zeros_like(z).scatter_add_(1, i, q)
    G = tau * (p - mass)
    gap, vgap = z.amax(1, keepdim=True) - z, val.amax(1, keepdim=True) - val
    rel, vrel = UNIT + 4 * U * gap, UNIT + 4 * U * vgap
    # exponents 8 u apart at the most for what still counts: p below 2^-126 is flushed to zero
    bG = tau * (2 * rel * p + torch.zeros_like(z).scatter_add_(1, i, 2 * vrel * q)) + (
        torch.finfo(dtype).eps / 2 + 4 * U) * G.abs() + tau * 2.0 ** -120
    off = rel.gather(1, i) + vrel + 4 * U * (lq.abs() + at.abs())
    bl = tau ** 2 * torch.where(held, q * (2 * off + 2 * vrel * (lq - at).abs()), torch.zeros_like(q)).sum(1)
    return tau ** 2 * terms.sum(1), G, bl + 1e-30, bG


def check(z, idx, val, tau):
    loss, G = lm.distill_loss(z, idx, val, temperature=tau)
    rl, rG, bl, bG = definition(z, idx, val, tau)
    assert loss.isfinite().all() and G.isfinite().all()
    assert float(((loss.double() - rl).abs() / bl).max()) <= 1.0
    assert float(((G.double() - rG).abs() / bG).max()) <= 1.0


# rows of one CTA each (16 KB), and of the kernel for long rows with two and with one CTA on an SM
SIZES = [(4099, torch.float32), (9001, torch.float32), (20001, torch.float32), (4099, torch.bfloat16),
         (20001, torch.bfloat16), (40001, torch.bfloat16)]


@pytest.mark.parametrize("V,dt", SIZES)
@pytest.mark.parametrize("offset", [-3e38, -1e10, -1e5, -1000.0, 1000.0, 1e5, 1e7, 1e10, 3e38])
def test_a_common_offset_of_the_logits(V, dt, offset):
    """Rows of equal logits, and rows whose logits lie a few last places of the offset apart."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V)
    N, K = 5, 7
    z = torch.full((N, V), offset, dtype=torch.float32, device="cuda").to(dt)
    steps = torch.randint(-40, 1, (N, V), generator=g, device="cuda")
    unit = abs(offset) * torch.finfo(dt).eps
    z = (z.double() + steps * unit).clamp(-torch.finfo(dt).max, torch.finfo(dt).max).to(dt)
    z[0] = z[0, 0]
    z[1] = torch.tensor(offset, device="cuda").to(dt)
    z[2, ::5] = 0.0
    idx = torch.stack([torch.randperm(V, generator=g, device="cuda")[:K] for _ in range(N)])
    # the teacher holds entries near the maximum as well as far ones
    idx[:, 0] = z.float().argmax(1)
    val = torch.randn(N, K, generator=g, device="cuda")
    for tau in (1.0, 0.5, 4.0):
        loss, G = lm.distill_loss(z, idx, val, temperature=tau)
        rl, rG, bl, bG = definition(z, idx, val, tau)
        ok = rl < 1e30                       # (a far entry's loss may pass fp32; its row's gradient does not)
        assert G.isfinite().all() and loss[ok].isfinite().all()
        assert float(((loss.double() - rl).abs() / bl)[ok].max()) <= 1.0
        assert float(((G.double() - rG).abs() / bG).max()) <= 1.0


@pytest.mark.parametrize("V,dt", [(4099, torch.float32), (20001, torch.float32)])
@pytest.mark.parametrize("offset", [0.0, 60.0, 1000.0, -2000.0])
def test_a_student_near_its_hard_label(V, dt, offset):
    """1 - p of about 1e-5: loss and the label's gradient are what is left of a difference."""
    g = torch.Generator(device="cuda")
    g.manual_seed(V + 1)
    N = 300
    z = torch.randn(N, V, generator=g, device="cuda")
    idx = torch.randint(V, (N, 1), generator=g, device="cuda")
    z.scatter_(1, idx, math.log(V * 1.65) + 11.0)
    z += offset
    check(z.to(dt), idx, torch.zeros(N, 1, device="cuda"), 1.0)


@pytest.mark.parametrize("V", [4099, 20001])
@pytest.mark.parametrize("tau", [2.0 ** -60, 2.0 ** -20, 2.0 ** 10])
def test_temperatures_near_the_ends_of_their_range(V, tau):
    g = torch.Generator(device="cuda")
    g.manual_seed(V + 2)
    z = 3.0 * torch.randn(6, V, generator=g, device="cuda")
    idx = torch.randint(V, (6, 5), generator=g, device="cuda")
    idx[:, 0] = z.argmax(1)
    check(z, idx, torch.randn(6, 5, generator=g, device="cuda"), tau)


@pytest.mark.parametrize("V", [4099, 20001])
def test_the_highest_temperature_is_the_uniform_distribution(V):
    z = torch.randn(4, V, device="cuda")
    idx = torch.tensor([[0, 1, 2, 3]] * 4, device="cuda")
    tau = 2.0 ** 60
    loss, G = lm.distill_loss(z, idx, torch.randn(4, 4, device="cuda"), temperature=tau)
    want = torch.full_like(G, tau / V)
    want[:, :4] -= tau / 4
    assert loss.isfinite().all() and torch.allclose(G, want, rtol=1e-5)
