"""The language-model operators in 64 bits on the CPU or the GPU, written from their formulas
with torch, and the error bounds the kernels are held to.

Bounds are per element and count roundings: u16 = 2^-8 is half a step of bf16, u32 = 2^-24 of
fp32.  A tensor-core product of K terms accumulates in K/16 steps, each off by at most two
last places of the running sum, whose magnitude is at most sum |a||b|: STEP (K/16 + 1) sum |a||b|
with STEP = 2^-22 (six such sums where fp32 operands are split into planes).  The exponential
and logarithm units are off by at most 2^-21 relative.
"""
import math

import torch

U16, U32, STEP, UNIT = 2.0 ** -8, 2.0 ** -24, 2.0 ** -22, 2.0 ** -20


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def head(H, W, labels, weights):
    """loss, dH, dW in 64 bits; dropped rows zero.  Rows are flattened."""
    H2, W, t = H.reshape(-1, H.shape[-1]), W.double(), labels.reshape(-1).long()
    f = torch.ones(t.numel(), device=H.device, dtype=torch.float64) if weights is None else weights.reshape(-1).double()
    live = (t >= 0) & (t < W.shape[0]) & (f != 0)
    h, t, f = H2[live].double(), t[live], f[live]
    z = h @ W.T
    logp = torch.log_softmax(z, 1)
    rows = torch.arange(t.numel(), device=t.device)
    loss = torch.zeros(H2.shape[0], dtype=torch.float64, device=H.device)
    loss[live] = -f * logp[rows, t]
    g = logp.exp()
    gp = f[:, None].abs() * g          # |w| p, for the bounds
    g[rows, t] -= 1.0
    g = f[:, None] * g
    dH = torch.zeros(H2.shape, dtype=torch.float64, device=H.device)
    dH[live] = g @ W
    return dict(loss=loss.reshape(H.shape[:-1]), dH=dH.reshape(H.shape), dW=g.T @ h, live=live, z=z, g=g, gp=gp, h=h,
                W=W, f=f, rows=rows, t=t)


def head_bounds(r, dtype):
    """Per-element bounds of loss, dH and dW for inputs of `dtype`, of what `head` returned."""
    K, V = r["h"].shape[1], r["W"].shape[0]
    planes = 6 if dtype == torch.float32 else 1
    steps = lambda k: STEP * planes * (k / 16 + 1)  # noqa: E731
    # a logit, and with it every exponent: accumulation, the three dropped products of planes, and
    # the roundings of (z - lse) log2 e
    dz = (steps(K) + (4 * U32 if planes == 6 else 0)) * (r["h"].abs() @ r["W"].abs().T)
    top = dz.amax(1) if dz.numel() else dz.sum(1)
    zmax = r["z"].abs().amax(1) if r["z"].numel() else r["z"].sum(1)
    rel = 2 * top + 8 * U32 * zmax + UNIT          # relative error of a probability
    loss = torch.zeros(r["live"].numel(), dtype=torch.float64, device=r["z"].device)
    loss[r["live"]] = r["f"].abs() * (2 * top + 8 * U32 * zmax + UNIT * (1 + math.log(V)))
    ug = U16 if planes == 1 else 4 * U32           # g as an operand
    # (the exponential unit flushes a probability below 2^-126 to zero: off by that much, times w)
    dg = rel[:, None] * r["gp"] + (ug + 4 * U32) * r["g"].abs() + 2.0 ** -126 * r["f"][:, None].abs()
    ga = r["g"].abs() + dg
    N = r["h"].shape[0]
    uo = half_step(dtype)
    dH = torch.zeros(r["live"].numel(), K, dtype=torch.float64, device=r["z"].device)
    dH[r["live"]] = dg @ r["W"].abs() + steps(V) * (ga @ r["W"].abs()) + uo * (r["g"] @ r["W"]).abs() * 1.01
    dW = dg.T @ r["h"].abs() + steps(N) * (ga.T @ r["h"].abs()) + uo * (r["g"].T @ r["h"]).abs() * 1.01
    tiny = 1e-38   # results below the normal range
    return loss + tiny, dH + tiny, dW + tiny


def distill(logits, idx, val, weights, tau):
    """loss and Gout in 64 bits, and their bounds."""
    V, dtype = logits.shape[-1], logits.dtype
    z, i, v = logits.reshape(-1, V).double(), idx.reshape(-1, idx.shape[-1]).long(), val.reshape(-1, idx.shape[-1]).double()
    f = torch.ones(z.shape[0], device=z.device, dtype=torch.float64) if weights is None else weights.reshape(-1).double()
    there = (i >= 0) & (i < V)
    live = (f != 0) & (there & (v > -math.inf)).any(1)
    loss, bl = torch.zeros_like(f), torch.zeros_like(f)
    G, bg = torch.zeros_like(z), torch.zeros_like(z)
    if live.any():
        z, i, v, f, there = z[live], i[live].clamp(0, V - 1), v[live], f[live], there[live]
        q = torch.softmax((v / tau).masked_fill(~there, -math.inf), 1)
        logp = torch.log_softmax(z / tau, 1)
        at = logp.gather(1, i)
        lq = torch.where(q > 0, q.clamp(min=1e-300).log(), torch.zeros_like(q))
        terms = torch.where(q > 0, q * (lq - at), torch.zeros_like(q))
        loss[live] = f * tau ** 2 * terms.sum(1)
        p, mass = logp.exp(), torch.zeros_like(z).scatter_add_(1, i, q)
        G[live] = f[:, None] * tau * (p - mass)
        # exponents: a rounding of z log2e / tau and of the difference, per unit of their size
        zf = torch.where(p > 1e-30, z.abs(), torch.zeros_like(z)).amax(1)   # of the entries that count
        vf = torch.where(there & v.isfinite(), v.abs(), torch.zeros_like(v)).amax(1)
        rel = UNIT + 8 * U32 * (zf / tau), UNIT + 8 * U32 * (vf / tau)
        atf = torch.where(q > 0, at, torch.zeros_like(at)).abs()
        size = (q * (lq.abs() + atf + 1)).sum(1)
        bl[live] = f.abs() * tau ** 2 * (2 * rel[0] + 2 * rel[1]) * size
        bg[live] = f[:, None].abs() * tau * (2 * rel[0][:, None] * p + 2 * rel[1][:, None] * mass) + (
            half_step(dtype) + 4 * U32) * G[live].abs()
    tiny = 1e-37
    return loss.reshape(logits.shape[:-1]), G.reshape(logits.shape), bl.reshape(logits.shape[:-1]) + tiny, \
        bg.reshape(logits.shape) + tiny


def embed_sums(ids, G, vocab, scale, weights=None):
    """Squared norms per sample, the weighted table gradient, and their bounds."""
    B, T = ids.shape
    d = G.shape[-1]
    grad = torch.zeros(vocab, d, dtype=torch.float64, device=G.device)
    size, count = torch.zeros_like(grad), torch.zeros(vocab, dtype=torch.float64, device=G.device)
    sq, bsq = (torch.zeros(B, dtype=torch.float64, device=G.device) for _ in range(2))
    for b in range(B):
        t = ids[b].long()
        there = (t >= 0) & (t < vocab)
        t, g = t[there], G[b][there].double() * scale
        mine = torch.zeros_like(grad).index_add_(0, t, g)
        mabs = torch.zeros_like(grad).index_add_(0, t, g.abs())
        n = torch.zeros_like(count).index_add_(0, t, torch.ones_like(t, dtype=torch.float64))
        sq[b] = (mine * mine).sum()
        # each row's sum is off by (n + 2) u32 of its magnitude; then a sum of d + T squares
        bsq[b] = ((2 * (n[:, None] + 3) * U32 * mabs * (mine.abs() + (n[:, None] + 3) * U32 * mabs)).sum()
                  + (d + T + 16) * U32 * sq[b])
        c = 1.0 if weights is None else float(weights[b])
        grad += c * mine
        size += abs(c) * mabs
        count += n
    return sq, grad, bsq + 1e-37, (count[:, None] + 4) * U32 * size + 1e-37


def check(got, ref, bound, what=""):
    """Every element within its bound; where the reference is not finite, the same NaN or infinity."""
    got = got.double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = ref.isfinite()
    assert torch.equal(got.isnan(), ref.isnan()), what
    assert torch.equal(got[~fine & ~ref.isnan()], ref[~fine & ~ref.isnan()]), what
    if fine.any():
        over = ((got - ref).abs() / bound)[fine]
        assert float(over.max()) <= 1.0, f"{what}: {float(over.max()):.3g} times the bound"
        return float(over.max())
    return 0.0
