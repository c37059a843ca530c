"""A private training step of a small language model, per sample against autograd in 64 bits, and the
parameters beside the stack on every kind of step (needs a B200).

The model: a trained token table, one linear layer in the stack, a frozen head of its own.
"""
import math
import statistics
import time

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import GrapeStep, grape, lm  # noqa: E402


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def test_a_private_step_with_a_head_of_its_own_against_autograd():
    """Losses, dH, dA, the per-sample norms of the table's gradient, the clip over both shares and the
    clipped sum.  fp32 throughout: each of the chain's three products (256 to 700 terms) is off by at
    most K 2^-24 = 4.2e-5 of its factors' norms, which are less than ten times the product's."""
    B, T, d, V, C = 6, 40, 256, 700, 0.05
    g = rng(31)
    table = torch.randn(V, d, generator=g, device="cuda") / math.sqrt(d)
    head = torch.randn(V, d, generator=g, device="cuda") * (2.0 / math.sqrt(d))
    W = torch.randn(d, d, generator=g, device="cuda") / math.sqrt(d)
    ids = torch.randint(V, (B, T), generator=g, device="cuda")
    ids[:, 10:20] = ids[:, :10]                       # repeated tokens
    labels = torch.roll(ids, -1, 1)
    labels[:, -1] = -100
    ids[1, 25:], labels[1, 24:] = -1, -100            # a padded sample
    ids[4], labels[4] = -1, -100                      # and one of nothing else
    live = labels >= 0
    weights = live.float() / live.sum(1, keepdim=True).clamp(min=1)
    scale = math.sqrt(d)

    A = lm.embed(table, ids, scale=scale, dtype="f32")
    H = A @ W
    out = lm.head_loss(H, head, labels, weights=weights)
    dA = out.dH @ W.T
    order = lm.embed_order(ids, V)
    sq = lm.embed_sqnorms(order, dA, scale=scale)
    step = GrapeStep([(d, d)], r=128, C=C, sigma=0.0, seed=5, B=B, T=T, dtype="f32")
    A2, G2, W2 = A.view(B * T, d), out.dH.view(B * T, d), W.clone()
    alone = step.sqnorms([A2], [G2], 0).clone()
    step.set_extra_sqnorms(sq)
    step.step([A2], [G2], [W2], 0)
    c = step.clip_tensor()
    dE = lm.embed_grad(order, dA, weights=c, scale=scale)
    torch.cuda.synchronize()

    E64, W64, U64 = table.double(), W.double(), head.double()
    want_dE = torch.zeros_like(E64)
    close = lambda a, b: float((a.double() - b).norm()) <= 1e-3 * float(b.norm()) + 1e-12  # noqa: E731
    for i in range(B):
        E = E64.clone().requires_grad_(True)
        a = torch.where((ids[i] >= 0)[:, None], E[ids[i].clamp(min=0)] * scale, torch.zeros((), dtype=torch.float64, device="cuda"))
        a.retain_grad()
        h = a @ W64
        h.retain_grad()
        z = torch.log_softmax(h @ U64.T, 1)
        rows = torch.arange(T, device="cuda")
        losses = -weights[i].double() * z[rows, labels[i].clamp(min=0)]
        losses.sum().backward()
        assert close(out.loss[i], losses.detach()) and close(out.dH[i], h.grad) and close(dA[i], a.grad)
        n = float(E.grad.square().sum())
        assert abs(float(sq[i]) - n) <= 2e-3 * n + 1e-12
        joint = math.sqrt(float(alone[i]) + n)
        assert abs(float(c[i]) - min(1.0, C / joint if joint else 1.0)) <= 2e-3
        want_dE += float(c[i]) * E.grad
    assert close(dE, want_dE) and float(c.min()) < 0.9 and float(c[4]) == 1.0
    step.close()


def stack(B=4, T=64, d=256, layers=2, seed=9):
    g = rng(seed)
    A = [torch.randn(B * T, d, generator=g, device="cuda").bfloat16() for _ in range(layers)]
    G = [(0.02 * torch.randn(B * T, d, generator=g, device="cuda")).bfloat16() for _ in range(layers)]
    W = [torch.randn(d, d, generator=g, device="cuda") for _ in range(layers)]
    return B, T, d, A, G, W


@pytest.mark.parametrize("how", ["step", "ghost", "stored", "recompute", "host", "masked", "accumulate", "bound"])
def test_extra_norms_reach_every_kind_of_step(how):
    """Two steps each, so that a share that stayed in the norms of the step before would show."""
    B, T, d, A, G, W = stack()
    extra = torch.tensor([0.0, 2.0, 0.5, 30.0], device="cuda")
    g = GrapeStep([(d, d)] * 2, r=128, C=1.0, sigma=0.0, seed=1, B=B, T=T)
    if how == "ghost":
        g.set_norm_method(grape.GRAPE_NORM_GHOST)
    if how in ("stored", "recompute"):
        g.set_aggregation(grape.GRAPE_AGG_STORE if how == "stored" else grape.GRAPE_AGG_RECOMPUTE)
    g.set_extra_sqnorms(extra)
    if how == "masked":
        g.enable_compaction(T + 8)
        pad = lambda x: torch.cat([x.view(B, T, -1), torch.full_like(x.view(B, T, -1)[:, :8], 3.0)], 1).contiguous()  # noqa: E731
        mask = (torch.arange(T + 8, device="cuda") < T).repeat(B, 1).to(torch.uint8)
        Am, Gm = [pad(x) for x in A], [pad(x) for x in G]
    for s in range(2):
        if how == "host":
            g.step_host([x.cpu() for x in A], [x.cpu() for x in G], W, s)
        elif how == "masked":
            g.step_masked(Am, Gm, W, mask, s)
        elif how == "accumulate":
            g.accumulate(A, G, s)
            g.apply(W, s)
        elif how == "bound":
            g.bind(A, G, W).step(s)
        else:
            g.step(A, G, W, s)
        torch.cuda.synchronize()
        got, c = torch.from_numpy(g.norms()).double(), g.clip_tensor().double().cpu()
        n = (g.sqnorms(A, G, s).double() + extra).sqrt().cpu()
        assert torch.allclose(got, n, rtol=1e-5)
        assert torch.allclose(c, torch.where(n > 1, 1 / n, torch.ones_like(n)), rtol=1e-5)
    g.close()


def test_extra_norms_with_a_process_group():
    import torch.distributed as dist

    from random_gradient_projection_b200.data_parallel import dp_step
    B, T, d, A, G, W = stack(seed=10)
    extra = torch.tensor([1.0, 0.0, 4.0, 9.0], device="cuda")
    g = GrapeStep([(d, d)] * 2, r=128, C=1.0, sigma=0.0, seed=1, B=B, T=T)
    g.set_extra_sqnorms(extra)
    dist.init_process_group("gloo", store=dist.HashStore(), rank=0, world_size=1)
    try:
        dp_step(g, A, G, W, 0)
        torch.cuda.synchronize()
    finally:
        dist.destroy_process_group()
    n = (g.sqnorms(A, G, 0).double() + extra).sqrt().cpu()
    assert torch.allclose(torch.from_numpy(g.norms()).double(), n, rtol=1e-5)
    g.close()


def test_distillation_feeds_a_layer_of_the_stack():
    """The head as a layer: S = sum_i c_i P^T A_i^T Gout_i of the definition's Gout.  A, Gout and P
    are held in bf16 and so is A P: four roundings of 2^-9 at most that average out, 2e-2 as for
    every step."""
    B, T, d, V = 3, 50, 256, 1024
    g = rng(17)
    A = torch.randn(B, T, d, generator=g, device="cuda").bfloat16()
    W = torch.randn(d, V, generator=g, device="cuda") / math.sqrt(d)
    logits = (A.view(-1, d).float() @ W).bfloat16().view(B, T, V)
    idx = torch.randint(-1, V, (B, T, 6), generator=g, device="cuda")
    val = torch.randn(B, T, 6, generator=g, device="cuda")
    weights = torch.full((B, T), 1.0 / T, device="cuda")
    weights[1, 30:] = 0.0
    loss, Gout = lm.distill_loss(logits, idx, val, weights=weights, temperature=2.0)
    step = GrapeStep([(d, V)], r=128, C=0.05, sigma=0.0, seed=3, B=B, T=T)
    step.step([A.view(B * T, d)], [Gout.view(B * T, V)], [W.clone()], 0)
    torch.cuda.synchronize()
    rl, rG, bl, _ = ref.distill(logits, idx, val, weights, 2.0)
    ref.check(loss, rl, bl, "loss")
    P, c = torch.from_numpy(step.P(0)).double().cuda(), step.clip_tensor().double()
    S = sum(c[i] * P.T @ A[i].double().T @ rG[i] for i in range(B))
    got = torch.from_numpy(step.S(0)).double().cuda()
    assert float((got - S).norm() / S.norm()) <= 2e-2 and float(c.min()) < 1.0
    step.close()


def test_graphs_are_kept_when_the_norms_lie_elsewhere_each_step():
    """`set_extra_sqnorms(lm.embed_sqnorms(...))` of every step is another tensor: the captured step is
    replayed on it all the same (capturing it anew each time took 249 us against 43)."""
    B, T, d, A, G, W = stack(layers=8)
    g = GrapeStep([(d, d)] * 8, r=128, C=1.0, sigma=0.0, seed=1, B=B, T=T)
    g.set_graph(True)
    pool = torch.rand(12, B, device="cuda") * 40.0

    def run(steps, address):
        took = []
        for s in range(steps):
            x = pool[address(s)]
            t = time.perf_counter()
            g.set_extra_sqnorms(x)
            g.step(A, G, W, s)
            took.append(time.perf_counter() - t)
            torch.cuda.synchronize()
            n = (g.sqnorms(A, G, s).double() + x).sqrt().cpu()
            assert torch.allclose(torch.from_numpy(g.norms()).double(), n, rtol=1e-5)
        return statistics.median(took)
    run(3, lambda s: 0)
    fixed, moving = run(24, lambda s: 0), run(24, lambda s: s % 12)
    print(f"median host time of a step: fixed {fixed * 1e6:.0f} us, moving {moving * 1e6:.0f} us")
    assert moving <= 3 * fixed        # (5.8 times with a capture each; room for a busy host)
    # and without the share, and with it again
    for x in (None, pool[3], None, pool[5]):
        g.set_extra_sqnorms(x)
        g.step(A, G, W, 30)
        torch.cuda.synchronize()
        n = (g.sqnorms(A, G, 30).double() + (0.0 if x is None else x)).sqrt().cpu()
        assert torch.allclose(torch.from_numpy(g.norms()).double(), n, rtol=1e-5)
    g.close()
