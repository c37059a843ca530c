"""The language-model operators with the step they serve, as a private training step uses them:
embedding -> stack -> head loss, one clip over the stack's and the table's gradient, and calls on
streams, captured calls and shared handles (needs a B200)."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import GrapeStep, grape, lm  # noqa: E402


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def batch(B=6, T=40, d=256, V=700, seed=3, dtype=torch.bfloat16):
    g = rng(seed)
    table = (torch.randn(V, d, generator=g, device="cuda") / math.sqrt(d)).to(dtype)
    W = (torch.randn(d, d, generator=g, device="cuda") / math.sqrt(d)).float()
    ids = torch.randint(V, (B, T), generator=g, device="cuda")
    labels = torch.roll(ids, -1, 1)
    labels[:, -1] = -100
    labels[1, 20:] = -100            # a padded sample
    return table, W, ids, labels


def test_a_private_step_of_a_small_language_model():
    """table -> A -> one linear layer -> head (the table itself) -> loss; Gout of the layer, the
    table's gradient through the lookup, and one clip over both."""
    B, T, d, V, C = 6, 40, 256, 700, 0.5
    table, W, ids, labels = batch(B, T, d, V)
    scale = math.sqrt(d)
    weights = torch.zeros(B, T, device="cuda")
    live = labels >= 0
    weights[live] = (1.0 / live.sum(1).clamp(min=1).float())[:, None].expand(B, T)[live]   # a sample's mean

    A = lm.embed(table, ids, scale=scale)                       # B x T x d, bf16
    H = (A.float() @ W).to(torch.bfloat16)
    out = lm.head_loss(H, table, labels, weights=weights)
    Gout = out.dH
    dA = (Gout.float() @ W.T).to(torch.bfloat16)                # back through the layer
    order = lm.embed_order(ids, V)
    sq = lm.embed_sqnorms(order, dA, scale=scale)

    g = GrapeStep([(d, d)], r=128, C=C, sigma=0.0, seed=5, B=B, T=T)
    A2, G2, W2 = A.view(B * T, d), Gout.view(B * T, d), W.clone()
    alone = g.sqnorms([A2], [G2], 0).clone()
    g.set_extra_sqnorms(sq)
    g.step([A2], [G2], [W2], 0)
    c = g.clip_tensor()
    grad = lm.embed_grad(order, dA, weights=c, scale=scale)
    torch.cuda.synchronize()

    # the joint norm and its clip factor, from the two shares
    n = (alone.double() + sq.double()).sqrt()
    assert torch.allclose(torch.from_numpy(g.norms()).double(), n.cpu(), rtol=1e-5)
    want = torch.where(n > C, C / n, torch.ones_like(n))
    assert torch.allclose(c.double(), want, rtol=1e-5) and bool((want < 1).any())
    # every sample's table gradient, clipped: against the definition
    rsq, rgrad, bsq, bgrad = ref.embed_sums(ids, dA, V, scale, c)
    ref.check(sq, rsq, bsq, "sqnorms"), ref.check(grad, rgrad, bgrad, "grad")
    # the loss chain against torch's own graph in 64 bits
    E = table.double().requires_grad_(True)
    z = (H.double() @ E.T.detach())
    loss = torch.nn.functional.cross_entropy(z.view(-1, V), labels.view(-1), reduction="none", ignore_index=-100)
    assert torch.allclose(out.loss.double().view(-1), loss * weights.view(-1), rtol=1e-4, atol=1e-5)
    # without the share the step clips by the stack alone again
    g.set_extra_sqnorms(None)
    g.step([A2], [G2], [W2], 1)
    alone = g.sqnorms([A2], [G2], 1).double().sqrt()
    assert torch.allclose(torch.from_numpy(g.norms()).double(), alone.cpu(), rtol=1e-5)
    g.close()


@pytest.mark.parametrize("path", [grape.GRAPE_PATH_SIMT, grape.GRAPE_PATH_TC])
def test_extra_norms_in_graph_replays_and_on_both_paths(path):
    B, T, d = 4, 64, 256
    gen = rng(9)
    A = torch.randn(B * T, d, generator=gen, device="cuda").bfloat16()
    G = (0.02 * torch.randn(B * T, d, generator=gen, device="cuda")).bfloat16()
    W = torch.randn(d, d, generator=gen, device="cuda")
    extra = torch.zeros(B, device="cuda")
    g = GrapeStep([(d, d)], r=128, C=1.0, sigma=0.0, seed=1, B=B, T=T, path=path)
    g.set_graph(True)
    base = g.sqnorms([A], [G], 0).double()
    for step, x in enumerate((0.0, 3.0, 70.0)):     # the buffer is refilled between replays
        extra.fill_(x)
        g.set_extra_sqnorms(extra)
        g.step([A], [G], [W], step)
        torch.cuda.synchronize()
        n = (g.sqnorms([A], [G], step).double() + x).sqrt()
        assert torch.allclose(torch.from_numpy(g.norms()).double(), n.cpu(), rtol=1e-5)
        assert torch.allclose(g.clip_tensor().double(), torch.where(n > 1, 1 / n, torch.ones_like(n)), rtol=1e-5)
    assert base.isfinite().all()
    g.close()


def calls(seed):
    """One call of every operator on inputs of this seed: the inputs' tensors and a function."""
    g = rng(seed)
    ids = torch.randint(-1, 3000, (5, 700), generator=g, device="cuda")
    G = torch.randn(5, 700, 320, generator=g, device="cuda").bfloat16()
    table = torch.randn(3000, 320, generator=g, device="cuda")
    H = torch.randn(900, 320, generator=g, device="cuda").bfloat16()
    Wv = (torch.randn(3000, 320, generator=g, device="cuda") / 8).bfloat16()
    big = (torch.randn(41000, 512, generator=g, device="cuda") / 9).bfloat16()
    H2 = torch.randn(600, 512, generator=g, device="cuda").bfloat16()
    labels = torch.randint(-1, 3000, (900,), generator=g, device="cuda")
    labels2 = torch.randint(-1, 41000, (600,), generator=g, device="cuda")
    logits = torch.randn(300, 33000, generator=g, device="cuda").bfloat16()
    small = torch.randn(300, 3001, generator=g, device="cuda")
    idx = torch.randint(-1, 3000, (300, 20), generator=g, device="cuda")
    val = torch.randn(300, 20, generator=g, device="cuda")

    def run(stream=None):
        order = lm.embed_order(ids, 3000, stream=stream)
        head = lm.head_loss(H, Wv, labels, weight_grad=True, stream=stream)
        one = lm.head_loss(H2, big, labels2, stream=stream)          # one pass over the vocabulary
        return [lm.embed(table, ids, stream=stream), order.positions, lm.embed_sqnorms(order, G, stream=stream),
                lm.embed_grad(order, G, stream=stream), head.loss, head.dH, head.dW, one.loss, one.dH,
                *lm.distill_loss(logits, idx, val, stream=stream), *lm.distill_loss(small, idx, val, stream=stream)]
    return run


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_do_not_depend_on_the_stream_or_on_overlap():
    runs = [calls(1), calls(2)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for k in (0, 1):
            got[k].append(runs[k](stream=streams[k]))           # two at once, on streams of their own
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(same(g, want[k]) for g in got[k])
    with torch.cuda.stream(streams[0]):                         # or on the current one
        inside = runs[1]()
    torch.cuda.synchronize()
    assert same(inside, want[1])


def test_captured_calls_replay_and_share_nothing():
    """Two captures, replayed in turn and again, next to an eager call: each has its own workspace."""
    runs = [calls(4), calls(5)]
    want = [r() for r in runs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(r())
        graphs.append(g)
    side = torch.cuda.Stream()
    for _ in range(3):
        graphs[0].replay()
        with torch.cuda.stream(side):
            eager = runs[1]()
        graphs[1].replay()
    torch.cuda.synchronize()
    assert same(outs[0], want[0]) and same(outs[1], want[1]) and same(eager, want[1])


def test_a_step_follows_a_captured_loss_on_the_same_stream():
    table, W, ids, labels = batch()
    H = torch.randn(6, 40, 256, device="cuda").bfloat16()
    g = torch.cuda.CUDAGraph()
    lm.head_loss(H, table, labels)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = lm.head_loss(H, table, labels)
    H.copy_(torch.randn(6, 40, 256, device="cuda").bfloat16())   # new inputs for the replay
    g.replay()
    want = lm.head_loss(H, table, labels)
    torch.cuda.synchronize()
    assert torch.equal(out.dH, want.dH) and torch.equal(out.loss, want.loss)


def test_rows_behind_the_batch_stay_as_they_were():
    out = torch.full((80, 64), 7.0, device="cuda")
    table = torch.randn(30, 64, device="cuda")
    lm.embed(table, torch.zeros(70, dtype=torch.int32, device="cuda"), dtype="f32", out=out[:70])
    buf = torch.full((9, 5003), 7.0, device="cuda")
    z = torch.randn(8, 5003, device="cuda")
    idx = torch.zeros(8, 1, dtype=torch.int32, device="cuda")
    lm.distill_loss(z, idx, torch.zeros(8, 1, device="cuda"), out=buf[:8])
    torch.cuda.synchronize()
    assert bool((out[70:] == 7).all()) and bool((buf[8] == 7).all())
    assert not bool((out[:70] == 7).any())
