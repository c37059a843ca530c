"""Embedding, head loss and distillation against their 64-bit definitions (needs a B200)."""
import math

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import lm  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def tokens(g, shape, V, outside=0.0, dtype=torch.int64):
    n = math.prod(shape)
    t = (torch.exp(torch.rand(n, generator=g, device="cuda") * math.log(V + 1)).long() - 1).clamp(0, V - 1)
    if outside:
        bad = torch.rand(n, generator=g, device="cuda") < outside
        t[bad] = torch.where(torch.arange(n, device="cuda") % 2 == 0, -1, V + 3)[bad]
    return t.to(dtype).view(*shape)


# ---- embedding ------------------------------------------------------------------------

@pytest.mark.parametrize("n,V,d,tdt,odt,ids", [
    (1, 1, 1, "f32", "f32", torch.int32), (7, 50, 8, "bf16", "bf16", torch.int64),
    (64, 1000, 256, "f32", "bf16", torch.int64), (33, 77, 31, "bf16", "f32", torch.int32),
    (300, 513, 100, "f32", "bf16", torch.int64), (129, 300, 4096, "f32", "f32", torch.int32),
    (5, 40, 1030, "bf16", "bf16", torch.int32), (0, 10, 16, "f32", "bf16", torch.int64)])
def test_embed(n, V, d, tdt, odt, ids):
    g = rng(n + d)
    table = normal(g, V, d).to(DT[tdt])
    t = tokens(g, (n,), V, 0.2, ids)
    got = lm.embed(table, t, scale=3.7, dtype=odt)
    there = (t >= 0) & (t < V)
    want = table.float()[t.long().clamp(0, V - 1)] * torch.tensor(3.7, device="cuda")
    want = torch.where(there[:, None], want, torch.zeros_like(want)).to(DT[odt])
    assert got.dtype == DT[odt] and torch.equal(got, want)


def test_embed_masked_rows_are_zero_whatever_the_table_holds():
    table = torch.full((4, 16), math.nan, device="cuda")
    ids = torch.tensor([[-1, 4], [9, -7]], device="cuda")
    got = lm.embed(table, ids, dtype="f32")
    assert got.shape == (2, 2, 16) and torch.equal(got, torch.zeros_like(got))


@pytest.mark.parametrize("B,T,V,outside", [
    (1, 1, 1, 0), (1, 5, 2, 0.5), (3, 17, 255, 0.1), (2, 1000, 256, 0.1), (4, 700, 65535, 0), (1, 2048, 65536, 0.2),
    (3, 683, 50, 0), (5, 3001, 50265, 0.1), (8, 8192, 300, 0.05), (1, 70000, 100000, 0.9), (2, 0, 10, 0),
    (1, 4000, 1 << 29, 0)])
def test_embed_order_is_the_stable_sort(B, T, V, outside):
    ids = tokens(rng(B * T), (B, T), V, outside, torch.int32 if T % 2 else torch.int64)
    order = lm.embed_order(ids, V)
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < V), flat, torch.full_like(flat, V))
    want = torch.argsort(key, stable=True)
    assert torch.equal(order.positions.long(), want)
    assert torch.equal(order.tokens.long(), key[want])


@pytest.mark.parametrize("B,T,V,d,dt,outside", [
    (1, 1, 1, 1, "f32", 0), (2, 9, 5, 8, "bf16", 0.2), (4, 16, 1000, 256, "bf16", 0), (3, 50, 7, 300, "f32", 0.1),
    (16, 40, 300, 264, "bf16", 0.1), (5, 129, 33, 31, "bf16", 0.3), (2, 700, 1, 40, "f32", 0), (6, 511, 3, 100, "bf16", 0),
    (4, 2100, 50, 1024, "bf16", 0.05), (3, 100, 64, 4096, "f32", 0), (2, 3, 20, 16, "bf16", 1.0), (2, 0, 5, 8, "f32", 0),
    (0, 4, 5, 12, "bf16", 0), (1, 37000, 40, 64, "bf16", 0.01)])
@pytest.mark.parametrize("weighted", [False, True])
def test_embed_sums(B, T, V, d, dt, outside, weighted):
    g = rng(B * T + d)
    ids = tokens(g, (B, T), V, outside)
    G = normal(g, B, T, d).to(DT[dt])
    w = torch.rand(B, generator=g, device="cuda") if weighted else None
    G[(ids < 0) | (ids >= V)] = math.nan   # a dropped position's rows are not read
    order = lm.embed_order(ids, V)
    sq, grad = lm.embed_sqnorms(order, G, scale=1.7), lm.embed_grad(order, G, weights=w, scale=1.7)
    rsq, rgrad, bsq, bgrad = ref.embed_sums(ids, G, V, 1.7, w)
    print("of the bounds:", ref.check(sq, rsq, bsq, "sqnorms"), ref.check(grad, rgrad, bgrad, "grad"))
    again = lm.embed_grad(order, G, weights=w, scale=1.7), lm.embed_sqnorms(order, G, scale=1.7)
    assert torch.equal(again[0], grad) and torch.equal(again[1], sq)


# ---- distillation ------------------------------------------------------------------------

def distill_inputs(N, V, K, dt, seed=0, absent=0.2, vdt="f32", ids=torch.int32):
    g = rng(seed + N * V + K)
    logits = (2.0 * normal(g, N, V)).to(DT[dt])
    idx = torch.randint(V, (N, K), generator=g, device="cuda")
    idx[torch.rand(N, K, generator=g, device="cuda") < absent] = -1
    val = (3.0 * normal(g, N, K)).to(DT[vdt])
    return logits, idx.to(ids), val, 0.1 + torch.rand(N, generator=g, device="cuda")


@pytest.mark.parametrize("N,V,K,dt,tau", [
    (1, 1, 1, "f32", 1.0), (3, 7, 2, "bf16", 2.0), (5, 33, 40, "f32", 0.5), (16, 1000, 8, "f32", 1.0),
    (9, 4096, 5, "bf16", 1.0), (4, 4099, 64, "bf16", 1.5), (7, 8193, 1, "f32", 1.0), (6, 32768, 17, "bf16", 0.7),
    (5, 50265, 32, "bf16", 2.0), (3, 50265, 700, "f32", 1.0), (2, 131075, 128, "bf16", 1.0), (2, 70001, 1024, "f32", 4.0)])
def test_distill(N, V, K, dt, tau):
    logits, idx, val, w = distill_inputs(N, V, K, dt, vdt="bf16" if N % 2 else "f32",
                                         ids=torch.int64 if N % 3 else torch.int32)
    loss, G = lm.distill_loss(logits, idx, val, weights=w, temperature=tau)
    rl, rG, bl, bG = ref.distill(logits, idx, val, w, tau)
    print("of the bounds:", ref.check(loss, rl, bl, "loss"), ref.check(G, rG, bG, "Gout"))
    # in place, and without weights
    loss1, G1 = lm.distill_loss(logits, idx, val, temperature=tau)
    inplace = logits.clone()
    loss2, G2 = lm.distill_loss(inplace, idx, val, temperature=tau, out=inplace)
    assert G2.data_ptr() == inplace.data_ptr() and torch.equal(G1, G2) and torch.equal(loss1, loss2)
    rl, rG, bl, bG = ref.distill(logits, idx, val, None, tau)
    ref.check(loss1, rl, bl, "loss"), ref.check(G1, rG, bG, "Gout")


@pytest.mark.parametrize("N,V,K,dt", [
    (700, 20001, 40, "bf16"), (700, 16385, 64, "bf16"), (400, 60001, 100, "f32"), (500, 33000, 128, "f32"),
    (330, 110003, 9, "bf16"), (900, 9001, 130, "f32"), (320, 20001, 129, "bf16")])
def test_distill_many_rows_per_block(N, V, K, dt):
    """Several rows in turn on every SM, some of them without weight or teacher; in place too."""
    logits, idx, val, w = distill_inputs(N, V, K, dt)
    w[::5] = 0.0
    w[7:40] = 0.0
    logits[w == 0] = math.nan
    idx[3::11] = -1
    loss, G = lm.distill_loss(logits, idx, val, weights=w, temperature=1.3)
    for a in range(0, N, 100):
        rl, rG, bl, bG = ref.distill(logits[a:a + 100], idx[a:a + 100], val[a:a + 100], w[a:a + 100], 1.3)
        ref.check(loss[a:a + 100], rl, bl, "loss"), ref.check(G[a:a + 100], rG, bG, "Gout")
    for _ in range(3):
        inplace = logits.clone()
        again = lm.distill_loss(inplace, idx, val, weights=w, temperature=1.3, out=inplace)
        assert torch.equal(again[0], loss) and torch.equal(inplace, G)


@pytest.mark.parametrize("V", [5000, 40001])
def test_distill_masked_rows_and_infinities(V):
    logits, idx, val, w = distill_inputs(8, V, 6, "bf16", absent=0.0)
    w[1] = 0.0
    logits[1] = math.nan                      # no weight: not read
    idx[2] = torch.tensor([-1, V, -9, V + 1000, -1, -2], device="cuda")
    logits[2] = math.inf                      # no valid entry
    logits[3, 10:4000] = -math.inf            # a masked vocabulary
    idx[3] = torch.arange(6, device="cuda")
    logits[4] = torch.finfo(torch.bfloat16).min
    logits[4, 7], logits[4, 9] = 1.0, 2.0     # all but two at the type's lowest value
    idx[4] = torch.tensor([7, 9, -1, -1, -1, -1], device="cuda")
    val[5, 1:] = -math.inf                    # one entry holds the whole mass
    logits[6, 3] = math.nan                   # a live row's NaN is the formula's
    loss, G = lm.distill_loss(logits, idx, val, weights=w)
    rl, rG, bl, bG = ref.distill(logits, idx, val, w, 1.0)
    ref.check(loss, rl, bl, "loss"), ref.check(G, rG, bG, "Gout")
    for n in (1, 2):
        assert float(loss[n]) == 0.0 and not G[n].any()
    assert loss[6].isnan() and G[6].isnan().all() and G[[0, 3, 4, 5, 7]].isfinite().all()


@pytest.mark.parametrize("V", [300, 30000])
def test_distill_the_same_index_twice(V):
    logits, _, val, _ = distill_inputs(4, V, 5, "f32")
    idx = torch.tensor([[3, 3, 7, 3, 7], [0, V - 1, 0, 1, 2], [5, 5, 5, 5, 5], [9, -1, 9, V, 9]], device="cuda")
    loss, G = lm.distill_loss(logits, idx, val)
    rl, rG, bl, bG = ref.distill(logits, idx, val, None, 1.0)
    ref.check(loss, rl, bl, "loss"), ref.check(G, rG, bG, "Gout")


def test_distill_the_same_index_in_several_warps():
    logits, idx, val, w = distill_inputs(300, 40000, 100, "bf16", absent=0.1)
    idx[:, 70:] = idx[:, :30]                 # every index again, far behind its first place
    idx[5] = 17
    loss, G = lm.distill_loss(logits, idx, val, weights=w)
    rl, rG, bl, bG = ref.distill(logits, idx, val, w, 1.0)
    ref.check(loss, rl, bl, "loss"), ref.check(G, rG, bG, "Gout")


def test_distill_one_entry_is_a_hard_label():
    logits, idx, val, w = distill_inputs(12, 999, 1, "f32", absent=0.0)
    loss, G = lm.distill_loss(logits, idx, val, weights=w)
    z = logits.double()
    want = -w.double() * torch.log_softmax(z, 1).gather(1, idx.long())[:, 0]
    assert torch.allclose(loss.double(), want, rtol=1e-5, atol=1e-5)


# ---- vocabulary head ------------------------------------------------------------------------

def head_inputs(N, d, V, dt, seed=0, outside=0.0, ids=torch.int64, weighted=True):
    g = rng(seed + N * d + V)
    W = normal(g, V, d) * (2.5 / math.sqrt(d))
    labels = tokens(g, (N,), V, outside)
    lean = 3.0 * torch.rand(N, 1, generator=g, device="cuda") / 2.5
    H = (normal(g, N, d) + lean * W[labels.clamp(0, V - 1)]).to(DT[dt])
    w = 0.1 + torch.rand(N, generator=g, device="cuda") if weighted else None
    return H, W.to(DT[dt]), labels.to(ids), w


def check_head(H, W, labels, w, **kw):
    got = lm.head_loss(H, W, labels, weights=w, grad=True, weight_grad=True, **kw)
    r = ref.head(H, W, labels, w)
    bl, bH, bW = ref.head_bounds(r, H.dtype)
    print("of the bounds:", ref.check(got.loss, r["loss"], bl.view(r["loss"].shape), "loss"),
          ref.check(got.dH, r["dH"], bH.view(r["dH"].shape), "dH"), ref.check(got.dW, r["dW"], bW, "dW"))
    return got


HEAD = [(64, 64, 256), (1, 8, 1), (1, 64, 1000), (256, 256, 512), (300, 264, 1000), (257, 72, 2049), (130, 1024, 700),
        (512, 512, 5003), (77, 100, 333), (33, 31, 257), (1000, 136, 12000), (1024, 64, 600), (1025, 72, 600)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("N,d,V", HEAD)
def test_head(N, d, V, dt):
    H, W, labels, w = head_inputs(N, d, V, dt, outside=0.1 if N > 100 else 0.0)
    got = check_head(H, W, labels, w)
    # each output by itself is the same
    only = lm.head_loss(H, W, labels, weights=w, grad=False)
    assert only.dH is None and only.dW is None and torch.equal(only.loss, got.loss)
    assert torch.equal(lm.head_loss(H, W, labels, weights=w).dH, got.dH)
    assert torch.equal(lm.head_loss(H, W, labels, weights=w, grad=False, weight_grad=True).dW, got.dW)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_head_masked_rows_cost_nothing_and_reach_nothing(dt):
    H, W, labels, w = head_inputs(700, 128, 600, dt, outside=0.5, ids=torch.int32)
    w[::7] = 0.0
    dropped = (labels < 0) | (labels >= 600) | (w == 0)
    H[dropped] = math.nan
    got = check_head(H, W, labels, w)
    assert not got.loss[dropped].any() and not got.dH[dropped].any()
    clean = torch.where(dropped[:, None], torch.zeros_like(H), H)
    same = lm.head_loss(clean, W, labels, weights=w, weight_grad=True)
    for a, b in zip(got, same):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_head_without_a_live_row(dt):
    H, W, labels, _ = head_inputs(2000, 512, 9000, dt)     # of a size for one pass
    got = lm.head_loss(H, W, torch.full_like(labels, -100))
    assert not got.loss.any() and not got.dH.any()
    H, W, labels, _ = head_inputs(40, 64, 300, dt)
    got = lm.head_loss(H, W, torch.full_like(labels, -100), weight_grad=True)
    assert not got.loss.any() and not got.dH.any() and not got.dW.any()
    got = lm.head_loss(H[:0], W, labels[:0], weight_grad=True)
    assert got.loss.shape == (0,) and got.dH.shape == (0, 64) and got.dW.shape == W.shape and not got.dW.any()


def test_head_in_several_pieces_of_the_vocabulary():
    """More rows and columns than one piece of the logits' gradient holds."""
    H, W, labels, w = head_inputs(16500, 64, 9000, "bf16", outside=0.02)
    check_head(H, W, labels, w)


def test_head_infinite_and_large_logits():
    H, W, labels, _ = head_inputs(64, 64, 512, "bf16", weighted=False)
    H *= 40.0                                  # logits of some hundreds: nearly one-hot rows
    check_head(H, W, labels, None)
    H[5] = math.nan                            # a live row's NaN is its own in loss and dH
    got = lm.head_loss(H, W, labels)
    assert got.loss[5].isnan() and got.dH[5].isnan().all()
    keep = torch.arange(64, device="cuda") != 5
    assert got.loss[keep].isfinite().all() and got.dH[keep].isfinite().all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_head_input_gradient_in_one_pass(dt):
    """The gradient of H alone, of a size that takes one pass over the vocabulary, for usual rows and
    where one row, or every row, has a loss too large for its reference."""
    H, W, labels, w = head_inputs(520, 512, 40001, dt, outside=0.05)
    w[3] = 0.0
    H[3] = math.nan
    for scale in (None, 5, "all"):
        if scale == 5:      # one row far from its label: a loss of some hundreds
            H[7] = (-60.0 * W[labels[7].clamp(min=0)].float()).to(H.dtype)
        if scale == "all":
            H = (H.float() * 50.0).to(H.dtype)
        got = lm.head_loss(H, W, labels, weights=w)
        r = ref.head(H, W, labels, w)
        bl, bH, _ = ref.head_bounds(r, H.dtype)
        print("of the bounds:", float(r["loss"].max()), ref.check(got.loss, r["loss"], bl, "loss"),
              ref.check(got.dH, r["dH"], bH, "dH"))
        only = lm.head_loss(H, W, labels, weights=w, grad=False).loss
        assert torch.allclose(got.loss, only, rtol=2e-5, atol=2e-5)


def test_head_one_pass_infinite_logits():
    H, W, labels, _ = head_inputs(300, 512, 70000, "bf16", weighted=False)
    H[5] = math.nan                            # the row's own NaN
    W[69000] = 0.0
    W[69000, 0] = math.inf                     # logits of +inf or -inf, by the sign of h
    H[:, 0] = -1.0
    labels[labels == 69000] = 0
    got = lm.head_loss(H, W, labels)
    keep = torch.arange(300, device="cuda") != 5
    Wf = W.clone()
    Wf[69000] = 0.0
    z = H[keep].double() @ Wf.double().T
    z[:, 69000] = -math.inf
    want = -torch.log_softmax(z, 1).gather(1, labels[keep][:, None])[:, 0]
    assert got.loss[5].isnan() and torch.allclose(got.loss[keep].double(), want, rtol=1e-5, atol=1e-5)
    H[9, 0] = 1.0                              # one row meets +inf: no softmax
    got = lm.head_loss(H, W, labels)
    keep[9] = False
    want = -torch.log_softmax(z, 1).gather(1, labels[torch.arange(300, device="cuda") != 5][:, None])[:, 0]
    assert got.loss[9].isnan() or float(got.loss[9]) == math.inf
    sel = keep[torch.arange(300, device="cuda") != 5]
    assert torch.allclose(got.loss[keep].double(), want[sel], rtol=1e-5, atol=1e-5)


def test_head_gradients_against_differences():
    H, W, labels, w = head_inputs(20, 48, 130, "f32")
    got = lm.head_loss(H, W, labels, weights=w, weight_grad=True)
    g = rng(5)
    for x, dx in ((H, got.dH), (W, got.dW)):
        u = normal(g, *x.shape)
        eps = 1e-2
        up, down = (lm.head_loss(*((x + s * eps * u, W) if x is H else (H, x + s * eps * u)), labels, weights=w,
                                 grad=False).loss.double().sum() for s in (1, -1))
        want = float((u.double() * dx.double()).sum())
        # the third derivative's share is about eps^2, the losses' rounding about 1e-5 / eps
        assert abs(float(up - down) / (2 * eps) - want) <= 5e-3 * (1 + float((u.double() * dx.double()).abs().sum()))
