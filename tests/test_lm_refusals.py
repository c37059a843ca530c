"""What the language-model entry points refuse, before any device work (no GPU needed): the C calls
by their arguments, the torch calls by their tensors."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from random_gradient_projection_b200 import grape, lm  # noqa: E402

P = 4096          # an aligned address that is never read: every call below is refused first
F32, BF16 = grape.GRAPE_F32, grape.GRAPE_BF16


@pytest.fixture(scope="module")
def lib():
    from random_gradient_projection_b200 import build
    build.build()
    return grape.lib()


def refused(call, *args):
    with pytest.raises(grape.GrapeError) as e:
        call(*args)
    assert e.value.code == grape.GRAPE_EINVAL, e.value
    return str(e.value)


def edit(args, **kw):
    return [kw.get(k, v) for k, v in args.items()]


EMBED = dict(table=P, tdt=F32, ids=P, id_bytes=8, n=4, V=10, d=8, scale=1.0, odt=BF16, out=P, st=0)


@pytest.mark.parametrize("kw,msg", [
    (dict(tdt=2), "dtypes"), (dict(odt=-1), "dtypes"), (dict(id_bytes=2), "id_bytes"), (dict(n=-1), "number of ids"),
    (dict(n=(1 << 30) + 1), "number of ids"), (dict(V=0), "vocab"), (dict(V=(1 << 30) + 1), "vocab"), (dict(d=0), "d must"), (dict(d=(1 << 20) + 1), "d must"), (dict(ids=0), "ids"),
    (dict(ids=P + 4), "ids"), (dict(table=0), "null"), (dict(out=P + 8), "aligned"), (dict(scale=float("nan")), "scale")])
def test_embed_refuses(lib, kw, msg):
    assert msg in refused(grape.grape_embed, *edit(EMBED, **kw))


def test_embed_of_nothing_is_a_no_op(lib):
    grape.grape_embed(*edit(EMBED, n=0, ids=0, table=0, out=0))


@pytest.mark.parametrize("kw,msg", [
    (dict(B=-1), "B, T"), (dict(T=-1), "B, T"), (dict(B=1 << 20, T=1 << 20), "2^30"), (dict(V=0), "vocab"), (dict(V=(1 << 30) + 1), "vocab"), (dict(d=0), "d must"), (dict(d=(1 << 20) + 1), "d must"),
    (dict(dtype=5), "dtype"), (dict(G=0), "Gout"), (dict(G=P + 2), "Gout"), (dict(ws=0), "workspace"),
    (dict(order=P + 4), "order"), (dict(out=0), "not be null"), (dict(scale=float("inf")), "scale")])
def test_embed_sums_refuse(lib, kw, msg):
    args = dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=BF16, scale=1.0, ws=P, out=P, st=0)
    assert msg in refused(grape.grape_embed_sqnorms, *edit(args, **kw))
    grad = dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=BF16, scale=1.0, w=0, ws=P, out=P, st=0)
    assert msg in refused(grape.grape_embed_grad, *edit(grad, **kw))


def test_embed_order_refuses(lib):
    assert "order" in refused(grape.grape_embed_order, P, 8, 4, 10, 0, 0)
    assert "order" in refused(grape.grape_embed_order, P, 8, 4, 10, P + 4, 0)
    assert "ids" in refused(grape.grape_embed_order, 0, 8, 4, 10, P, 0)
    assert "aligned" in refused(grape.grape_embed_grad, P, 2, 3, 10, 8, P, BF16, 1.0, P + 1, P, P, 0)


HEAD = dict(H=P, W=P, labels=P, id_bytes=8, w=0, N=4, d=8, V=10, dtype=BF16, ws=P, loss=P, dH=P, dW=P, st=0)


@pytest.mark.parametrize("kw,msg", [
    (dict(N=-1), "N must"), (dict(N=(1 << 30) + 1), "N must"), (dict(d=0), "d must"), (dict(V=0), "vocab"),
    (dict(d=(1 << 20) + 1), "d must"), (dict(V=(1 << 30) + 1), "vocab"), (dict(N=1 << 30, V=1 << 29), "too large"), (dict(dtype=3), "dtype"),
    (dict(id_bytes=1), "id_bytes"), (dict(labels=0), "ids"), (dict(labels=P + 2), "ids"), (dict(W=0), "W must"),
    (dict(W=P + 8), "W must"), (dict(H=0), "H and loss"), (dict(loss=0), "H and loss"), (dict(H=P + 2), "aligned"),
    (dict(dH=P + 4), "aligned"), (dict(dW=P + 4), "aligned"), (dict(ws=0), "workspace"), (dict(w=P + 2), "aligned")])
def test_head_refuses(lib, kw, msg):
    assert msg in refused(grape.grape_head_loss, *edit(HEAD, **kw))


DISTILL = dict(z=P, dtype=F32, N=4, V=10, idx=P, id_bytes=4, val=P, vdt=F32, K=3, w=0, tau=1.0, loss=P, out=P, st=0)


@pytest.mark.parametrize("kw,msg", [
    (dict(dtype=2), "dtypes"), (dict(vdt=2), "dtypes"), (dict(id_bytes=3), "id_bytes"), (dict(N=-1), "N must"),
    (dict(N=1 << 31), "N must"), (dict(V=0), "vocab"), (dict(V=(1 << 30) + 1), "vocab"), (dict(K=0), "K must"), (dict(K=1025), "K must"), (dict(tau=0.0), "temperature"),
    (dict(tau=-1.0), "temperature"), (dict(tau=float("inf")), "temperature"), (dict(z=0), "null"), (dict(out=0), "null"),
    (dict(z=P + 4), "16-byte"), (dict(idx=P + 2), "element size"), (dict(val=P + 2), "element size"), (dict(w=P + 1), "element size")])
def test_distill_refuses(lib, kw, msg):
    assert msg in refused(grape.grape_distill_loss, *edit(DISTILL, **kw))


def test_extra_norms_and_clip_pointer_validate_the_handle(lib):
    assert lib.grape_set_extra_sqnorms(None, None) == grape.GRAPE_EINVAL
    assert lib.grape_clip_ptr(None, ctypes.byref(ctypes.c_void_p())) == grape.GRAPE_EINVAL


def test_workspaces_are_as_documented(lib):
    """Sizes need no device, never shrink with the problem, and the head's piece stays bounded."""
    assert grape.grape_embed_order_bytes(0, 5) >= 1
    assert grape.grape_embed_order_bytes(1000, 5000) >= 4 * 1000 * 4 + 5000 // 8
    assert refused(grape.grape_embed_order_bytes, -1, 5) and refused(grape.grape_embed_workspace_bytes, 1, -1, 5, 8)
    small = grape.grape_head_loss_bytes(64, 256, 1000, BF16, True, False)
    assert small < grape.grape_head_loss_bytes(64, 256, 1000, BF16, True, True) + 1 < (8 << 20)
    # 8192 x 4096 x 128000: the logits alone would be 2 GiB in bf16
    big = grape.grape_head_loss_bytes(8192, 4096, 128000, BF16, True, True)
    rows, piece, sums, acc = 8192 * 4096 * 2, 256 << 20, 8192 * 500 * 8, 8192 * 4096 * 4
    assert big <= rows + piece + sums + acc + (1 << 20)
    assert refused(grape.grape_head_loss_bytes, 4, 0, 10, BF16, True, True)


def cpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype)


@pytest.fixture
def device(monkeypatch):
    """No GPU is asked for: tensors are on the host, and the current device is 0."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


@pytest.mark.parametrize("call,msg", [
    (lambda: lm.embed(cpu(4, 8), cpu(3, dtype=torch.int32)), "table: need a tensor on the current"),
    (lambda: lm.embed(cpu(4, 8)[:, ::2], cpu(3, dtype=torch.int32)), "contiguous"),
    (lambda: lm.embed(cpu(4), cpu(3, dtype=torch.int32)), "shape"),
    (lambda: lm.embed([1.0], cpu(3, dtype=torch.int32)), "torch tensor"),
    (lambda: lm.embed_order(cpu(3, dtype=torch.int64), 5), "shape"),
    (lambda: lm.embed_order(cpu(3, 2), 5), "need one of"),
    (lambda: lm.head_loss(cpu(3, 8), cpu(5, 8), cpu(3, dtype=torch.int64)), "current CUDA device"),
    (lambda: lm.distill_loss(cpu(3, 8).double().T, cpu(3, 1, dtype=torch.int32), cpu(3, 1)), "contiguous"),
])
def test_torch_calls_refuse(device, call, msg):
    with pytest.raises(ValueError, match=msg):
        call()


def test_torch_calls_check_shapes_and_types_against_each_other(monkeypatch, device):
    """With the device check out of the way: everything else is checked before an address is taken."""
    real = lm._tensor

    def host(x, what, dev, shape=None, dtypes=None):
        try:
            return real(x, what, dev, shape, dtypes)
        except ValueError as e:
            if "current CUDA device" not in str(e):
                raise
            return x
    monkeypatch.setattr(lm, "_tensor", host)
    H, W, t = cpu(3, 8), cpu(5, 8), cpu(3, dtype=torch.int64)
    bad = [
        lambda: lm.head_loss(H, cpu(5, 9), t), lambda: lm.head_loss(H, W.bfloat16(), t), lambda: lm.head_loss(H, W, t[:2]),
        lambda: lm.head_loss(H, W, t.float()), lambda: lm.head_loss(H, W, t, weights=cpu(2)),
        lambda: lm.head_loss(H, W, t, weights=cpu(3).double()), lambda: lm.head_loss(H.double(), W.double(), t),
        lambda: lm.head_loss(cpu(8), W, t), lambda: lm.head_loss(H.view(1, 3, 8), W, t),
        lambda: lm.distill_loss(H, t.view(3, 1), cpu(3, 2)), lambda: lm.distill_loss(H, t.view(3, 1), cpu(3, 1).half()),
        lambda: lm.distill_loss(H, t.view(3, 1)[:2], cpu(2, 1)), lambda: lm.distill_loss(H, t.view(3, 1), cpu(3, 1), out=cpu(3, 9)),
        lambda: lm.distill_loss(H, t.view(3, 1), cpu(3, 1), out=H.bfloat16()), lambda: lm.distill_loss(H, t.view(3, 1), cpu(3, 1), weights=cpu(4)),
        lambda: lm.embed(W, t, dtype="f16"), lambda: lm.embed(W.half(), t), lambda: lm.embed(cpu(0, 8), t),
        lambda: lm.embed_grad(lm.EmbedOrder(1, 3, 5, cpu(64, dtype=torch.uint8)), cpu(1, 4, 8)),
        lambda: lm.embed_grad(lm.EmbedOrder(1, 3, 5, cpu(64, dtype=torch.uint8)), cpu(1, 3, 8), weights=cpu(2)),
        lambda: lm.embed_sqnorms(lm.EmbedOrder(1, 3, 5, cpu(64, dtype=torch.uint8)), cpu(1, 3, 0)),
    ]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    z = cpu(40, 8)
    with pytest.raises(ValueError, match="overlap"):
        lm.distill_loss(z[:30], cpu(30, 1, dtype=torch.int32), cpu(30, 1), out=z[10:])
