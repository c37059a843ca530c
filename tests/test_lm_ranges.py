"""Numbers that a C argument cannot hold are refused, not bent (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")

from random_gradient_projection_b200 import grape, lm  # noqa: E402
from test_lm_refusals import DISTILL, EMBED, HEAD, P, cpu, device, edit, lib, refused  # noqa: E402, F401


@pytest.mark.parametrize("tau", [1e-46, 1e-40, 2.0 ** -61, 2.0 ** 61, 1e39, 1e300, float("nan")])
def test_temperatures_without_a_factor_in_fp32_are_refused(lib, tau):
    """log2(e) / tau and tau^2 have to be finite and normal in fp32."""
    assert "temperature" in refused(grape.grape_distill_loss, *edit(DISTILL, tau=tau))


@pytest.mark.parametrize("scale", [1e39, -1e300])
def test_scales_that_overflow_fp32_are_refused(lib, scale):
    assert "scale" in refused(grape.grape_embed, *edit(EMBED, scale=scale))
    sums = dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=grape.GRAPE_BF16, scale=scale, ws=P, out=P, st=0)
    assert "scale" in refused(grape.grape_embed_sqnorms, *edit(sums))
    grad = dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=grape.GRAPE_BF16, scale=scale, w=0, ws=P, out=P, st=0)
    assert "scale" in refused(grape.grape_embed_grad, *edit(grad))


WRAP = [(1 << 32) + 5, (1 << 40) + 7, -(1 << 32) + 3]


@pytest.mark.parametrize("n", WRAP)
def test_sizes_beyond_an_int32_are_refused(lib, n):
    """(1 << 32) + 5 as an int32 would be 5: another vocabulary, and wrong results."""
    for call, args, keys in [
            (grape.grape_embed, EMBED, ("V", "d")), (grape.grape_head_loss, HEAD, ("V", "d")),
            (grape.grape_distill_loss, DISTILL, ("V", "K")),
            (grape.grape_embed_sqnorms, dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=1, scale=1.0, ws=P, out=P, st=0), ("B", "T", "V", "d")),
            (grape.grape_embed_grad, dict(order=P, B=2, T=3, V=10, d=8, G=P, dtype=1, scale=1.0, w=0, ws=P, out=P, st=0), ("B", "T", "V", "d")),
            (grape.grape_embed_order, dict(ids=P, id_bytes=8, n=4, V=10, order=P, st=0), ("V",)),
            (grape.grape_embed_order_bytes, dict(n=4, V=10), ("V",)),
            (grape.grape_embed_workspace_bytes, dict(B=2, T=3, V=10, d=8), ("B", "T", "V", "d")),
            (grape.grape_head_loss_bytes, dict(N=4, d=8, V=10, dtype=1, dH=True, dW=True), ("d", "V"))]:
        for k in keys:
            with pytest.raises(ValueError, match="int32"):
                call(*edit(args, **{k: n}))


@pytest.mark.parametrize("vocab", WRAP)
def test_a_vocabulary_beyond_an_int32_is_refused(lib, device, monkeypatch, vocab):
    monkeypatch.setattr(lm, "_tensor", lambda x, *a: x)
    with pytest.raises(ValueError, match="int32"):
        lm.embed_order(cpu(2, 3, dtype=torch.int64), vocab)
