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
