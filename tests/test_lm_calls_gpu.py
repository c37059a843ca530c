"""Calls of the language-model entry points that the documentation allows, as a program may make them:
the first call of a process inside a capture, stream handles, buffers past 2^31 elements (needs a B200)."""
import subprocess
import sys

import pytest
from conftest import ROOT

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import lm_reference as ref  # noqa: E402
from random_gradient_projection_b200 import lm  # noqa: E402

FIRST = """
import torch
from random_gradient_projection_b200 import lm
B, T, V, d = 4, 9000, 40000, 256
torch.manual_seed(0)
ids = torch.randint(V, (B, T), device="cuda")
G = torch.randn(B, T, d, device="cuda").bfloat16()
table = torch.randn(V, d, device="cuda")
H, W = torch.randn(300, d, device="cuda").bfloat16(), torch.randn(V, d, device="cuda").bfloat16()
labels = torch.randint(V, (300,), device="cuda")
z, idx, val = torch.randn(20, V, device="cuda"), torch.randint(V, (20, 9), device="cuda"), torch.randn(20, 9, device="cuda")
def run():
    order = lm.embed_order(ids, V)
    head, both = lm.head_loss(H, W, labels), lm.head_loss(H.float(), W.float(), labels, weight_grad=True)
    return [lm.embed(table, ids), order.positions, lm.embed_sqnorms(order, G), lm.embed_grad(order, G), *head[:2], *both,
            *lm.distill_loss(z, idx, val), *lm.distill_loss(z[:, :700].contiguous(), idx % 700, val)]
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = run()          # nothing of the library has run before
graph.replay()
want = run()
torch.cuda.synchronize()
print(all(torch.equal(a, b) for a, b in zip(got, want)), len(got))
"""


def test_the_first_call_of_a_process_may_be_captured():
    out = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    assert out.stdout.split() == ["True", "13"]


def test_streams_by_object_and_by_handle():
    table = torch.randn(50, 64, device="cuda")
    ids = torch.randint(-1, 50, (3, 40), device="cuda")
    want = lm.embed(table, ids)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream, 0, torch.cuda.default_stream()):
        got = lm.embed(table, ids, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_distillation_past_two_to_the_31_elements():
    N, V = 17000, 128001
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_()
    idx = torch.randint(V, (N, 4), device="cuda")
    val = torch.randn(N, 4, device="cuda")
    assert z.numel() > 2 ** 31
    last = slice(N - 40, N)
    keep = z[last].clone()
    loss, G = lm.distill_loss(z, idx, val, out=z)
    rl, rG, bl, bG = ref.distill(keep, idx[last], val[last], None, 1.0)
    ref.check(loss[last], rl, bl, "loss"), ref.check(G[last], rG, bG, "Gout")
    assert loss.isfinite().all()


def test_short_distillation_rows_past_two_to_the_31_elements():
    N, V = 2300000, 1000
    z = torch.empty(N, V, dtype=torch.bfloat16, device="cuda").normal_()
    idx = torch.randint(V, (N, 2), device="cuda")
    val = torch.randn(N, 2, device="cuda")
    last = slice(N - 300, N)
    keep = z[last].clone()
    loss, G = lm.distill_loss(z, idx, val, out=z)
    rl, rG, bl, bG = ref.distill(keep, idx[last], val[last], None, 1.0)
    ref.check(loss[last], rl, bl, "loss"), ref.check(G[last], rG, bG, "Gout")


def test_embedding_past_two_to_the_31_elements():
    """The table, its gradient and Gout each beyond 2^31 elements."""
    V, d, B, T = 530000, 4096, 2, 263000
    ids = torch.randint(V, (B, T), device="cuda")
    ids[0, :3], ids[1, -3:] = V - 1, V - 1
    G = torch.empty(B, T, d, dtype=torch.bfloat16, device="cuda").normal_()
    assert V * d > 2 ** 31 and G.numel() > 2 ** 31
    order = lm.embed_order(ids, V)
    grad, sq = lm.embed_grad(order, G), lm.embed_sqnorms(order, G)
    at = [(0, 0), (0, 1), (0, 2), (1, T - 3), (1, T - 2), (1, T - 1)]
    more = ((ids == V - 1).nonzero()).tolist()
    rows = torch.stack([G[b, t] for b, t in {tuple(x) for x in more} | set(at)]).double()
    bound = (rows.shape[0] + 4) * ref.U32 * rows.abs().sum(0) + 1e-37
    assert bool(((grad[V - 1].double() - rows.sum(0)).abs() <= bound).all())
    # 1.1e9 squares a sample; each of about 65000 pairs of equal tokens adds twice a product of N(0, 4096):
    # 3e4 together, 3e-5 of the sum
    n = torch.stack([G[b].float().square().sum(dtype=torch.float64) for b in range(B)])
    assert torch.allclose(sq.double(), n, rtol=1e-3)
    table = grad
    out = lm.embed(table, torch.tensor([V - 1, 0, V - 2], device="cuda"), dtype="f32")
    assert torch.equal(out, table[[V - 1, 0, V - 2]])
    del grad, table, out
    big = lm.embed(torch.randn(100, d, device="cuda"), ids % 100)         # the output beyond 2^31 too
    assert big.numel() > 2 ** 31 and bool((big[1, -1] == big[0, 0]).all()) == bool(ids[1, -1] % 100 == ids[0, 0] % 100)


@pytest.mark.parametrize("N,d,V", [(525000, 4096, 40), (560000, 64, 4000)])
def test_head_past_two_to_the_31_elements(N, d, V):
    """H and dH, or the logits' gradient in the workspace, beyond 2^31 elements."""
    H = torch.empty(N, d, dtype=torch.bfloat16, device="cuda").normal_()
    W = (torch.randn(V, d, device="cuda") / d ** 0.5).bfloat16()
    labels = torch.randint(V, (N,), device="cuda")
    labels[5] = -1
    assert max(N * d, N * V) > 2 ** 31
    got = lm.head_loss(H, W, labels)
    for part in (slice(0, 300), slice(N - 300, N)):
        r = ref.head(H[part], W, labels[part], None)
        bl, bH, _ = ref.head_bounds(r, H.dtype)
        ref.check(got.loss[part], r["loss"], bl, "loss"), ref.check(got.dH[part], r["dH"], bH, "dH")
