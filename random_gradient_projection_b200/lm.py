"""The two ends of a language model around the stack of linear layers, for torch tensors.

``embed`` gives the first layer's A, ``head_loss`` and ``distill_loss`` the losses and the
last Gout, and ``embed_order`` / ``embed_sqnorms`` / ``embed_grad`` the embedding table's
gradient per sample: its squared norm, which joins the layers' before the clip, and the
clipped sum.  Formulas and layouts are in include/grape.h.

Every call checks its tensors and raises ValueError for a wrong size, type, device or
stride before the library sees an address; outputs and workspaces come from torch's allocator
on the stream the call runs on, so a call may be captured into a CUDA graph, and calls on
different streams share nothing.
"""
from __future__ import annotations

import contextlib
from typing import NamedTuple, Optional

from . import grape
from .grape import GRAPE_BF16, GRAPE_F32


class HeadLoss(NamedTuple):
    loss: "torch.Tensor"            # noqa: F821  per row, weighted
    dH: Optional["torch.Tensor"]    # noqa: F821
    dW: Optional["torch.Tensor"]    # noqa: F821


class EmbedOrder:
    """A batch's tokens sorted by (token, position); of ``embed_order``."""

    def __init__(self, B: int, T: int, vocab: int, buffer):
        self.B, self.T, self.vocab, self.buffer = B, T, vocab, buffer

    def _list(self, k: int):
        import torch
        n = self.B * self.T
        start = k * ((n * 4 + 255) // 256 * 256)
        return self.buffer[start:start + 4 * n].view(torch.int32)

    @property
    def positions(self):
        """Positions (row-major in B x T) in the order of their tokens; dropped ones last."""
        return self._list(0)

    @property
    def tokens(self):
        """The tokens in that order; ``vocab`` for the dropped ones."""
        return self._list(1)


def _dtype(x, what: str) -> int:
    import torch
    t = getattr(x, "dtype", None)
    if t == torch.float32:
        return GRAPE_F32
    if t == torch.bfloat16:
        return GRAPE_BF16
    raise ValueError(f"{what}: need a float32 or bfloat16 tensor, got {t or type(x).__name__}")


def _tensor(x, what: str, shape=None, dtypes=None):
    """A contiguous CUDA tensor on the current device, of this shape (None: any size there)."""
    import torch
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{what}: need a torch tensor, got {type(x).__name__}")
    if dtypes is not None and x.dtype not in dtypes:
        raise ValueError(f"{what}: need one of {[str(t) for t in dtypes]}, got {x.dtype}")
    if shape is not None and (x.dim() != len(shape) or any(s is not None and s != g for s, g in zip(shape, x.shape))):
        raise ValueError(f"{what}: need shape {tuple('any' if s is None else s for s in shape)}, got {tuple(x.shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: need a contiguous tensor, got strides {x.stride()}")
    if not x.is_cuda or x.device.index != torch.cuda.current_device():
        raise ValueError(f"{what}: need a tensor on the current CUDA device, got one on {x.device}")
    return x


def _ids(x, what: str, shape=None) -> int:
    import torch
    _tensor(x, what, shape, (torch.int32, torch.int64))
    return x.element_size()


def _weights(x, n: int, what: str = "weights"):
    import torch
    if x is not None:
        _tensor(x, what, (n,), (torch.float32,))


def _out(x, shape, dtype, what: str):
    """`x` checked, or a new tensor (on the stream that is current)."""
    import torch
    if x is None:
        return torch.empty(shape, dtype=dtype, device="cuda")
    return _tensor(x, what, shape, (dtype,))


def _torch_dtype(dtype):
    import torch
    if dtype in ("bf16", GRAPE_BF16, torch.bfloat16):
        return torch.bfloat16
    if dtype in ("f32", GRAPE_F32, torch.float32):
        return torch.float32
    raise ValueError(f"dtype: need 'bf16' or 'f32', got {dtype!r}")


@contextlib.contextmanager
def _on(stream):
    """Makes `stream` (None: the current one) current, so that what is allocated belongs to it,
    and yields its handle."""
    import torch
    if stream is None:
        yield torch.cuda.current_stream().cuda_stream
        return
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    with torch.cuda.stream(torch.cuda.ExternalStream(handle)):
        yield handle


def _bytes(n: int):
    import torch
    return torch.empty(max(int(n), 1), dtype=torch.uint8, device="cuda")


def embed(table, ids, scale: float = 1.0, dtype="bf16", out=None, stream=None):
    """``scale * table[ids]`` in ``dtype``: ids of any shape, rows of ids outside the table zero."""
    _tensor(table, "table", (None, None))
    tdt = _dtype(table, "table")
    id_bytes = _ids(ids, "ids")
    V, d = table.shape
    if V < 1 or d < 1:
        raise ValueError(f"table: need at least one row and one column, got {tuple(table.shape)}")
    odt = _torch_dtype(dtype)
    with _on(stream) as st:
        out = _out(out, (*ids.shape, d), odt, "out")
        grape.grape_embed(table, tdt, ids, id_bytes, ids.numel(), V, d, float(scale), _dtype(out, "out"), out, st)
    return out


def embed_order(ids, vocab: int, stream=None) -> EmbedOrder:
    """The order of a batch's ids (B x T), for ``embed_sqnorms`` and ``embed_grad``."""
    id_bytes = _ids(ids, "ids", (None, None))
    B, T = ids.shape
    n = grape.grape_embed_order_bytes(B * T, int(vocab))
    with _on(stream) as st:
        order = EmbedOrder(B, T, int(vocab), _bytes(n))
        grape.grape_embed_order(ids, id_bytes, B * T, order.vocab, order.buffer, st)
    return order


def _embed_args(order: EmbedOrder, Gout):
    import torch
    _tensor(Gout, "Gout", (order.B, order.T, None))
    _tensor(order.buffer, "order", None, (torch.uint8,))
    d = Gout.shape[2]
    if d < 1:
        raise ValueError(f"Gout: need at least one column, got {tuple(Gout.shape)}")
    return _dtype(Gout, "Gout"), d, grape.grape_embed_workspace_bytes(order.B, order.T, order.vocab, d)


def embed_sqnorms(order: EmbedOrder, Gout, scale: float = 1.0, out=None, stream=None):
    """Each sample's squared norm of the embedding table's gradient (B floats)."""
    import torch
    dt, d, n = _embed_args(order, Gout)
    with _on(stream) as st:
        out = _out(out, (order.B,), torch.float32, "out")
        grape.grape_embed_sqnorms(order.buffer, order.B, order.T, order.vocab, d, Gout, dt, float(scale), _bytes(n),
                                  out, st)
    return out


def embed_grad(order: EmbedOrder, Gout, weights=None, scale: float = 1.0, out=None, stream=None):
    """The embedding table's gradient (vocab x d, fp32), every sample's share times its weight."""
    import torch
    dt, d, n = _embed_args(order, Gout)
    _weights(weights, order.B)
    with _on(stream) as st:
        out = _out(out, (order.vocab, d), torch.float32, "out")
        grape.grape_embed_grad(order.buffer, order.B, order.T, order.vocab, d, Gout, dt, float(scale), weights,
                               _bytes(n), out, st)
    return out


def head_loss(H, W, labels, weights=None, grad: bool = True, weight_grad: bool = False, stream=None) -> HeadLoss:
    """Softmax cross entropy of the head ``H @ W.T`` without its logits: losses, and on request
    the gradients of H (``grad``) and of W (``weight_grad``), in H's type.

    H is N x d or B x T x d, labels N or B x T; a label outside the vocabulary, or weight 0,
    drops the token."""
    import torch
    if not isinstance(H, torch.Tensor) or H.dim() not in (2, 3):
        raise ValueError("H: need a tensor of 2 or 3 dimensions")
    _tensor(H, "H")
    dt = _dtype(H, "H")
    rows, d = H.shape[:-1], H.shape[-1]
    N = H.numel() // d if d else 0
    _tensor(W, "W", (None, d), (H.dtype,))
    V = W.shape[0]
    id_bytes = _ids(labels, "labels", rows)
    if weights is not None:
        _tensor(weights, "weights", rows, (torch.float32,))
    n = grape.grape_head_loss_bytes(N, d, V, dt, bool(grad), bool(weight_grad))
    with _on(stream) as st:
        loss = torch.empty(rows, dtype=torch.float32, device="cuda")
        dH = torch.empty_like(H) if grad else None
        dW = torch.empty_like(W) if weight_grad else None
        grape.grape_head_loss(H, W, labels, id_bytes, weights, N, d, V, dt, _bytes(n), loss, dH, dW, st)
    return HeadLoss(loss, dH, dW)


def distill_loss(logits, indices, values, weights=None, temperature: float = 1.0, out=None, stream=None):
    """(losses, Gout) of distillation from a teacher's top logits: ``values`` at vocabulary
    numbers ``indices`` (..., K), a negative index for an absent entry.

    ``out`` may be ``logits`` itself: Gout then replaces them."""
    import torch
    if not isinstance(logits, torch.Tensor) or logits.dim() not in (2, 3):
        raise ValueError("logits: need a tensor of 2 or 3 dimensions")
    _tensor(logits, "logits")
    dt = _dtype(logits, "logits")
    rows, V = logits.shape[:-1], logits.shape[-1]
    id_bytes = _ids(indices, "indices", (*rows, None))
    K = indices.shape[-1]
    _tensor(values, "values", (*rows, K))
    vdt = _dtype(values, "values")
    if weights is not None:
        _tensor(weights, "weights", rows, (torch.float32,))
    if out is not None:
        _tensor(out, "out", logits.shape, (logits.dtype,))
        a, b, size = logits.data_ptr(), out.data_ptr(), logits.numel() * logits.element_size()
        if a != b and abs(a - b) < size:
            raise ValueError("out: may be the logits themselves, but not overlap them in part")
    N = logits.numel() // V if V else 0
    with _on(stream) as st:
        out = torch.empty_like(logits) if out is None else out
        loss = torch.empty(rows, dtype=torch.float32, device="cuda")
        grape.grape_distill_loss(logits, dt, N, V, indices, id_bytes, values, vdt, K, weights, float(temperature),
                                 loss, out, st)
    return loss, out
