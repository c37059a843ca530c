"""The two ends of a language model around the stack of linear layers, for torch tensors.

``embed`` gives the first layer's A, ``head_loss`` and ``distill_loss`` the losses and the
last Gout, and ``embed_order`` / ``embed_sqnorms`` / ``embed_grad`` the embedding table's
gradient per sample: its squared norm, which joins the layers' before the clip, and the
clipped sum.  Formulas and layouts are in include/grape.h.

Every call checks its tensors and raises ValueError for a wrong size, type, device or
stride before the library sees an address; what the library itself refuses (addresses off the
16-byte rule, numbers outside their range) raises GrapeError.  Outputs and workspaces come from
torch's allocator on the stream the call runs on, so a call may be captured into a CUDA graph, and
calls on different streams share nothing.  Inputs (an EmbedOrder among them) that were made on
another stream than the call's are the caller's to order and to keep, as with any torch operation.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

from . import grape
from .grape import GRAPE_BF16, GRAPE_F32

try:
    import torch
except ImportError:   # the package itself does not need it
    torch = None


class HeadLoss(NamedTuple):
    loss: "torch.Tensor"            # per row, weighted
    dH: Optional["torch.Tensor"]
    dW: Optional["torch.Tensor"]


class EmbedOrder:
    """A batch's tokens sorted by (token, position); of ``embed_order``."""

    def __init__(self, B: int, T: int, vocab: int, buffer):
        self.B, self.T, self.vocab, self.buffer = B, T, vocab, buffer

    def _list(self, k: int):
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


# ---- checks, of every tensor and before any address is passed on --------------------------

def _dtype(x, what: str) -> int:
    t = x.dtype
    if t is torch.float32:
        return GRAPE_F32
    if t is torch.bfloat16:
        return GRAPE_BF16
    raise ValueError(f"{what}: need a float32 or bfloat16 tensor, got {t}")


def _tensor(x, what: str, dev: int, shape=None, dtypes=None):
    """A contiguous CUDA tensor on device `dev` (the current one), of this shape (None: any size)."""
    if not isinstance(x, torch.Tensor):
        raise ValueError(f"{what}: need a torch tensor, got {type(x).__name__}")
    if dtypes is not None and x.dtype not in dtypes:
        raise ValueError(f"{what}: need one of {[str(t) for t in dtypes]}, got {x.dtype}")
    if shape is not None and x.shape != shape:
        got = x.shape
        if len(got) != len(shape) or any(w is not None and w != n for w, n in zip(shape, got)):
            raise ValueError(f"{what}: need shape {tuple('any' if w is None else w for w in shape)}, got {tuple(got)}")
    if not x.is_contiguous():
        raise ValueError(f"{what}: need a contiguous tensor, got strides {x.stride()}")
    if x.get_device() != dev or not x.is_cuda:
        raise ValueError(f"{what}: need a tensor on the current CUDA device, got one on {x.device}")
    return x


def _ids(x, what: str, dev: int, shape=None) -> int:
    _tensor(x, what, dev, shape, (torch.int32, torch.int64))
    return 4 if x.dtype is torch.int32 else 8


def _weights(x, dev: int, shape):
    """Address of the weights (0: none)."""
    if x is None:
        return 0
    return _tensor(x, "weights", dev, shape, (torch.float32,)).data_ptr()


def _out(x, shape, dtype, dev: int, like):
    """`x` checked, or a new tensor beside `like` (on the stream that is current)."""
    return like.new_empty(shape, dtype=dtype) if x is None else _tensor(x, "out", dev, shape, (dtype,))


def _torch_dtype(dtype):
    if dtype in ("bf16", GRAPE_BF16, torch.bfloat16):
        return torch.bfloat16
    if dtype in ("f32", GRAPE_F32, torch.float32):
        return torch.float32
    raise ValueError(f"dtype: need 'bf16' or 'f32', got {dtype!r}")


# the current stream's handle, without the stream object around it where torch offers that
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)


class _On:
    """Makes `stream` (None: the current one) current, so that what is allocated belongs to it;
    entering gives its handle."""

    def __init__(self, stream):
        self.stream, self.inner = stream, None

    def __enter__(self):
        if self.stream is None:
            if _raw_stream is not None:
                return _raw_stream(torch.cuda.current_device())
            return torch.cuda.current_stream().cuda_stream
        handle = self.stream if isinstance(self.stream, int) else self.stream.cuda_stream
        self.inner = torch.cuda.stream(torch.cuda.ExternalStream(handle))
        self.inner.__enter__()
        return handle

    def __exit__(self, *exc):
        if self.inner is not None:
            self.inner.__exit__(*exc)


def _scratch(n: int, like):
    return like.new_empty((max(n, 1),), dtype=torch.uint8)


# ---- embedding -----------------------------------------------------------------------------

def embed(table, ids, scale: float = 1.0, dtype="bf16", out=None, stream=None):
    """``scale * table[ids]`` in ``dtype``: ids of any shape, rows of ids outside the table zero."""
    dev = torch.cuda.current_device()
    _tensor(table, "table", dev, (None, None))
    tdt = _dtype(table, "table")
    id_bytes = _ids(ids, "ids", dev)
    V, d = table.shape
    if V < 1 or d < 1:
        raise ValueError(f"table: need at least one row and one column, got {tuple(table.shape)}")
    odt = _torch_dtype(dtype)
    with _On(stream) as st:
        out = _out(out, (*ids.shape, d), odt, dev, table)
        grape.grape_embed(table.data_ptr(), tdt, ids.data_ptr(), id_bytes, ids.numel(), V, d, scale,
                          GRAPE_F32 if odt is torch.float32 else GRAPE_BF16, out.data_ptr(), st)
    return out


def embed_order(ids, vocab: int, stream=None) -> EmbedOrder:
    """The order of a batch's ids (B x T), for ``embed_sqnorms`` and ``embed_grad``."""
    id_bytes = _ids(ids, "ids", torch.cuda.current_device(), (None, None))
    B, T = ids.shape
    vocab = int(vocab)
    n = grape.grape_embed_order_bytes(B * T, vocab)
    with _On(stream) as st:
        order = EmbedOrder(B, T, vocab, _scratch(n, ids))
        grape.grape_embed_order(ids.data_ptr(), id_bytes, B * T, vocab, order.buffer.data_ptr(), st)
    return order


def _embed_args(order: EmbedOrder, Gout, dev: int):
    _tensor(Gout, "Gout", dev, (order.B, order.T, None))
    _tensor(order.buffer, "order", dev)
    d = Gout.shape[2]
    if d < 1:
        raise ValueError(f"Gout: need at least one column, got {tuple(Gout.shape)}")
    return _dtype(Gout, "Gout"), d, grape.grape_embed_workspace_bytes(order.B, order.T, order.vocab, d)


def embed_sqnorms(order: EmbedOrder, Gout, scale: float = 1.0, out=None, stream=None):
    """Each sample's squared norm of the embedding table's gradient (B floats)."""
    dev = torch.cuda.current_device()
    dt, d, n = _embed_args(order, Gout, dev)
    with _On(stream) as st:
        out = _out(out, (order.B,), torch.float32, dev, Gout)
        ws = _scratch(n, Gout)
        grape.grape_embed_sqnorms(order.buffer.data_ptr(), order.B, order.T, order.vocab, d, Gout.data_ptr(), dt, scale,
                                  ws.data_ptr(), out.data_ptr(), st)
    return out


def embed_grad(order: EmbedOrder, Gout, weights=None, scale: float = 1.0, out=None, stream=None):
    """The embedding table's gradient (vocab x d, fp32), every sample's share times its weight."""
    dev = torch.cuda.current_device()
    dt, d, n = _embed_args(order, Gout, dev)
    w = _weights(weights, dev, (order.B,))
    with _On(stream) as st:
        out = _out(out, (order.vocab, d), torch.float32, dev, Gout)
        ws = _scratch(n, Gout)
        grape.grape_embed_grad(order.buffer.data_ptr(), order.B, order.T, order.vocab, d, Gout.data_ptr(), dt, scale, w,
                               ws.data_ptr(), out.data_ptr(), st)
    return out


# ---- losses --------------------------------------------------------------------------------

def head_loss(H, W, labels, weights=None, grad: bool = True, weight_grad: bool = False, stream=None) -> HeadLoss:
    """Softmax cross entropy of the head ``H @ W.T`` without its logits: losses, and on request
    the gradients of H (``grad``) and of W (``weight_grad``), in H's type.

    H is N x d or B x T x d, labels N or B x T; a label outside the vocabulary, or weight 0,
    drops the token."""
    dev = torch.cuda.current_device()
    _tensor(H, "H", dev)
    if H.dim() not in (2, 3):
        raise ValueError(f"H: need 2 or 3 dimensions, got {tuple(H.shape)}")
    dt = _dtype(H, "H")
    rows, d = H.shape[:-1], H.shape[-1]
    _tensor(W, "W", dev, (None, d), (H.dtype,))
    V = W.shape[0]
    id_bytes = _ids(labels, "labels", dev, rows)
    w = _weights(weights, dev, rows)
    N = labels.numel()
    n = grape.grape_head_loss_bytes(N, d, V, dt, grad, weight_grad)
    with _On(stream) as st:
        loss = H.new_empty(rows, dtype=torch.float32)
        dH = torch.empty_like(H) if grad else None
        dW = torch.empty_like(W) if weight_grad else None
        ws = _scratch(n, H)
        grape.grape_head_loss(H.data_ptr(), W.data_ptr(), labels.data_ptr(), id_bytes, w, N, d, V, dt, ws.data_ptr(),
                              loss.data_ptr(), dH.data_ptr() if grad else 0, dW.data_ptr() if weight_grad else 0, st)
    return HeadLoss(loss, dH, dW)


def distill_loss(logits, indices, values, weights=None, temperature: float = 1.0, out=None, stream=None):
    """(losses, Gout) of distillation from a teacher's top logits: ``values`` at vocabulary
    numbers ``indices`` (..., K); an index outside the vocabulary is an absent entry.

    ``out`` may be ``logits`` itself: Gout then replaces them."""
    dev = torch.cuda.current_device()
    _tensor(logits, "logits", dev)
    if logits.dim() not in (2, 3):
        raise ValueError(f"logits: need 2 or 3 dimensions, got {tuple(logits.shape)}")
    dt = _dtype(logits, "logits")
    rows, V = logits.shape[:-1], logits.shape[-1]
    id_bytes = _ids(indices, "indices", dev, (*rows, None))
    K = indices.shape[-1]
    _tensor(values, "values", dev, (*rows, K))
    vdt = _dtype(values, "values")
    w = _weights(weights, dev, rows)
    if out is not None:
        _tensor(out, "out", dev, logits.shape, (logits.dtype,))
        a, b, size = logits.data_ptr(), out.data_ptr(), logits.numel() * logits.element_size()
        if a != b and abs(a - b) < size:
            raise ValueError("out: may be the logits themselves, but not overlap them in part")
    with _On(stream) as st:
        if out is None:
            out = torch.empty_like(logits)
        loss = logits.new_empty(rows, dtype=torch.float32)
        grape.grape_distill_loss(logits.data_ptr(), dt, loss.numel(), V, indices.data_ptr(), id_bytes,
                                 values.data_ptr(), vdt, K, w, temperature, loss.data_ptr(), out.data_ptr(), st)
    return loss, out
