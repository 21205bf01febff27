"""The operators that make a transformer block of the dense ones (:mod:`.dense`):

  attention    softmax(scale q k^T) v over whole, packed or cached sequences, differentiable
  layer_norm   (x - mean) / sqrt(var + eps) * weight + bias of rows, differentiable
  dropout      kept values / (1 - p) + residual, with a mask that is never stored, differentiable

PyTorch provides device memory and the current HIP stream; the computation
runs in the library's kernels through :mod:`._lib`.  Tensors live on one ROCm
device and are float32, float16 or bfloat16, all of one type.  The last
dimension is packed (anything else is copied first).
"""
from __future__ import annotations

import functools

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .dense import _call, _check, _differentiated, _ld, _rows
from .splat import _FMT



def _once(backward):
    """once_differentiable, without its gradient mode's switch where that is off already
    (it takes some microseconds of autograd's thread)."""
    checked = once_differentiable(backward)

    @functools.wraps(backward)
    def run(ctx, *grads):
        return (checked if torch.is_grad_enabled() else backward)(ctx, *grads)
    return run


# ---------------------------------------------------------------- attention

MAX_HEAD_DIM = 128
_MAX_ROW, _MAX_HEAD, _MAX_HEADS = 1 << 22, 1 << 24, 1 << 28   # the kernels' largest strides


def _heads(t: torch.Tensor) -> torch.Tensor:
    """t [..., heads, D] as the kernels read it: rows of whole 16 bytes that begin on
    16 bytes.  The tensor itself where it is so; else a copy, with zeros up to a
    multiple."""
    per = 16 // t.element_size()
    d, strides = t.shape[-1], t.stride()
    if d % per:
        return torch.nn.functional.pad(t, (0, -d % per))
    batch, row, head = strides[0], strides[-3], strides[-2]
    if ((strides[-1] != 1 or (batch | row | head) % per or t.data_ptr() % 16 or row > _MAX_ROW or head > _MAX_HEAD
         or head * (t.shape[-2] - 1) > _MAX_HEADS) and t.numel()):
        return t.clone(memory_format=torch.contiguous_format)
    return t


def _place(t):
    """(pointer, row, head, batch) of [batch, tokens, heads, D] or [tokens, heads, D]."""
    if t is None:
        return None, 0, 0, 0
    strides = t.stride()
    if len(strides) == 4:
        return t.data_ptr(), strides[1], strides[2], strides[0]
    return t.data_ptr(), strides[0], strides[1], 0


def _attention_args(q, k, v, o, lse, meta, index, *gradients):
    """pdr_attention of tensors that _heads has seen; index: (offsets, key_offsets, key_lengths);
    gradients: dy, dq, dk and dv, or none."""
    offsets, key_offsets, key_lengths = index
    batch = q.shape[0] if offsets is None else offsets.shape[0] - 1
    causal, scale = meta
    heads, d = q.shape[-2:]
    # in the struct's order; what is left out is 0
    return _lib.pdr_attention(
        _FMT[q.dtype], causal, batch, heads, k.shape[-2], d, q.shape[-3], k.shape[-3],
        None if offsets is None else offsets.data_ptr(),
        None if offsets is None else key_offsets.data_ptr(),
        None if key_lengths is None else key_lengths.data_ptr(), scale,
        *_place(q), *_place(k), *_place(v), *_place(o), None if lse is None else lse.data_ptr(),
        *(x for t in gradients for x in _place(t)))


def _packed(t):
    """Room for a result of t's shape."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _attention_forward(q, k, v, meta, index, keep):
    """(o, lse) of tensors that _heads has seen; lse only with `keep`."""
    o, lse = _packed(q), None
    if keep:
        lse = torch.empty((k.shape[-2], q.shape[:-2].numel(), q.shape[-2] // k.shape[-2]),
                          dtype=torch.float32, device=q.device)
    _call("pdr_attention_forward", _attention_args(q, k, v, o, lse, meta, index), q.device)
    return o, lse


def _to_dim(t, d):
    return t if t.shape[-1] == d else t[..., :d].contiguous()


class Attention(torch.autograd.Function):
    """Attention of whole, packed or cached sequences; keeps the result and each
    row's log of the sum of exponentials for the backward."""

    @staticmethod
    def forward(ctx, q, k, v, meta, *index):
        d = q.shape[-1]
        q, k, v = _heads(q), _heads(k), _heads(v)
        o, lse = _attention_forward(q, k, v, meta, index, True)
        ctx.save_for_backward(q, k, v, o, lse, *index)
        ctx.meta = (meta, d)
        return _to_dim(o, d)

    @staticmethod
    @_once
    def backward(ctx, dy):
        q, k, v, o, lse, *index = ctx.saved_tensors
        meta, d = ctx.meta
        need = ctx.needs_input_grad
        dq = _packed(q) if need[0] else None
        dk, dv = (_packed(k), _packed(v)) if need[1] or need[2] else (None, None)
        dy = _heads(dy)
        _call("pdr_attention_backward", _attention_args(q, k, v, o, lse, meta, index, dy, dq, dk, dv), q.device)
        return (*(_to_dim(g, d) if n else None for g, n in zip((dq, dk, dv), need)),
                None, None, None, None)


def _check_index(name: str, t, like, length=None):
    if not isinstance(t, torch.Tensor) or t.dtype != torch.int32 or t.dim() != 1:
        raise ValueError("%s must be an int32 tensor of one dimension" % name)
    if t.device != like.device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, like.device))
    if length is not None and t.shape[0] != length:
        raise ValueError("%s must be [%d]" % (name, length))
    return t.contiguous()


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = False,
              scale: float | None = None, offsets: torch.Tensor | None = None,
              key_offsets: torch.Tensor | None = None,
              key_lengths: torch.Tensor | None = None) -> torch.Tensor:
    """softmax(scale q k^T) v for each sequence and head; q's shape.

    Sequences of one length: q [B, Sq, Hq, D], k and v [B, Sk, Hk, D]; Hq is a
    multiple of Hk, and query head h reads key head h // (Hq // Hk).
    key_lengths (int32 [B], on the device): how many of its Sk keys each sequence
    has, as for a cache that is being filled.  The queries are its last ones: where
    queries are padded too, pack the sequences instead.
    Packed sequences: q [T, Hq, D], k and v [Tk, Hk, D] with offsets (int32
    [n + 1], on the device, not descending): sequence b has the queries
    offsets[b] .. offsets[b + 1] - 1, and the same keys or those of key_offsets.
    Tokens outside of all sequences get zeros.
    causal: a query sees the keys up to its own, the last query being at the last
    key: j <= i + (keys - queries).  A query that sees no key gets zeros.
    scale: in [2^-64, 2^64]; D ** -0.5 by default.  D is at most 128.
    """
    _check("q", q)
    _check("k", k, q.dtype, q.device)
    _check("v", v, q.dtype, q.device)
    dim = 4 if offsets is None else 3
    if q.dim() != dim or k.dim() != dim:
        raise ValueError("q and k must be [B, S, H, D], or with offsets [T, H, D]")
    if k.shape != v.shape or q.shape[-1] != k.shape[-1] or dim == 4 and q.shape[0] != k.shape[0]:
        raise ValueError("q, k and v disagree: %s, %s, %s" % (tuple(q.shape), tuple(k.shape), tuple(v.shape)))
    heads, kv_heads, d = q.shape[-2], k.shape[-2], q.shape[-1]
    if not 0 < d <= MAX_HEAD_DIM:
        raise ValueError("heads must have 1 to %d values" % MAX_HEAD_DIM)
    if kv_heads < 1 or heads < 1 or heads % kv_heads:
        raise ValueError("q's heads must be a multiple of k's: %d, %d" % (heads, kv_heads))
    scale = d ** -0.5 if scale is None else float(scale)
    if not 2.0 ** -64 <= scale <= 2.0 ** 64:
        raise ValueError("scale must be in [2^-64, 2^64]")
    if offsets is None:
        if key_offsets is not None:
            raise ValueError("key_offsets needs offsets")
        if key_lengths is not None:
            key_lengths = _check_index("key_lengths", key_lengths, q, q.shape[0])
    else:
        if key_lengths is not None:
            raise ValueError("key_lengths is for sequences without offsets")
        offsets = _check_index("offsets", offsets, q)
        if offsets.shape[0] < 1:
            raise ValueError("offsets must have a value more than there are sequences")
        key_offsets = (offsets if key_offsets is None
                       else _check_index("key_offsets", key_offsets, q, offsets.shape[0]))
    meta, index = (bool(causal), scale), (offsets, key_offsets, key_lengths)
    if _differentiated(q, k, v):
        return Attention.apply(q, k, v, meta, *index)
    return _to_dim(_attention_forward(_heads(q), _heads(k), _heads(v), meta, index, False)[0], d)


# --------------------------------------------------------------- layer norm

def _pointer(t):
    return None if t is None else t.data_ptr()


def _norm_forward(x, weight, bias, eps, keep):
    """(y, stats); stats only with `keep`."""
    rows, cols = x.shape
    y, stats = _packed(x), None
    if keep:
        stats = torch.empty((rows, 2), dtype=torch.float32, device=x.device)
    _call("pdr_layer_norm_forward",
          _lib.pdr_layer_norm(_FMT[x.dtype], rows, cols, eps, x.data_ptr(), _ld(x), _pointer(weight), _pointer(bias),
                              y.data_ptr(), cols or 1, _pointer(stats)), x.device)
    return y, stats


class LayerNorm(torch.autograd.Function):
    """Layer norm of rows; keeps each row's mean and inverse deviation."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps):
        y, stats = _norm_forward(x, weight, bias, eps, True)
        ctx.save_for_backward(x, weight, stats)
        ctx.eps = eps
        return y

    @staticmethod
    @_once
    def backward(ctx, dy):
        # autograd's thread takes several times as long for a line as the caller's: few of them
        x, weight, stats = ctx.saved_tensors
        need_x, need_w, need_b, _ = ctx.needs_input_grad
        rows, cols = x.shape
        dy = _rows(dy)
        dx = torch.empty_like(x) if need_x else None
        dw = torch.empty_like(weight) if need_w else None
        db = x.new_empty(cols) if need_b else None
        _call("pdr_layer_norm_backward",
              _lib.pdr_layer_norm(_FMT[x.dtype], rows, cols, ctx.eps, x.data_ptr(), _ld(x),
                                  None if weight is None else weight.data_ptr(), None, None, 0, stats.data_ptr(),
                                  dy.data_ptr(), _ld(dy), dx.data_ptr() if need_x else None, cols or 1,
                                  dw.data_ptr() if need_w else None, db.data_ptr() if need_b else None), x.device)
        return dx, dw, db, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, eps: float = 1e-5) -> torch.Tensor:
    """(x - mean) / sqrt(var + eps) * weight + bias over the last dimension of x
    [..., N]; weight and bias [N], or None for one and zero.  N is at most 2^30.

    The squares of centred values are summed in fp32 and have to be in its range.
    """
    _check("x", x)
    if x.dim() < 1:
        raise ValueError("x must be [..., N]")
    n = x.shape[-1]
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None:
            _check(name, t, x.dtype, x.device, 1)
            if t.shape[0] != n:
                raise ValueError("%s must be [%d]" % (name, n))
    eps = float(eps)
    if not 0 <= eps < float("inf"):
        raise ValueError("eps must be finite and not negative")
    args = (_rows(x), None if weight is None else weight.contiguous(),
            None if bias is None else bias.contiguous(), eps)
    y = LayerNorm.apply(*args) if _differentiated(x, weight, bias) else _norm_forward(*args, False)[0]
    return y if x.dim() == 2 else y.view(x.shape)


# ------------------------------------------------------------------ dropout

def _dropout(x, residual, p, seed, offset):
    y = _packed(x)
    rows, cols = x.shape
    whole = not isinstance(seed, torch.Tensor)
    _call("pdr_dropout",
          _lib.pdr_dropout_args(_FMT[x.dtype], rows, cols, p, seed if whole else 0, offset,
                                None if whole else seed.data_ptr(), x.data_ptr(), _ld(x), _pointer(residual),
                                0 if residual is None else _ld(residual), y.data_ptr(), cols or 1), x.device)
    return y


class Dropout(torch.autograd.Function):
    """Dropout of rows; the backward draws the same bits again."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, offset):
        if isinstance(seed, torch.Tensor):
            ctx.save_for_backward(seed)
            ctx.seed = None
        else:
            ctx.seed = seed
        ctx.meta = (p, offset)
        return _dropout(x, residual, p, seed, offset)

    @staticmethod
    @_once
    def backward(ctx, dy):
        seed = ctx.saved_tensors[0] if ctx.seed is None else ctx.seed
        p, offset = ctx.meta
        dx = _dropout(_rows(dy), None, p, seed, offset) if ctx.needs_input_grad[0] else None
        return dx, dy if ctx.needs_input_grad[1] else None, None, None, None


def dropout(x: torch.Tensor, p: float, seed, offset: int = 0,
            residual: torch.Tensor | None = None) -> torch.Tensor:
    """x / (1 - p) where an element is kept, 0 elsewhere, + residual (x's shape).

    Which elements are kept is a function of (seed, offset, element) alone: 16 bits
    of Philox 4x32-10 each, compared with p 2^16 (p is taken to a multiple of 2^-16).
    seed: a whole number below 2^64, or an int64 tensor of one element on x's
    device, which is read when the kernels run, so that replays of a captured
    graph may draw anew; it may not change between a forward and its backward.
    offset: a whole number below 2^64, such as a layer's and a step's, for masks
    under one seed.
    """
    _check("x", x)
    p = float(p)
    if not 0 <= p <= 1:
        raise ValueError("p must be in [0, 1]")
    if isinstance(seed, torch.Tensor):
        if seed.dtype != torch.int64 or seed.numel() != 1 or seed.device != x.device:
            raise ValueError("seed must be a whole number, or an int64 tensor of one element on %s" % x.device)
    elif int(seed) != seed or not 0 <= seed < 1 << 64:
        raise ValueError("seed must be a whole number in [0, 2^64)")
    else:
        seed = int(seed)
    if int(offset) != offset or not 0 <= offset < 1 << 64:
        raise ValueError("offset must be a whole number in [0, 2^64)")
    if residual is not None:
        _check("residual", residual, x.dtype, x.device)
        if residual.shape != x.shape:
            raise ValueError("residual must be %s" % (tuple(x.shape),))
    flat = x if x.dim() else x.view(1)
    rest = None
    if residual is not None:
        rest = _rows(residual if residual.dim() else residual.view(1))
    args = (_rows(flat), rest, p, seed, int(offset))
    y = Dropout.apply(*args) if _differentiated(x, residual) else _dropout(*args)
    return y if x.dim() == 2 else y.view(x.shape)
