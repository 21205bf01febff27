"""Dense operators beside the splatting layer: the network that predicts the
Gaussians' raw values and the optimiser that trains it.

  linear          act(x w^T + bias) + residual, differentiable
  gated_mlp       (act(x w_gate^T) * (x w_up^T)) w_out^T + residual, differentiable
  orthogonalize   the Newton-Schulz products of the Muon optimiser
  Muon            the optimiser itself

PyTorch provides device memory and the current HIP stream; the computation
runs in the library's kernels through :mod:`._lib`.  Tensors live on one ROCm
device and are float32, float16 or bfloat16, all of one type.  Rows may be
strided; the last dimension is packed (anything else is copied first).
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from .splat import _FMT

# the current stream's handle, without the stream object around it
_raw_stream = torch._C._cuda_getCurrentRawStream

_ACTS = {"none": _lib.PDR_ACT_NONE, "relu": _lib.PDR_ACT_RELU, "silu": _lib.PDR_ACT_SILU,
         "gelu": _lib.PDR_ACT_GELU}


def _check(name: str, t, dtype=None, device=None, dim=None):
    if (dtype is not None and isinstance(t, torch.Tensor) and t.dtype == dtype
            and t.device == device and dim in (None, t.dim())):
        return   # like a tensor that has passed
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError("%s must be a tensor on a ROCm device" % name)
    if t.dtype not in _FMT:
        raise ValueError("%s must be float32, float16 or bfloat16" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s" % (name, dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, not on %s" % (name, t.device, device))
    if dim is not None and t.dim() != dim:
        raise ValueError("%s must have %d dimension(s)" % (name, dim))


def _activation(name: str) -> int:
    if name not in _ACTS:
        raise ValueError("activation must be one of %s" % ", ".join(sorted(_ACTS)))
    return _ACTS[name]


_MAX_LD = 1 << 22   # the kernels' largest distance between rows


def _rows(t: torch.Tensor) -> torch.Tensor:
    """t as [rows, columns] with packed columns; a view where its strides allow."""
    if t.dim() != 2:
        t = t.reshape(t.shape[:-1].numel(), t.shape[-1])
    if t.numel() and (t.stride(1) != 1 and t.shape[1] > 1
                      or not t.shape[1] <= t.stride(0) <= _MAX_LD):
        t = t.contiguous()
    return t


def _ld(t: torch.Tensor) -> int:
    rows, cols = t.shape
    return (t.stride(0) if rows > 1 else cols) or 1


def _kept_ld(n: int) -> int:
    """pdr_dense_kept_ld."""
    return (n + 7) // 8 * 8


_CALLS = {}


def _call(name: str, args, device):
    """Run an entry point in a workspace of its size, on the current stream."""
    if torch.cuda.current_device() != device.index:
        with torch.cuda.device(device):
            return _call(name, args, device)
    if name not in _CALLS:
        lib = _lib.lib()
        _CALLS[name] = (getattr(lib, name + "_workspace_bytes"), getattr(lib, name))
    size_of, run = _CALLS[name]
    rc = size = size_of(args)
    if size > 0:
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        rc = run(args, ws.data_ptr(), size, _raw_stream(device.index))
    elif size == 0:
        rc = run(args, None, 0, _raw_stream(device.index))
    if rc < 0:
        raise _lib.PdrError(rc, name)


def _has_tangent(t) -> bool:
    # outside a dual level (what unpack_dual looks at first) nothing has one, and
    # its answer takes 0.3 us a tensor
    return forward_ad._current_level >= 0 and forward_ad.unpack_dual(t).tangent is not None


def _differentiated(*tensors) -> bool:
    """Whether autograd has to see the call: for a gradient, or to refuse a tangent
    (forward mode), which would otherwise be lost."""
    grad = torch.is_grad_enabled()
    return any(t is not None and (grad and t.requires_grad or _has_tangent(t)) for t in tensors)


# ------------------------------------------------------------------- linear

def _linear_args(x, w, activation, out_dtype):
    """pdr_linear of the operands; the results' fields follow."""
    return _lib.pdr_linear(_FMT[x.dtype], _FMT[out_dtype], activation, x.shape[0], w.shape[0],
                           x.shape[1], x.data_ptr(), _ld(x), w.data_ptr(), _ld(w))


def _linear_forward(x, w, bias, residual, activation, out_dtype, keep):
    """(y, slope); slope only with `keep`."""
    a = _linear_args(x, w, activation, out_dtype)
    y = torch.empty((x.shape[0], w.shape[0]), dtype=out_dtype, device=x.device)
    a.y, a.ldy = y.data_ptr(), w.shape[0] or 1
    if bias is not None:
        a.bias = bias.data_ptr()
    if residual is not None:
        a.res, a.ldr = residual.data_ptr(), _ld(residual)
    slope = None
    if keep and activation != _lib.PDR_ACT_NONE:
        kind = torch.float16 if x.dtype == torch.bfloat16 else torch.float32
        slope = torch.empty((x.shape[0], _kept_ld(w.shape[0])), dtype=kind, device=x.device)
        a.slope = slope.data_ptr()
    _call("pdr_linear_forward", a, x.device)
    return y, slope


class Linear(torch.autograd.Function):
    """act(x w^T + bias) + residual of rows; keeps act' for the backward."""

    @staticmethod
    def forward(ctx, x, w, bias, residual, activation, out_dtype):
        y, slope = _linear_forward(x, w, bias, residual, activation, out_dtype,
                                   any(ctx.needs_input_grad[:3]))
        ctx.save_for_backward(x, w, slope)
        ctx.meta = (activation, out_dtype, bias is not None)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w, slope = ctx.saved_tensors
        activation, out_dtype, has_bias = ctx.meta
        need_x, need_w, need_b, need_r = ctx.needs_input_grad[:4]
        dx = dw = db = None
        if need_x or need_w or (need_b and has_bias):
            a = _linear_args(x, w, activation, out_dtype)
            rows = _rows(dy)
            a.dy, a.lddy = rows.data_ptr(), _ld(rows)
            if slope is not None:
                a.slope = slope.data_ptr()
            if need_x:
                dx = torch.empty((a.M, a.K), dtype=x.dtype, device=x.device)
                a.dx, a.lddx = dx.data_ptr(), max(a.K, 1)
            if need_w:
                dw = torch.empty((a.N, a.K), dtype=x.dtype, device=x.device)
                a.dw, a.lddw = dw.data_ptr(), max(a.K, 1)
            if need_b and has_bias:
                db = torch.empty((a.N,), dtype=x.dtype, device=x.device)
                a.dbias = db.data_ptr()
            _call("pdr_linear_backward", a, x.device)
        return dx, dw, db, dy if need_r else None, None, None


def linear(x: torch.Tensor, weight: torch.Tensor, bias: torch.Tensor | None = None,
           residual: torch.Tensor | None = None, activation: str = "none",
           out_dtype: torch.dtype | None = None) -> torch.Tensor:
    """act(x weight^T + bias) + residual, x [..., K], weight [N, K] -> [..., N].

    activation: "none", "relu", "silu" or "gelu" (the error-function form).
    out_dtype: x's type (default) or float32, which keeps the sums' precision;
    residual has this type and the result's shape.
    """
    _check("x", x)
    _check("weight", weight, x.dtype, x.device, 2)
    out_dtype = out_dtype or x.dtype
    if out_dtype not in (x.dtype, torch.float32):
        raise ValueError("out_dtype must be x's type or float32")
    if x.dim() < 1 or x.shape[-1] != weight.shape[1]:
        raise ValueError("x [..., K] and weight [N, K] disagree: %s, %s"
                         % (tuple(x.shape), tuple(weight.shape)))
    shape = (*x.shape[:-1], weight.shape[0])
    if bias is not None:
        _check("bias", bias, x.dtype, x.device, 1)
        if bias.shape[0] != weight.shape[0]:
            raise ValueError("bias must be [%d]" % weight.shape[0])
        bias = bias.contiguous()
    if residual is not None:
        _check("residual", residual, out_dtype, x.device)
        if residual.shape != shape:
            raise ValueError("residual must be %s" % (shape,))
        residual = _rows(residual)
    args = (_rows(x), _rows(weight), bias, residual, _activation(activation), out_dtype)
    if _differentiated(x, weight, bias, residual):
        y = Linear.apply(*args)
    else:
        y, _ = _linear_forward(*args, False)
    return y if x.dim() == 2 else y.view(shape)


# -------------------------------------------------------------- gated block

def _gated_args(x, w_in, w_out, activation):
    """pdr_gated_mlp of the operands; the results' fields follow."""
    return _lib.pdr_gated_mlp(_FMT[x.dtype], activation, x.shape[0], x.shape[1], w_out.shape[1],
                              w_out.shape[0], x.data_ptr(), _ld(x), w_in.data_ptr(), _ld(w_in),
                              w_out.data_ptr(), _ld(w_out))


def _gated_forward(x, w_in, w_out, residual, activation, keep):
    """(y, h, gu); gu only with `keep`."""
    a = _gated_args(x, w_in, w_out, activation)
    rows, cols = x.shape[0], w_out.shape[0]
    y = torch.empty((rows, cols), dtype=x.dtype, device=x.device)
    a.y, a.ldy = y.data_ptr(), cols or 1
    if residual is not None:
        a.res, a.ldr = residual.data_ptr(), _ld(residual)
    ld = _kept_ld(w_out.shape[1])
    h = torch.empty((rows, ld), dtype=x.dtype, device=x.device)
    a.h = h.data_ptr()
    gu = None
    if keep:
        gu = torch.empty((rows, 2, ld), dtype=torch.float32, device=x.device)
        a.gu = gu.data_ptr()
    _call("pdr_gated_mlp_forward", a, x.device)
    return y, h, gu


class GatedMLP(torch.autograd.Function):
    """The gated block of rows; keeps the gate and up sums (fp32) and their
    gated product for the backward."""

    @staticmethod
    def forward(ctx, x, w_in, w_out, residual, activation):
        y, h, gu = _gated_forward(x, w_in, w_out, residual, activation,
                                  any(ctx.needs_input_grad[:2]))
        ctx.save_for_backward(x, w_in, w_out, h, gu)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_in, w_out, h, gu = ctx.saved_tensors
        need = ctx.needs_input_grad
        dx = dwi = dwo = None
        if any(need[:3]):
            a = _gated_args(x, w_in, w_out, ctx.activation)
            rows = _rows(dy)
            a.dy, a.lddy = rows.data_ptr(), _ld(rows)
            a.h = h.data_ptr()
            if gu is not None:
                a.gu = gu.data_ptr()
            if need[0]:
                dx = torch.empty((a.M, a.D), dtype=x.dtype, device=x.device)
                a.dx, a.lddx = dx.data_ptr(), max(a.D, 1)
            if need[1]:
                dwi = torch.empty((2 * a.F, a.D), dtype=x.dtype, device=x.device)
                a.dw_in, a.ldd_in = dwi.data_ptr(), max(a.D, 1)
            if need[2]:
                dwo = torch.empty((a.O, a.F), dtype=x.dtype, device=x.device)
                a.dw_out, a.ldd_out = dwo.data_ptr(), max(a.F, 1)
            _call("pdr_gated_mlp_backward", a, x.device)
        return dx, dwi, dwo, dy if need[3] else None, None


def gated_mlp(x: torch.Tensor, w_in: torch.Tensor, w_out: torch.Tensor,
              residual: torch.Tensor | None = None, activation: str = "silu") -> torch.Tensor:
    """(act(x w_gate^T) * (x w_up^T)) w_out^T + residual.

    x [..., D]; w_in [2F, D], the gate's rows first, then the up rows; w_out
    [O, F]; residual and the result [..., O].
    """
    _check("x", x)
    _check("w_in", w_in, x.dtype, x.device, 2)
    _check("w_out", w_out, x.dtype, x.device, 2)
    if x.dim() < 1 or x.shape[-1] != w_in.shape[1] or w_in.shape[0] != 2 * w_out.shape[1]:
        raise ValueError("x [..., D], w_in [2F, D] and w_out [O, F] disagree: %s, %s, %s"
                         % (tuple(x.shape), tuple(w_in.shape), tuple(w_out.shape)))
    shape = (*x.shape[:-1], w_out.shape[0])
    if residual is not None:
        _check("residual", residual, x.dtype, x.device)
        if residual.shape != shape:
            raise ValueError("residual must be %s" % (shape,))
        residual = _rows(residual)
    args = (_rows(x), _rows(w_in), _rows(w_out), residual, _activation(activation))
    if _differentiated(x, w_in, w_out, residual):
        y = GatedMLP.apply(*args)
    else:
        y = _gated_forward(*args, False)[0]
    return y if x.dim() == 2 else y.view(shape)


# ------------------------------------------------------------ orthogonalize

MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _check_steps(steps, coefficients):
    if int(steps) != steps or steps < 0:
        raise ValueError("steps must be a whole number >= 0")
    if len(coefficients) != 3:
        raise ValueError("coefficients must be (a, b, c)")


@torch.no_grad()
def orthogonalize(g: torch.Tensor, steps: int = 5, coefficients=MUON_COEFFICIENTS,
                  eps: float = 1e-7, dtype: torch.dtype | None = None) -> torch.Tensor:
    """Bring the singular values of g [..., m, n] near one, by `steps` of
    X <- a X + (b A + c A^2) X with A = X X^T, from X = g / (|g|_F + eps).

    coefficients: (a, b, c); those under which singular values from [0, 1] run
    away from 1 leave the iterates' range and are refused (PdrError).
    dtype: the result's type; g's, or with a float32 g any, which is normalised
    before it is rounded.  bfloat16 results come from iterates of 11 bits (up to
    twice as far off as their own rounding), others from 22 bits.
    A step of an optimiser: the result is no function of g to autograd.
    """
    _check("g", g)
    if _has_tangent(g):
        raise NotImplementedError("orthogonalize has no forward-mode derivative")
    if g.dim() < 2:
        raise ValueError("g must be [..., m, n]")
    _check_steps(steps, coefficients)
    dtype = dtype or g.dtype
    if dtype not in _FMT or dtype != g.dtype != torch.float32:
        raise ValueError("dtype must be g's type, or g float32 and dtype float16 or bfloat16")
    m, n = g.shape[-2:]
    flat = g if g.dim() == 2 else g.reshape((g.shape[:-2].numel(), m, n))
    if g.numel() and (flat.stride(-1) != 1 and n > 1
                      or m > 1 and not n <= flat.stride(-2) <= _MAX_LD):
        flat = flat.contiguous()
    out = torch.empty(g.shape, dtype=dtype, device=g.device)
    a = _lib.pdr_orthogonalize_args()
    a.fmt, a.batch, a.m, a.n = _FMT[dtype], 1 if g.dim() == 2 else flat.shape[0], m, n
    a.g, a.ldg = flat.data_ptr(), flat.stride(-2) if m > 1 else max(n, 1)
    a.batch_g = flat.stride(0) if g.dim() > 2 else 0
    a.x, a.ldx, a.batch_x = out.data_ptr(), max(n, 1), m * n
    a.steps = int(steps)
    a.a, a.b, a.c = (float(v) for v in coefficients)
    a.eps = float(eps)
    a.g_f32 = dtype != g.dtype
    _call("pdr_orthogonalize", a, g.device)
    return out


class Muon(torch.optim.Optimizer):
    """Momentum whose update is orthogonalised, for weights of two dimensions.

    buf <- momentum buf + grad;  u = grad + momentum buf (nesterov) or buf;
    p <- p (1 - lr weight_decay) - lr max(1, m / n)^(1/2) orthogonalize(u).
    The momentum is kept in `state_dtype` (float32 by default).  Weights of one
    shape and type are orthogonalised in one batch, in `work_dtype` (their own
    type by default; bfloat16 takes a third of the products of float32 and
    float16, which start from the update in float32).
    """

    def __init__(self, params, lr: float = 0.02, momentum: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, steps: int = 5, coefficients=MUON_COEFFICIENTS,
                 eps: float = 1e-7, state_dtype: torch.dtype = torch.float32,
                 work_dtype: torch.dtype | None = None):
        super().__init__(params, dict(lr=lr, momentum=momentum, nesterov=nesterov,
                                      weight_decay=weight_decay, steps=steps,
                                      coefficients=tuple(coefficients), eps=eps,
                                      state_dtype=state_dtype, work_dtype=work_dtype))

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        try:
            self._check_group(self.param_groups[-1])
        except ValueError:
            self.param_groups.pop()
            raise

    @staticmethod
    def _check_group(group):
        if group["lr"] < 0 or not 0 <= group["momentum"] < 1 or group["weight_decay"] < 0:
            raise ValueError("lr and weight_decay must be >= 0 and momentum in [0, 1)")
        _check_steps(group["steps"], group["coefficients"])
        if not group["state_dtype"].is_floating_point:
            raise ValueError("state_dtype must be a floating-point type")
        if group["work_dtype"] is not None and group["work_dtype"] not in _FMT:
            raise ValueError("work_dtype must be float32, float16 or bfloat16")
        for p in group["params"]:
            if p.dim() != 2:
                raise ValueError("Muon updates weights of two dimensions, got %s"
                                 % (tuple(p.shape),))

    def load_state_dict(self, state_dict):
        """As torch.optim.Optimizer's, but the momentum is taken in `state_dtype`:
        the base class rounds it to the weight's type."""
        taken = []
        before = self.register_load_state_dict_pre_hook(lambda _, given: taken.append(given))
        after = self.register_load_state_dict_post_hook(lambda _: self._take_momentum(taken[0]),
                                                        prepend=True)
        try:
            super().load_state_dict(state_dict)
        finally:
            before.remove()
            after.remove()

    def _take_momentum(self, given):
        for group, saved in zip(self.param_groups, given["param_groups"]):
            for p, key in zip(group["params"], saved["params"]):
                if "momentum" in given["state"].get(key, ()):
                    self.state[p]["momentum"] = given["state"][key]["momentum"].to(
                        device=p.device, dtype=group["state_dtype"], copy=True)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            alike = {}
            for p in group["params"]:
                if p.grad is None:
                    continue
                state = self.state[p]
                if "momentum" not in state:
                    state["momentum"] = torch.zeros_like(p, dtype=group["state_dtype"])
                buf = state["momentum"]
                grad = p.grad.to(buf.dtype)
                buf.mul_(group["momentum"]).add_(grad)
                u = grad.add(buf, alpha=group["momentum"]) if group["nesterov"] else buf
                work = group["work_dtype"] or p.dtype
                # fp16 holds the orthogonalisation's values, not a gradient's range
                u = u.to(torch.float32 if work == torch.float16 else work)
                alike.setdefault((p.shape, p.dtype, p.device), []).append((p, u))
            for (shape, _, _), pairs in alike.items():
                scale = max(1.0, shape[0] / max(1, shape[1])) ** 0.5
                updates = orthogonalize(torch.stack([u for _, u in pairs]), group["steps"],
                                        group["coefficients"], group["eps"],
                                        dtype=group["work_dtype"] or pairs[0][0].dtype)
                for (p, _), u in zip(pairs, updates):
                    p.mul_(1 - group["lr"] * group["weight_decay"])
                    p.add_(u.to(p.dtype), alpha=-group["lr"] * scale)
        return loss
