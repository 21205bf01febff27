"""Plain fp64 forms of the dense operators, with worst-case error bounds.

Every bound is a sum of the roundings the operator makes, propagated through
the formulas:
  * a product over k values summed in fp32 is off by at most (k + 8) 2^-24 of
    the sum of its terms' magnitudes; with fp32 operands split into two fp16
    planes each, by a further 3 2^-22 of it (each operand is kept to 2^-22 and
    lo * lo, at most 2^-22, is left out) and 2^-39 of the operands' largest
    values where an element is below the planes' range;
  * a value stored in a 16-bit type is off by half a unit, u = 2^-8 (bf16) or
    2^-11 (fp16), of itself, and by half of the type's smallest step;
  * an activation or its slope, evaluated in fp32, is off by at most 2^-20 of
    1 + |z|, and moves by at most 1.3 times its argument's error.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
STEP = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}
EVAL = 2.0 ** -20
LIPSCHITZ = 1.3


def act(name, z):
    if name == "relu":
        return z.clamp_min(0)
    if name == "silu":
        return z * torch.sigmoid(z)
    if name == "gelu":
        return z * 0.5 * (1 + torch.erf(z / math.sqrt(2)))
    return z


def slope(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "silu":
        s = torch.sigmoid(z)
        return s * (1 + z * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(z / math.sqrt(2))) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def rounded(v, dtype):
    return U[dtype] * v.abs() + STEP[dtype]


def product(a, b, split, ea=None, eb=None):
    """a [m, k] times b [k, n], and the bound on its computation from operands
    that are off by ea and eb."""
    mag = a.abs() @ b.abs()
    k = a.shape[1]
    e = (k + 8) * 2.0 ** -24 * mag
    if split and a.numel() and b.numel():
        e = e + 3 * 2.0 ** -22 * mag + 2.0 ** -39 * (
            a.abs().max() * b.abs().sum(0, keepdim=True) + b.abs().max() * a.abs().sum(1, keepdim=True))
    if ea is not None:
        e = e + ea @ (b.abs() + (0 if eb is None else eb))
    if eb is not None:
        e = e + a.abs() @ eb
    return a @ b, e


def moved(name, z, ez, f):
    """Bound on f(z) (an activation or its slope) at an argument off by ez."""
    e = LIPSCHITZ * ez + EVAL * (1 + z.abs())
    if name == "none":
        return ez if f is act else torch.zeros_like(z)
    if f is slope and name == "relu":
        return (z.abs() <= ez).to(z.dtype)   # the side of the kink is open
    return e


def linear(x, w, bias, residual, name, dy, out_dtype):
    """{"y", "dx", "dw", "db"}: (value, bound) each, from 16- or 32-bit tensors."""
    dt, split = x.dtype, x.dtype == torch.float32
    X, W = x.double(), w.double()
    z, ez = product(X, W.t(), split)
    if bias is not None:
        z = z + bias.double()
        ez = ez + 2.0 ** -23 * z.abs()
    y, ey = act(name, z), moved(name, z, ez, act)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * (y.abs() + residual.double().abs())
    out = {"y": (y, ey + rounded(y, out_dtype) * (1 + 2.0 ** -8))}
    if dy is None:
        return out
    d = slope(name, z)
    ed = moved(name, z, ez, slope)
    if name != "none" and dt == torch.bfloat16:
        ed = ed + rounded(d, torch.float16)
    DY = dy.double()
    dz = DY * d
    ez_kept = DY.abs() * ed + 2.0 ** -23 * dz.abs()         # before its rounding to dt
    ez_in = ez_kept + rounded(dz, dt) * (1 + 2.0 ** -8)
    dx, ex = product(dz, W, split, ea=ez_in)
    dw, ew = product(dz.t(), X, split, ea=ez_in.t())
    db = dz.sum(0)
    eb = ez_kept.sum(0) + (dz.shape[0] + 8) * 2.0 ** -24 * dz.abs().sum(0)
    for k, v, e in (("dx", dx, ex), ("dw", dw, ew), ("db", db, eb)):
        out[k] = (v, e + rounded(v, dt) * (1 + 2.0 ** -8))
    return out


def gated(x, w_in, w_out, residual, name, dy):
    dt, split = x.dtype, x.dtype == torch.float32
    X, WI, WO = x.double(), w_in.double(), w_out.double()
    F = WO.shape[1]
    gu, egu = product(X, WI.t(), split)
    g, u, eg, eu = gu[:, :F], gu[:, F:], egu[:, :F], egu[:, F:]
    a, ea = act(name, g), moved(name, g, eg, act)
    h = a * u
    eh = ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -22 * h.abs()
    eh = eh + rounded(h, dt) * (1 + 2.0 ** -8)
    y, ey = product(h, WO.t(), split, ea=eh)
    if residual is not None:
        y = y + residual.double()
        ey = ey + 2.0 ** -23 * (y.abs() + residual.double().abs())
    out = {"y": (y, ey + rounded(y, dt) * (1 + 2.0 ** -8))}
    if dy is None:
        return out
    DY = dy.double()
    dh, edh = product(DY, WO, split)
    d, ed = slope(name, g), moved(name, g, eg, slope)
    dg, du = dh * u * d, dh * a
    edg = (edh * (u.abs() + eu) * (d.abs() + ed) + dh.abs() * (eu * (d.abs() + ed) + u.abs() * ed)
           + 2.0 ** -22 * dg.abs() + rounded(dg, dt) * (1 + 2.0 ** -8))
    edu = (edh * (a.abs() + ea) + dh.abs() * ea + 2.0 ** -22 * du.abs()
           + rounded(du, dt) * (1 + 2.0 ** -8))
    dgu, edgu = torch.cat((dg, du), 1), torch.cat((edg, edu), 1)
    for k, (v, e) in (("dx", product(dgu, WI, split, ea=edgu)),
                      ("dw_in", product(dgu.t(), X, split, ea=edgu.t())),
                      ("dw_out", product(DY.t(), h, split, eb=eh))):
        out[k] = (v, e + rounded(v, dt) * (1 + 2.0 ** -8))
    return out


def orthogonalize(g, steps, coefficients, eps):
    a, b, c = coefficients
    x = g.double()
    x = x / (x.pow(2).sum((-2, -1), keepdim=True).sqrt() + eps)
    tall = x.shape[-2] > x.shape[-1]
    if tall:
        x = x.mT
    for _ in range(steps):
        p = x @ x.mT
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.mT if tall else x


def within(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), what
    worst = ((got - value).abs() / bound).max().item()
    assert worst <= 1.0, "%s: %.3g times its bound" % (what, worst)
