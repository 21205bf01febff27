"""Plain fp64 forms of attention, layer norm and dropout, with worst-case error
bounds that are sums of the roundings the operators make (dense_ref has those of
sums, types and steps).

Attention, for a query i and key j:
  * a score, a sum over D products in fp32, is off by (D + 8) 2^-24 of its terms'
    magnitudes, and its exponent by a further 2^-22 of the score and the maximum
    or the log of the sum that is taken from it;
  * a weight's relative error is that, 2^-21 of exp2 and, where it enters a
    product, the type's rounding (in fp16 also 2^-25 of the largest weight, which
    is the type's smallest step);
  * sums over n weights: (n + 8) 2^-24 of the terms' magnitudes;
  * exp2 gives 0 for results below 2^-126, and the matrix instruction may take
    bf16 and fp32 operands below that as 0: weights and ds may be off by TINY.
The backward's delta is off by what the stored result is; in fp16, ds is held
under a power of two for each column that leaves 2^-36 of the column's largest.
"""
import math

import torch

from dense_ref import STEP, U, rounded

F = 2.0 ** -24
TINY = 2.0 ** -126


def within(got, ref, what):
    value, bound = ref
    got = got.detach().cpu().double()
    assert got.shape == value.shape, (what, got.shape, value.shape)
    if not got.numel():
        return
    assert torch.isfinite(got).all(), what
    share = (got - value).abs() / bound
    at = torch.unravel_index(share.argmax(), share.shape)
    at = tuple(int(i) for i in at)
    assert share[at] <= 1.0, "%s: %.3g times its bound at %s: %.6g for %.6g +- %.3g" % (
        what, share[at], at, got[at], value[at], bound[at])


def attention(q, k, v, dy, causal, scale, step=2.0 ** -25):
    """One sequence: q, dy [nq, H, D], k, v [nk, Hk, D] -> {"y", "dq", "dk", "dv"} of
    (value, bound); the gradients only with dy.  `step`: what a weight in fp16 may be off
    by below its range, of the largest (2^-37 where weights are held near the range's end)."""
    dt = q.dtype
    u = 0.0 if dt == torch.float32 else U[dt] * (1 + 2.0 ** -7)
    low = step if dt == torch.float16 else TINY
    nq, h, d = q.shape
    nk, hk = k.shape[:2]
    g = h // hk
    out = {n: torch.zeros(t.shape, dtype=torch.float64) for n, t in (("y", q), ("dq", q), ("dk", k), ("dv", v))}
    err = {n: torch.full_like(t, STEP[dt]) for n, t in out.items()}
    sees = torch.ones(nq, nk, dtype=torch.bool)
    if causal:
        sees = torch.arange(nk)[None] <= torch.arange(nq)[:, None] + (nk - nq)
    some = sees.any(1, keepdim=True) if nk else torch.zeros(nq, 1, dtype=torch.bool)
    for n in range(h):
        Q, K, V = q[:, n].double(), k[:, n // g].double(), v[:, n // g].double()
        if not nk or not nq:
            continue
        s = scale * (Q @ K.T)
        es = scale * (d + 8) * F * (Q.abs() @ K.abs().T)
        s = s.masked_fill(~sees, -math.inf)
        m = s.amax(1, keepdim=True)
        m = torch.where(some, m, torch.zeros_like(m))
        e = torch.exp(s - m)
        l = e.sum(1, keepdim=True)
        p = torch.where(some, e / l, torch.zeros_like(e))
        L = m + torch.log(torch.where(some, l, torch.ones_like(l)))
        seen_s = torch.where(sees, s, torch.zeros_like(s)).abs()
        rp = torch.where(sees, torch.expm1(es + 2.0 ** -22 * (seen_s + m.abs()) + es.amax(1, keepdim=True)) + 2.0 ** -21,
                         torch.zeros_like(s))
        rl = rp.amax(1, keepdim=True) + (nk + 8) * F
        mag = p @ V.abs()
        y = p @ V
        ey = (p * (rp + u)) @ V.abs() + (rl + (nk + 8) * F) * mag + low * (sees.double() @ V.abs()) / torch.where(some, l, torch.ones_like(l))
        out["y"][:, n], err["y"][:, n] = y, ey * 1.02 + rounded(y, dt) * (1 + 2.0 ** -7)
        if dy is None:
            continue
        DY = dy[:, n].double()
        delta = (DY * y).sum(1, keepdim=True)
        ed = (DY.abs() * err["y"][:, n]).sum(1, keepdim=True) + (d + 8) * F * (DY.abs() * y.abs()).sum(1, keepdim=True)
        dp = DY @ V.T
        edp = (d + 8) * F * (DY.abs() @ V.abs().T)
        rb = torch.where(sees, torch.expm1(es + rl + 2.0 ** -22 * (seen_s + L.abs())) + 2.0 ** -21, torch.zeros_like(s))
        ds = p * (dp - delta)
        eds = p * (1 + rb) * (edp + ed) + rb * ds.abs() + 2.0 ** -22 * p * (dp.abs() + delta.abs())
        eds = eds + u * (ds.abs() + eds) + sees * TINY * (1 + dp.abs() + delta.abs() + edp + ed)
        if dt == torch.float16:
            eds_q = eds + 2.0 ** -36 * ds.abs().amax(1, keepdim=True)
            eds_k = eds + 2.0 ** -36 * ds.abs().amax(0, keepdim=True)
        else:
            eds_q = eds_k = eds
        out["dq"][:, n] = scale * (ds @ K)
        err["dq"][:, n] = scale * (eds_q @ K.abs() + (nk + 8) * F * (ds.abs() @ K.abs()))
        out["dk"][:, n // g] += scale * (ds.T @ Q)
        err["dk"][:, n // g] += scale * (eds_k.T @ Q.abs() + (nq * g + 8) * F * (ds.abs().T @ Q.abs()))
        out["dv"][:, n // g] += p.T @ DY
        err["dv"][:, n // g] += (p * (rb + u + (nq * g + 8) * F) + sees * (2.0 ** -40 if dt == torch.float16 else TINY)).T @ DY.abs()
    for name in ("dq", "dk", "dv"):
        err[name] = err[name] * 1.02 + rounded(out[name], dt) * (1 + 2.0 ** -7)
    return {name: (out[name], err[name]) for name in out}


def layer_norm(x, weight, bias, eps, dy):
    """{"y", "dx", "dw", "db"}: (value, bound) of rows x [m, n]."""
    dt = x.dtype
    X, n = x.double(), x.shape[-1]
    W = torch.ones(n, dtype=torch.float64) if weight is None else weight.double()
    B = torch.zeros(n, dtype=torch.float64) if bias is None else bias.double()
    if not n:
        return {"y": (X, X), "dx": (X, X), "dw": (W, W), "db": (B, B)}
    mean = X.mean(-1, keepdim=True)
    c = X - mean
    var = (c * c).mean(-1, keepdim=True)
    r = 1 / torch.sqrt(var + eps)
    xh = c * r
    # a centred value: the mean's rounding, which the centred values' own sum takes out again, leaves (n + 8) 2^-24 of
    # their mean magnitude; r half of what the sum of squares is off by, and its own evaluation
    top = X.abs().amax(-1, keepdim=True)
    ec = F * c.abs() * 2 + (n + 8) * F * (c.abs().mean(-1, keepdim=True) + (n + 8) * F * top)
    rr = (n + 16) * F + (ec.amax(-1, keepdim=True) * r)
    exh = ec * r + xh.abs() * rr
    y = xh * W + B
    ey = exh * W.abs() + 2 * F * (y.abs() + B.abs())
    out = {"y": (y, ey * 1.02 + rounded(y, dt))}
    if dy is None:
        return out
    DY = dy.double()
    g = DY * W
    m, mx = g.mean(-1, keepdim=True), (g * xh).mean(-1, keepdim=True)
    em = (n + 8) * F * g.abs().mean(-1, keepdim=True)
    # the kept mean is rounded: xh comes with an offset that its own mean takes out
    exb = exh + 4 * F * xh.abs() + (n + 8) * F * (xh.abs().mean(-1, keepdim=True) + F * top * r)
    emx = (n + 8) * F * (g * xh).abs().mean(-1, keepdim=True) + (g.abs() * exb).mean(-1, keepdim=True)
    dx = r * (g - m - xh * mx)
    edx = r * (em + exb * (mx.abs() + emx) + xh.abs() * emx + 4 * F * (g.abs() + m.abs() + (xh * mx).abs())) + rr * dx.abs()
    rows = x.shape[0]
    dw, db = (DY * xh).sum(0), DY.sum(0)
    edw = (DY.abs() * exb).sum(0) + (rows + 8) * F * (DY * xh).abs().sum(0)
    edb = (rows + 8) * F * DY.abs().sum(0)
    for name, v, e in (("dx", dx, edx), ("dw", dw, edw), ("db", db, edb)):
        out[name] = (v, e * 1.02 + rounded(v, dt))
    return out


M32 = 0xFFFFFFFF


def philox(counter, key):
    """Philox 4x32 with 10 rounds, of Python's whole numbers."""
    x, k = list(counter), list(key)
    for _ in range(10):
        a, b = x[0] * 0xD2511F53, x[2] * 0xCD9E8D57
        x = [(b >> 32) ^ x[1] ^ k[0], b & M32, (a >> 32) ^ x[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return x


def kept(seed, offset, first, count, p):
    """Which of the elements [first, first + count) are kept."""
    t, out, words, block = round(p * 65536), [], None, None
    for i in range(first, first + count):
        if i // 8 != block:
            block = i // 8
            words = philox((block & M32, block >> 32, offset & M32, offset >> 32), (seed & M32, seed >> 32))
        out.append(((words[i % 8 // 2] >> (16 * (i & 1))) & 0xFFFF) >= t)
    return torch.tensor(out, dtype=torch.bool)


def dropout(x, residual, keep, p):
    t = round(p * 65536)
    v = torch.where(keep, x.double() * (65536 / (65536 - t) if t < 65536 else 0.0), torch.zeros((), dtype=torch.float64))
    e = 3 * F * v.abs()
    if residual is not None:
        v = v + residual.double()
        e = e + 2 * F * (v.abs() + residual.double().abs())
    return v, e + rounded(v, x.dtype) * (1 + 2.0 ** -7)
