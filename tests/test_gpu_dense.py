"""The dense operators (linear, gated block, Newton-Schulz, Muon) on the GPU
against plain fp64 forms, at the sizes, strides and values where they can go
wrong.  The tolerances are the worst-case bounds of dense_ref."""
import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
TYPES = (BF, HF, FP)


def dense():
    from differentiable_gaussian_splatting_pdr_amd import dense as d
    return d


def normal(seed, *shape, scale=1.0, dtype=FP):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def leaf(t, need=True):
    return t.cuda().requires_grad_(need)


def run_linear(M, K, N, dtype, act="none", bias=True, residual=True, out=None, seed=0):
    out = out or dtype
    x, w = normal(seed, M, K, dtype=dtype), normal(seed + 1, N, K, scale=max(K, 1) ** -0.5, dtype=dtype)
    b = normal(seed + 2, N, dtype=dtype) if bias else None
    r = normal(seed + 3, M, N, dtype=out) if residual else None
    dy = normal(seed + 4, M, N, dtype=out)
    want = ref.linear(x, w, b, r, act, dy, out)
    xs, ws = leaf(x), leaf(w)
    bs, rs = leaf(b) if bias else None, leaf(r) if residual else None
    y = dense().linear(xs, ws, bs, residual=rs, activation=act, out_dtype=out)
    assert y.dtype == out
    y.backward(dy.cuda())
    what = "%dx%dx%d %s %s" % (M, K, N, dtype, act)
    ref.within(y, want["y"], "y " + what)
    ref.within(xs.grad, want["dx"], "dx " + what)
    ref.within(ws.grad, want["dw"], "dw " + what)
    if bias:
        ref.within(bs.grad, want["db"], "db " + what)
    if residual:
        assert torch.equal(rs.grad.cpu(), dy)


SIZES = [(1, 1, 1), (1, 64, 128), (1, 1000, 37), (2, 8, 8), (3, 257, 5), (16, 128, 64), (17, 72, 130),
         (64, 63, 65), (127, 129, 255), (128, 128, 128), (129, 64, 127), (200, 520, 8), (255, 33, 21),
         (300, 256, 384), (513, 200, 264), (1030, 48, 6)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", SIZES)
def test_linear_sizes(M, K, N, dtype):
    run_linear(M, K, N, dtype, act="gelu", seed=M + K + N)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu"])
@pytest.mark.parametrize("bias,residual", [(False, False), (True, False), (False, True)])
def test_linear_epilogues(act, bias, residual, dtype):
    run_linear(70, 96, 88, dtype, act=act, bias=bias, residual=residual, seed=7)


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("act", ["none", "silu"])
def test_linear_kept_in_32_bits(act, dtype):
    run_linear(130, 100, 24, dtype, act=act, out=FP, seed=11)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_long_contractions(dtype):
    # few results, long sums: the contraction is cut and joined, in the
    # forward (K) and in the weight's gradient (M)
    run_linear(40, 5000, 24, dtype, seed=13)
    run_linear(9000, 24, 40, dtype, act="silu", seed=14)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(0, 16, 8), (5, 0, 8), (5, 16, 0), (0, 0, 0)])
def test_linear_empty(M, K, N, dtype):
    run_linear(M, K, N, dtype, act="silu")
    run_linear(M, K, N, dtype, bias=False, residual=False)


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_strides_and_leading_dimensions(dtype):
    d = dense()
    wide = normal(1, 2, 9, 50, dtype=dtype).cuda()
    x = wide[..., 3:44]                      # rows 50 apart, not on 16 bytes
    w = normal(2, 60, 33, dtype=dtype).cuda()[:41].t()   # packed the other way: copied
    r = normal(3, 33, 2, 9, dtype=dtype).cuda().permute(1, 2, 0)
    y = d.linear(x, w, residual=r)
    want = ref.linear(x.cpu().reshape(18, 41), w.cpu(), None, r.cpu().reshape(18, 33), "none", None, dtype)
    assert y.shape == (2, 9, 33)
    ref.within(y.reshape(18, 33), want["y"], "strided")
    one = d.linear(x[1, 4], w)               # a vector
    assert one.shape == (33,)
    # one row repeated: stride 0
    same = d.linear(x[1, 4].expand(7, 41), w)
    assert torch.equal(same, one.expand(7, 33))


@pytest.mark.parametrize("dtype", TYPES)
def test_linear_gradient_of_broadcast_and_strided_results(dtype):
    d = dense()
    x, w = leaf(normal(1, 12, 40, dtype=dtype)), leaf(normal(2, 16, 40, dtype=dtype))
    d.linear(x, w).sum().backward()          # dy is one value, expanded
    want = ref.linear(x.detach().cpu(), w.detach().cpu(), None, None, "none", torch.ones(12, 16, dtype=dtype), dtype)
    ref.within(x.grad, want["dx"], "dx")
    ref.within(w.grad, want["dw"], "dw")


def test_linear_only_what_is_needed():
    d = dense()
    x, w, b = normal(1, 33, 64, dtype=BF).cuda(), leaf(normal(2, 24, 64, dtype=BF)), leaf(normal(3, 24, dtype=BF))
    d.linear(x, w, b, activation="silu").sum().backward()
    assert x.grad is None and w.grad is not None and b.grad is not None
    x2, b2 = leaf(x.detach().clone()), leaf(b.detach().clone())
    (gb,) = torch.autograd.grad(d.linear(x2, w, b2, activation="silu").sum(), [b2])
    assert torch.equal(gb, b.grad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,K,N", [(3, 64, 48), (150, 64, 48), (150, 61, 47)])
def test_linear_not_finite_stays_in_its_row(M, K, N, dtype):
    d = dense()
    x, w = normal(1, M, K, dtype=dtype), normal(2, N, K, dtype=dtype)
    clean = d.linear(x.cuda(), w.cuda()).cpu()
    x[1, 5] = float("inf")
    x[2, K - 1] = float("nan")
    y = d.linear(x.cuda(), w.cuda()).cpu()
    assert not torch.isfinite(y[1]).any() and torch.isnan(y[2]).all()
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("scale", [1e-30, 1e-6, 1e6, 1e30])
def test_linear_fp32_range(scale):
    # the planes' scale follows the tensor; the other operand brings results back
    x, w = normal(1, 40, 72) * scale, normal(2, 24, 72) / scale
    want = ref.linear(x, w, None, None, "none", None, FP)
    ref.within(dense().linear(x.cuda(), w.cuda()), want["y"], "scale %g" % scale)


def run_gated(M, D, F, O, dtype, act="silu", residual=True, seed=0):
    x = normal(seed, M, D, dtype=dtype)
    wi = normal(seed + 1, 2 * F, D, scale=max(D, 1) ** -0.5, dtype=dtype)
    wo = normal(seed + 2, O, F, scale=max(F, 1) ** -0.5, dtype=dtype)
    r = normal(seed + 3, M, O, dtype=dtype) if residual else None
    dy = normal(seed + 4, M, O, dtype=dtype)
    want = ref.gated(x, wi, wo, r, act, dy)
    xs, wis, wos = leaf(x), leaf(wi), leaf(wo)
    rs = leaf(r) if residual else None
    y = dense().gated_mlp(xs, wis, wos, residual=rs, activation=act)
    y.backward(dy.cuda())
    what = "%dx%dx%dx%d %s %s" % (M, D, F, O, dtype, act)
    for k, t in (("y", y), ("dx", xs.grad), ("dw_in", wis.grad), ("dw_out", wos.grad)):
        ref.within(t, want[k], k + " " + what)
    if residual:
        assert torch.equal(rs.grad.cpu(), dy)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,D,F,O", [(1, 1, 1, 1), (1, 64, 96, 64), (4, 40, 33, 24), (16, 128, 64, 128),
                                     (17, 31, 65, 13), (128, 64, 64, 64), (130, 72, 136, 72),
                                     (257, 100, 70, 101), (300, 256, 130, 8)])
def test_gated_sizes(M, D, F, O, dtype):
    run_gated(M, D, F, O, dtype, seed=M + D + F)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", ["none", "relu", "gelu"])
def test_gated_activations(act, dtype):
    run_gated(50, 48, 56, 48, dtype, act=act, residual=False, seed=5)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,D,F,O", [(0, 8, 8, 8), (3, 0, 8, 8), (3, 8, 0, 8), (3, 8, 8, 0)])
def test_gated_empty(M, D, F, O, dtype):
    run_gated(M, D, F, O, dtype)


def test_gated_strided_rows():
    x = normal(1, 30, 80, dtype=BF).cuda()[:, 8:72]
    wi = normal(2, 96, 100, dtype=BF).cuda()[:, 1:65]
    wo = normal(3, 40, 48, dtype=BF).cuda()
    want = ref.gated(x.cpu(), wi.cpu(), wo.cpu(), None, "silu", None)
    ref.within(dense().gated_mlp(x, wi, wo), want["y"], "strided")


def test_gradients_against_differences():
    # fp32: a central difference along one direction, whose own errors are h^2
    # times a third derivative and the results' rounding over h: 1e-3 of the
    # derivative's scale covers both at h = 2^-7
    d = dense()
    h = 2.0 ** -7
    x, w, b = (normal(i, *s).cuda() for i, s in ((1, (20, 24)), (2, (16, 24)), (3, (16,))))
    wi, wo = normal(4, 2 * 40, 24, scale=0.2).cuda(), normal(5, 24, 40, scale=0.2).cuda()
    c, c2 = normal(6, 20, 16).cuda().double(), normal(7, 20, 24).cuda().double()
    for name in ("silu", "gelu"):
        for f, args, dots in ((lambda *a: d.linear(*a, activation=name), (x, w, b), c),
                              (lambda *a: d.gated_mlp(*a, activation=name), (x, wi, wo), c2)):
            leaves = [a.clone().requires_grad_() for a in args]
            y = f(*leaves)
            grads = torch.autograd.grad(y, leaves, dots.float())
            for i in range(3):
                v = normal(20 + i, *args[i].shape).cuda()
                v = v / v.norm()
                hi, lo = ([a + s * h * v if j == i else a for j, a in enumerate(args)] for s in (1, -1))
                diff = ((f(*hi).double() - f(*lo).double()) * dots).sum() / (2 * h)
                got = (grads[i].double() * v.double()).sum()
                assert abs(diff - got) <= 1e-3 * grads[i].double().norm(), (name, i)


# Iterates in one fp16 plane are rounded to 2^-12 of themselves three times a
# step (X, A, B), in two planes to 2^-22; the polynomial's derivative is at
# most 3.45, but it is 3.45 only where it is also the map's gain, so that a
# relative error grows at most by the steps' count; products add (m + n) 2^-24
# a step.  The result is rounded once more.
def ortho_bound(m, n, steps, dtype):
    plane = 2.0 ** -12 if dtype == BF else 2.0 ** -21
    return steps * 3 * (plane + (m + n) * 2.0 ** -24) + ref.U[dtype]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 40), (40, 1), (8, 64), (64, 8), (16, 16), (33, 129), (129, 33),
                                   (128, 128), (130, 520), (257, 100), (3, 17, 40), (2, 40, 17), (2, 2, 24, 24)])
def test_orthogonalize(shape, dtype):
    c = (3.4445, -4.7750, 2.0315)
    g = normal(sum(shape), *shape, scale=0.01, dtype=dtype)
    want = ref.orthogonalize(g, 5, c, 1e-7)
    got = dense().orthogonalize(g.cuda()).cpu()
    assert got.dtype == dtype and got.shape == g.shape
    off = ((got.double() - want).norm() / want.norm()).item()
    assert off <= ortho_bound(shape[-2], shape[-1], 5, dtype), off


@pytest.mark.parametrize("dtype", (BF, FP))
@pytest.mark.parametrize("shape", [(2049, 6001), (6001, 2049), (2, 1288, 2120)])
def test_orthogonalize_large(shape, dtype):
    # sizes whose symmetric products are computed by their lower tiles, in one
    # part and in several; the fp64 form runs on the GPU
    c = (3.4445, -4.7750, 2.0315)
    g = torch.randn(*shape, device="cuda", generator=torch.Generator("cuda").manual_seed(sum(shape))).to(dtype)
    want = ref.orthogonalize(g, 5, c, 1e-7)
    got = dense().orthogonalize(g).double()
    off = ((got - want).norm() / want.norm()).item()
    assert off <= ortho_bound(shape[-2], shape[-1], 5, dtype), off


@pytest.mark.parametrize("steps", [0, 1, 2, 7])
def test_orthogonalize_steps_and_coefficients(steps):
    c = (15 / 8, -10 / 8, 3 / 8)
    g = normal(3, 50, 70)
    want = ref.orthogonalize(g, steps, c, 1e-3)
    got = dense().orthogonalize(g.cuda(), steps=steps, coefficients=c, eps=1e-3).cpu()
    assert ((got.double() - want).norm() / want.norm()).item() <= ortho_bound(50, 70, max(steps, 1), FP)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1e-18, 1e-4, 1e4, 1e18])
def test_orthogonalize_does_not_see_scale(scale, dtype):
    if dtype == HF and not 1e-5 < scale < 1e5:
        pytest.skip("outside fp16's range")
    g = normal(4, 24, 40, dtype=FP)
    g = (g * min(scale, 1e4) if dtype == HF else g * scale).to(dtype)
    want = ref.orthogonalize(g, 5, (3.4445, -4.7750, 2.0315), 0.0)
    got = dense().orthogonalize(g.cuda(), eps=0.0).cpu()
    assert ((got.double() - want).norm() / want.norm()).item() <= ortho_bound(24, 40, 5, dtype)


def test_orthogonalize_odd_values():
    d = dense()
    z = d.orthogonalize(torch.zeros(3, 20, 30, device="cuda"))
    assert torch.equal(z, torch.zeros_like(z))
    g = normal(5, 3, 20, 30).cuda()
    clean = d.orthogonalize(g)
    g[1, 2, 3] = float("nan")
    got = d.orthogonalize(g)
    assert torch.isnan(got[1]).all() and torch.equal(got[0], clean[0]) and torch.equal(got[2], clean[2])
    assert d.orthogonalize(torch.empty(0, 5, 6, device="cuda")).shape == (0, 5, 6)
    assert d.orthogonalize(torch.empty(5, 0, device="cuda")).shape == (5, 0)
    # rank one: the one singular value goes where the polynomial takes 1, and
    # the iterates' roundings (2^-21 of |X|) enter directions where nothing
    # is, where each remaining step multiplies them by 3.4445: at most
    # 3.4445^5 (1 + 1/3.4445 + ...) = 1.41 * 3.4445^5 in all
    u, v = normal(6, 20, 1), normal(7, 1, 30)
    want = ref.orthogonalize(u @ v, 5, (3.4445, -4.7750, 2.0315), 1e-7)
    got = d.orthogonalize((u @ v).cuda()).cpu().double()
    assert ((got - want).norm() / want.norm()).item() <= 1.41 * 3.4445 ** 5 * 2.0 ** -21


def test_orthogonalize_strided():
    d = dense()
    g = normal(8, 4, 30, 50, dtype=BF).cuda()
    part = g[::2, 3:20, 8:48]
    assert torch.equal(d.orthogonalize(part), d.orthogonalize(part.contiguous()))
    turned = g[0].t()
    assert torch.equal(d.orthogonalize(turned), d.orthogonalize(turned.contiguous()))


def test_muon_step():
    d = dense()
    ps = [normal(i, 40, 24, dtype=FP).cuda().requires_grad_() for i in range(2)]
    ps.append(normal(9, 16, 32, dtype=BF).cuda().requires_grad_())
    before = [p.detach().cpu().double() for p in ps]
    opt = d.Muon(ps, lr=0.1, momentum=0.9, weight_decay=0.01)
    bufs = [torch.zeros_like(b) for b in before]
    for k in range(3):
        for i, p in enumerate(ps):
            p.grad = normal(100 + 10 * k + i, *p.shape, dtype=p.dtype).cuda()
        opt.step()
        for i, p in enumerate(ps):
            gr = p.grad.cpu().double()
            bufs[i] = 0.9 * bufs[i] + gr
            u = ref.orthogonalize((gr + 0.9 * bufs[i]).to(p.dtype), 5, (3.4445, -4.7750, 2.0315), 1e-7)
            before[i] = before[i] * (1 - 0.001) - 0.1 * max(1, p.shape[0] / p.shape[1]) ** 0.5 * u
            if p.dtype == BF:
                before[i] = p.detach().cpu().double() if (p.detach().cpu().double() - before[i]).abs().max() < 0.03 else None
            else:
                assert (p.detach().cpu().double() - before[i]).abs().max() < 2e-4
    with pytest.raises(ValueError):
        d.Muon([torch.zeros(3, device="cuda", requires_grad=True)])


def test_other_stream_and_repeat():
    # the same bits on another stream, and run after run
    d = dense()
    x, w, b = normal(1, 300, 136, dtype=BF).cuda(), normal(2, 72, 136, dtype=BF).cuda(), normal(3, 72, dtype=BF).cuda()
    wi, wo = normal(4, 2 * 88, 136, dtype=BF).cuda(), normal(5, 136, 88, dtype=BF).cuda()
    f = lambda: (d.linear(x, w, b, activation="gelu"), d.gated_mlp(x, wi, wo), d.orthogonalize(w))  # noqa: E731
    want = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = f()
    side.synchronize()
    for a, c in zip(want, got):
        assert torch.equal(a, c)


def test_captured_in_a_graph():
    d = dense()
    x, w = leaf(normal(1, 200, 100, dtype=BF)), leaf(normal(2, 60, 100, dtype=BF))
    wi, wo = leaf(normal(3, 2 * 50, 60, dtype=BF)), leaf(normal(4, 60, 50, dtype=BF))
    dy = normal(5, 200, 60, dtype=BF).cuda()

    def step():
        y = d.gated_mlp(d.linear(x, w, activation="silu"), wi, wo)
        grads = torch.autograd.grad(y, (x, w, wi, wo), dy)
        return (y.detach(), *grads, d.orthogonalize(grads[1]))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(4):
        with torch.no_grad():
            x.copy_(normal(10 + k, 200, 100, dtype=BF))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(eager, out):
            assert torch.equal(a, c), k


def test_refusals():
    d = dense()
    x, w = torch.zeros(4, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    for bad in (dict(x=x.cpu()), dict(x=x.int()), dict(weight=w.half()), dict(weight=w[0]),
                dict(weight=torch.zeros(6, 9, device="cuda")), dict(bias=torch.zeros(5, device="cuda")),
                dict(bias=torch.zeros(6)), dict(residual=torch.zeros(4, 5, device="cuda")),
                dict(residual=torch.zeros(4, 6, device="cuda").half()), dict(activation="tanh"),
                dict(out_dtype=torch.float16)):
        with pytest.raises(ValueError):
            d.linear(**{"x": x, "weight": w, **bad})
    wi, wo = torch.zeros(12, 8, device="cuda"), torch.zeros(8, 6, device="cuda")
    for bad in (dict(w_in=wi[:11]), dict(w_out=wo[:, :5]), dict(x=x[:, :7]), dict(x=x.bfloat16()),
                dict(activation="swish"), dict(residual=x[:, :7])):
        with pytest.raises(ValueError):
            d.gated_mlp(**{"x": x, "w_in": wi, "w_out": wo, **bad})
    for bad in (dict(g=x[0]), dict(steps=-1), dict(steps=1.5), dict(coefficients=(1, 2)), dict(g=x.cpu())):
        with pytest.raises(ValueError):
            d.orthogonalize(**{"g": x, **bad})
    from differentiable_gaussian_splatting_pdr_amd import PdrError
    with pytest.raises(PdrError):
        d.orthogonalize(x, coefficients=(1.0, float("nan"), 0.0))
    with pytest.raises(PdrError):
        d.orthogonalize(x, eps=-1.0)


def test_predictor_learns_through_the_splatting_layer():
    # the example: projections, gated blocks and Muon in front of the renderer
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import fit_predictor
    losses = fit_predictor.train(steps=30)
    assert all(v == v for v in losses)
    assert sum(losses[-5:]) / 5 < 0.7 * losses[0], losses


def test_muon_work_dtype():
    d = dense()
    p = normal(1, 48, 96).cuda().requires_grad_()
    q = p.detach().clone().requires_grad_()
    p.grad = normal(2, 48, 96).cuda()
    q.grad = p.grad.clone()
    d.Muon([p], lr=0.1, momentum=0.0, nesterov=False).step()
    d.Muon([q], lr=0.1, momentum=0.0, nesterov=False, work_dtype=BF).step()
    u = d.orthogonalize(p.grad.to(BF)).float()
    assert torch.equal(q, normal(1, 48, 96).cuda().add_(u, alpha=-0.1))
    assert (p - q).abs().max() < 0.1 * 0.05


def test_offsets_beyond_31_bits():
    # a result of 2.25e9 values (4.5 GB): its last rows, and the gradients that read it
    d = dense()
    M, K, N = 1_100_003, 16, 2048
    x = torch.randn(M, K, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(BF).requires_grad_()
    w = leaf(normal(2, N, K, scale=K ** -0.5, dtype=BF))
    y = d.linear(x, w)
    at = torch.tensor([0, 1, 524287, 524288, 1048575, 1048576, M - 130, M - 2, M - 1])
    rows = x.detach()[at.cuda()].cpu()
    ref.within(y[at.cuda()], ref.linear(rows, w.detach().cpu(), None, None, "none", None, BF)["y"], "y")
    dy = torch.zeros_like(y)
    some = normal(3, len(at), N, dtype=BF)
    dy[at.cuda()] = some.cuda()
    gx, gw = torch.autograd.grad(y, (x, w), dy)
    want = ref.linear(rows, w.detach().cpu(), None, None, "none", some, BF)
    ref.within(gx[at.cuda()], want["dx"], "dx")
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[at.cuda()] = False
    assert not gx[others].any()
    # the sum over a million rows of zeros and nine others
    ref.within(gw, want["dw"], "dw")


def test_twice_differentiated_is_refused():
    d = dense()
    x, w = leaf(normal(1, 70, 32)), leaf(normal(2, 16, 32))
    (g,) = torch.autograd.grad(d.linear(x, w, activation="silu").sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
