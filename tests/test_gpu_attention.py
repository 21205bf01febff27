"""Attention on the GPU against a plain fp64 form, at the lengths, layouts, masks
and values where it can go wrong.  The tolerances are blocks_ref's worst-case
bounds."""
import pytest
import torch

import blocks_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
TYPES = (BF, HF, FP)


def blocks():
    from differentiable_gaussian_splatting_pdr_amd import blocks as b
    return b


def normal(seed, *shape, scale=1.0, dtype=FP):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def leaf(t):
    return t.detach().cuda().requires_grad_()


def against(got, want, what):
    for name, t in got.items():
        ref.within(t, want[name], "%s %s" % (name, what))


def stack(wants):
    """One reference of several sequences'."""
    return {n: tuple(torch.stack([w[n][i] for w in wants]) for i in (0, 1)) for n in wants[0]}


def run_batch(B, nq, nk, h, hk, d, dtype, causal, scale=None, train=True, seed=0, spread=1.0):
    q, k, v = (normal(seed + i, B, n, m, d, dtype=dtype, scale=spread) for i, (n, m) in enumerate(((nq, h), (nk, hk), (nk, hk))))
    dy = normal(seed + 3, B, nq, h, d, dtype=dtype) if train else None
    c = d ** -0.5 if scale is None else scale
    want = stack([ref.attention(q[b], k[b], v[b], dy[b] if train else None, causal, c) for b in range(B)])
    qs, ks, vs = (leaf(t) for t in (q, k, v))
    got = {}
    if train:
        y = blocks().attention(qs, ks, vs, causal=causal, scale=scale)
        got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(y, (qs, ks, vs), dy.cuda())))
    with torch.no_grad():
        got["y"] = blocks().attention(qs, ks, vs, causal=causal, scale=scale)
    if train:
        assert torch.equal(got["y"], y)
    against(got, want, "%s %s" % ((B, nq, nk, h, hk, d, causal), dtype))


SIZES = [(1, 1, 1, 1, 1, 8), (1, 1, 300, 4, 1, 64), (2, 3, 5, 2, 2, 16), (1, 31, 31, 3, 3, 20), (1, 33, 64, 2, 1, 64),
         (1, 64, 63, 2, 2, 64), (2, 65, 129, 6, 2, 72), (1, 128, 128, 2, 2, 128), (1, 129, 65, 5, 1, 128), (1, 200, 260, 4, 4, 1),
         (1, 130, 130, 8, 1, 96), (1, 257, 257, 1, 1, 128), (3, 40, 40, 10, 5, 33)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("size", SIZES)
def test_sizes(size, causal, dtype):
    run_batch(*size, dtype, causal, seed=sum(size))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,nq,nk,h,hk,d", [(1, 1, 700, 4, 4, 64), (2, 1, 1500, 8, 1, 128), (1, 4, 2000, 8, 2, 128), (1, 5, 600, 6, 1, 72),
                                            (3, 1, 1, 2, 2, 64), (1, 32, 513, 1, 1, 64), (5, 2, 33, 4, 2, 128)])
def test_few_queries(B, nq, nk, h, hk, d, dtype):
    """At most 32 rows a sequence and key head: waves and workgroups that share the keys."""
    run_batch(B, nq, nk, h, hk, d, dtype, True, seed=nk)
    run_batch(B, nq, nk, h, hk, d, dtype, False, train=False, seed=nk)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nk", [(70, 3), (3, 1), (40, 0), (300, 200), (0, 5), (0, 0)])
def test_queries_without_keys(nq, nk, dtype):
    # causal, more queries than keys: the first see nothing
    run_batch(2, nq, nk, 4, 2, 64, dtype, True, seed=3)
    if nk == 0:
        run_batch(2, nq, nk, 4, 2, 64, dtype, False, seed=3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale,spread", [(1.0, 3.0), (0.01, 1.0), (0.5, 0.05)])
def test_scales(scale, spread, dtype):
    # scores up to hundreds: one key takes nearly all; and scores near zero
    run_batch(1, 150, 150, 2, 1, 64, dtype, True, scale=scale, spread=spread, seed=9)


def offsets_of(lengths, before=0):
    out = [before]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def run_packed(lengths, key_lengths, h, hk, d, dtype, causal, before=0, after=0, seed=0):
    qo, ko = offsets_of(lengths, before), offsets_of(key_lengths or lengths, before)
    T, Tk = qo[-1] + after, ko[-1] + after
    q, dy = (normal(seed + i, T, h, d, dtype=dtype) for i in (0, 1))
    k, v = (normal(seed + i, Tk, hk, d, dtype=dtype) for i in (2, 3))
    want = {n: (torch.zeros(t.shape, dtype=torch.float64), torch.full(t.shape, 1e-300, dtype=torch.float64))
            for n, t in (("y", q), ("dq", q), ("dk", k), ("dv", v))}
    for b in range(len(lengths)):
        at, kat = slice(qo[b], qo[b + 1]), slice(ko[b], ko[b + 1])
        one = ref.attention(q[at], k[kat], v[kat], dy[at], causal, d ** -0.5)
        for n in one:
            for i in (0, 1):
                want[n][i][at if n in ("y", "dq") else kat] = one[n][i]
    for value, bound in want.values():
        bound[(bound == 0) & (value == 0)] = 1e-300   # exact zeros
    qs, ks, vs = (leaf(t) for t in (q, k, v))
    offs = torch.tensor(qo, dtype=torch.int32, device="cuda")
    koffs = torch.tensor(ko, dtype=torch.int32, device="cuda") if key_lengths else None
    y = blocks().attention(qs, ks, vs, causal=causal, offsets=offs, key_offsets=koffs)
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(y, (qs, ks, vs), dy.cuda())), y=y)
    against(got, want, "packed %s" % dtype)
    # what runs without a gradient is the same
    assert torch.equal(blocks().attention(qs.detach(), ks.detach(), vs.detach(), causal=causal, offsets=offs, key_offsets=koffs), y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths", [[5], [0], [], [1, 0, 7, 130, 0], [128, 128, 64], [127, 129, 1, 63], [300, 0, 0, 2, 77]])
def test_packed(lengths, causal, dtype):
    run_packed(lengths, None, 6, 2, 64, dtype, causal, seed=len(lengths))


@pytest.mark.parametrize("dtype", TYPES)
def test_packed_with_tokens_outside(dtype):
    # before the first and behind the last sequence: zeros, and zero gradients
    run_packed([40, 0, 130], None, 4, 4, 40, dtype, True, before=3, after=200, seed=5)
    run_packed([2, 1], None, 4, 1, 128, dtype, False, before=150, after=1, seed=6)
    run_packed([], None, 2, 1, 64, dtype, True, before=0, after=9, seed=7)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
def test_packed_with_other_keys(causal, dtype):
    run_packed([3, 0, 100, 5, 1], [200, 4, 0, 2, 90], 4, 2, 64, dtype, causal, before=2, after=3, seed=8)
    run_packed([1, 1, 2, 1], [300, 33, 700, 0], 8, 2, 128, dtype, causal, seed=9)


def test_packed_many_sequences():
    # more than the search looks at in one step
    lengths = [(i * 7) % 6 for i in range(150)]
    run_packed(lengths, None, 2, 1, 64, BF, True, seed=1)
    lengths = [i % 3 for i in range(5000)]
    lengths[77], lengths[4099] = 140, 67
    run_packed(lengths, None, 2, 2, 8, FP, False, seed=2)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("nq", [1, 3, 60])
def test_cache(nq, causal, dtype):
    """Key lengths, some beyond what there is; what lies behind them does not matter."""
    d, h, hk, S = 64, 4, 2, 900
    lengths = [0, 1, nq, 33, 899, 900, 5000, -4]
    B = len(lengths)
    q, dy = normal(1, B, nq, h, d, dtype=dtype), normal(4, B, nq, h, d, dtype=dtype)
    k, v = normal(2, B, S, hk, d, dtype=dtype), normal(3, B, S, hk, d, dtype=dtype)
    held = [max(0, min(n, S)) for n in lengths]
    want = {n: (torch.zeros(t.shape, dtype=torch.float64), torch.full(t.shape, 1e-300, dtype=torch.float64))
            for n, t in (("y", q), ("dq", q), ("dk", k), ("dv", v))}
    for b, n in enumerate(held):
        one = ref.attention(q[b], k[b, :n], v[b, :n], dy[b], causal, d ** -0.5)
        for name in one:
            for i in (0, 1):
                want[name][i][b, slice(None) if name in ("y", "dq") else slice(0, n)] = one[name][i]
        k[b, n:], v[b, n:] = float("nan"), float("inf")
    for value, bound in want.values():
        bound[(bound == 0) & (value == 0)] = 1e-300
    qs, ks, vs = (leaf(t) for t in (q, k, v))
    lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    y = blocks().attention(qs, ks, vs, causal=causal, key_lengths=lens)
    got = dict(zip(("dq", "dk", "dv"), torch.autograd.grad(y, (qs, ks, vs), dy.cuda())), y=y)
    against(got, want, "cache %s" % dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nk,h", [(150, 150, 2), (3, 200, 2), (1, 90, 4), (40, 300, 1)])
def test_not_finite_behind_the_mask(nq, nk, h, dtype):
    """Results of queries that do not see an infinity or NaN are those without it; the others' are not finite."""
    b, d = blocks(), 64
    q, k, v = normal(1, 1, nq, h, d, dtype=dtype), normal(2, 1, nk, 1, d, dtype=dtype), normal(3, 1, nk, 1, d, dtype=dtype)
    clean = b.attention(q.cuda(), k.cuda(), v.cuda(), causal=True).cpu()
    for at in (nk - 1, nk - nq // 2 - 1, nk - nq):
        for bad in (float("nan"), float("inf"), -float("inf")):
            first = max(0, at - (nk - nq))   # the first query that sees it
            w = v.clone()
            w[0, at, 0, 5] = bad
            y = b.attention(q.cuda(), k.cuda(), w.cuda(), causal=True).cpu()
            assert torch.equal(y[:, :first], clean[:, :first]), (at, bad)
            keep = [i for i in range(d) if i != 5]
            assert torch.allclose(y[..., keep].float(), clean[..., keep].float(), rtol=2 ** -7, atol=2 ** -9)
            got = y[0, first:, :, 5]
            # a weight that is 0 in fp32 makes NaN of an infinity; none is here
            assert torch.isnan(got).all() if bad != bad else (got == bad).all(), (at, bad)
            x = k.clone()
            x[0, at, 0, 5] = bad
            y = b.attention(q.cuda(), x.cuda(), v.cuda(), causal=True).cpu()
            assert torch.equal(y[:, :first], clean[:, :first]), (at, bad)


@pytest.mark.parametrize("dtype", TYPES)
def test_not_finite_in_other_sequences(dtype):
    """Neither results nor gradients of a sequence depend on what others hold."""
    b, d, offs = blocks(), 40, torch.tensor([0, 30, 75, 140], dtype=torch.int32, device="cuda")
    ts = [normal(i, 140, n, d, dtype=dtype) for i, n in ((1, 4), (2, 2), (3, 2), (4, 4))]

    def run(ts):
        q, k, v = (leaf(t) for t in ts[:3])
        y = b.attention(q, k, v, causal=True, offsets=offs)
        return [y.detach().cpu()] + [g.cpu() for g in torch.autograd.grad(y, (q, k, v), ts[3].cuda())]
    clean = run(ts)
    for i in range(4):
        bad = [t.clone() for t in ts]
        bad[i][30:75] = float("nan")
        for got, want in zip(run(bad), clean):
            assert torch.equal(got[:30], want[:30]) and torch.equal(got[75:], want[75:]), i


@pytest.mark.parametrize("dtype", TYPES)
def test_layouts(dtype):
    """Views: parts of one projection, heads before tokens, rows on odd places, expanded keys, packed the other way."""
    b, d = blocks(), 64
    parts = normal(1, 2, 70, 8, d, dtype=dtype).cuda()
    q, k, v = parts.split((4, 2, 2), 2)
    want = stack([ref.attention(q[i].cpu(), k[i].cpu(), v[i].cpu(), None, True, d ** -0.5) for i in (0, 1)])["y"]
    plain = b.attention(q.contiguous(), k.contiguous(), v.contiguous(), causal=True)
    ref.within(plain, want, "layouts")
    odd = torch.zeros(2, 70, 8, d + 3, dtype=dtype, device="cuda")[..., 1:1 + d]
    odd.copy_(parts)
    heads_first = parts.transpose(1, 2).contiguous().transpose(1, 2)
    turned = parts.transpose(2, 3).contiguous().transpose(2, 3)
    for p in (parts, odd, heads_first, turned):
        assert torch.equal(b.attention(*p.split((4, 2, 2), 2), causal=True), plain)
    # the same keys for both sequences, and one row of keys throughout
    one = b.attention(q, k[:1].expand(2, -1, -1, -1), v[:1].expand(2, -1, -1, -1), causal=True)
    assert torch.equal(one, b.attention(q, k[:1].repeat(2, 1, 1, 1), v[:1].repeat(2, 1, 1, 1), causal=True))
    same = b.attention(q, k[:, :1].expand(-1, 70, -1, -1), v[:, :1].expand(-1, 70, -1, -1), causal=True)
    assert torch.equal(same, b.attention(q, k[:, :1].repeat(1, 70, 1, 1), v[:, :1].repeat(1, 70, 1, 1), causal=True))


@pytest.mark.parametrize("dtype", TYPES)
def test_gradients_of_views_and_broadcast_inputs(dtype):
    b, d = blocks(), 40
    parts = leaf(normal(1, 2, 50, 6, d, dtype=dtype))
    dy = normal(2, 2, 50, 4, d, dtype=dtype)
    q, k, v = parts.split((4, 1, 1), 2)
    (g,) = torch.autograd.grad(b.attention(q, k, v, causal=True), parts, dy.cuda())
    q, k, v = (t.detach().cpu() for t in (q, k, v))
    want = stack([ref.attention(q[i], k[i], v[i], dy[i], True, d ** -0.5) for i in (0, 1)])
    against(dict(zip(("dq", "dk", "dv"), g.split((4, 1, 1), 2))), want, "views")
    # one sequence's keys for both: its gradient is the two's sum, which autograd rounds
    k1, v1 = leaf(k[:1]), leaf(v[:1])
    y = b.attention(q.cuda(), k1.expand(2, -1, -1, -1), v1.expand(2, -1, -1, -1), causal=True)
    gk, gv = torch.autograd.grad(y, (k1, v1), dy.cuda())
    want = stack([ref.attention(q[i], k[0], v[0], dy[i], True, d ** -0.5) for i in (0, 1)])
    for n, t in (("dk", gk), ("dv", gv)):
        value = want[n][0].sum(0, keepdim=True)
        ref.within(t, (value, want[n][1].sum(0, keepdim=True) + ref.rounded(value, dtype)), n)
    # an incoming gradient that is one value
    q1, k1, v1 = (leaf(t) for t in (q, k, v))
    got = torch.autograd.grad(b.attention(q1, k1, v1).sum(), (q1, k1, v1))
    one = torch.ones(50, 4, d, dtype=dtype)
    against(dict(zip(("dq", "dk", "dv"), got)), stack([ref.attention(q[i], k[i], v[i], one, False, d ** -0.5) for i in (0, 1)]), "ones")


def test_only_what_is_needed():
    b = blocks()
    q, k, v = (normal(i, 1, 40, 2, 64, dtype=BF).cuda() for i in range(3))
    dy = normal(4, 1, 40, 2, 64, dtype=BF).cuda()
    a = [t.clone().requires_grad_() for t in (q, k, v)]
    want = torch.autograd.grad(b.attention(*a, causal=True), a, dy)
    for i in range(3):
        a = [q, k, v]
        a[i] = a[i].clone().requires_grad_()
        (g,) = torch.autograd.grad(b.attention(*a, causal=True), a[i], dy)
        assert torch.equal(g, want[i])


def test_gradients_against_differences():
    # fp32: a central difference along one direction; h^2 times a third derivative and the results' rounding over h are
    # both below 1e-3 of the derivative's scale at h = 2^-7
    b, h = blocks(), 2.0 ** -7
    ts = [normal(i, 60, n, 24).cuda() for i, n in ((1, 6), (2, 2), (3, 2))]
    ways = [normal(i, *t.shape).cuda() for i, t in zip((4, 5, 6), ts)]
    offs = torch.tensor([0, 17, 17, 60], dtype=torch.int32, device="cuda")
    dy = normal(7, *ts[0].shape).cuda()
    f = lambda *a: (b.attention(*a, causal=True, offsets=offs).double() * dy.double()).sum()  # noqa: E731
    leaves = [t.clone().requires_grad_() for t in ts]
    grads = torch.autograd.grad(b.attention(*leaves, causal=True, offsets=offs), leaves, dy)
    for i in range(3):
        up, down = list(ts), list(ts)
        up[i], down[i] = ts[i] + h * ways[i], ts[i] - h * ways[i]
        want = (f(*up) - f(*down)) / (2 * h)
        got = (grads[i].double() * ways[i].double()).sum()
        size = grads[i].double().norm() * ways[i].double().norm()
        assert abs(got - want) < 1e-3 * size


@pytest.mark.parametrize("nq,nk", [(1, 700), (200, 200)])
def test_other_stream_and_repeat(nq, nk):
    b = blocks()
    q, k, v = (normal(i, 2, n, m, 64, dtype=BF).cuda().requires_grad_() for i, (n, m) in enumerate(((nq, 8), (nk, 2), (nk, 2))))

    def f():
        y = b.attention(q, k, v, causal=True)
        return (y.detach(), *torch.autograd.grad(y, (q, k, v), torch.ones_like(y)))
    want = f()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = f()
    side.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)


def test_offsets_beyond_31_bits():
    # a cache of 2.4e9 values a tensor, of which the last sequence's last head is looked at
    b = blocks()
    B, S, hk, d = 3, 100_003, 64, 128
    g = torch.Generator("cuda").manual_seed(1)
    k = torch.empty(B, S, hk, d, dtype=BF, device="cuda")
    v = torch.empty_like(k)
    for t in (k, v):
        for i in range(B):
            t[i].normal_(generator=g)
    q = torch.randn(B, 1, hk, d, device="cuda", generator=g).to(BF)
    lens = torch.tensor([7, 0, S], dtype=torch.int32, device="cuda")
    y = b.attention(q, k, v, causal=True, key_lengths=lens)
    assert not y[1].any()
    for seq, n in ((0, 7), (2, S)):
        for head in (0, hk - 1):
            s = (k[seq, :n, head].double() @ q[seq, 0, head].double()) * d ** -0.5
            want = torch.softmax(s, 0) @ v[seq, :n, head].double()
            # weights and result are rounded to bf16: 2^-8 of sum p |v| and of the value; sums and exponents far less
            bound = 2.1 * 2.0 ** -8 * (torch.softmax(s, 0) @ v[seq, :n, head].double().abs())
            assert ((y[seq, 0, head].double() - want).abs() <= bound).all()
    # many queries over the same keys
    q = torch.randn(B, 40, hk, d, device="cuda", generator=g).to(BF)
    lens[0] = 300
    y = b.attention(q, k[:, -300:], v[:, -300:], causal=True, key_lengths=lens)
    one = ref.attention(q[2, :, -2:].cpu(), k[2, -300:, -2:].cpu(), v[2, -300:, -2:].cpu(), None, True, d ** -0.5)["y"]
    ref.within(y[2, :, -2:], one, "many")


def test_refusals():
    b = blocks()
    q, k = torch.zeros(2, 4, 4, 8, device="cuda"), torch.zeros(2, 5, 2, 8, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(q=q, k=k, v=k)
    b.attention(**good)
    for bad in (dict(q=q.cpu()), dict(q=q.half()), dict(k=k.int()), dict(q=q[0]), dict(v=k[:, :4]), dict(k=k[:1], v=k[:1]),
                dict(q=q[:, :, :3]), dict(q=q[..., :7]), dict(q=q[:, :, :0]), dict(k=k[:, :, :0], v=k[:, :, :0]), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(key_lengths=i32(1)),
                dict(key_lengths=i32(1, 2).long()), dict(key_lengths=i32(1, 2).cpu()), dict(key_lengths=[1, 2]), dict(offsets=i32(0, 4)),
                dict(key_offsets=i32(0, 4))):
        with pytest.raises(ValueError):
            b.attention(**{**good, **bad})
    good = dict(q=q[0], k=k[0], v=k[0], offsets=i32(0, 4))
    b.attention(**good)
    for bad in (dict(offsets=i32(0, 4).long()), dict(offsets=i32(0, 4).cpu()), dict(offsets=i32()), dict(offsets=i32(0, 4).view(1, 2)),
                dict(key_offsets=i32(0, 2, 4)), dict(key_lengths=i32(4)), dict(q=q)):
        with pytest.raises(ValueError):
            b.attention(**{**good, **bad})
    wide = torch.zeros(1, 2, 1, 136, device="cuda")
    with pytest.raises(ValueError):
        b.attention(wide, wide, wide)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("n,h,hk,d", [(130, 4, 4, 64), (700, 2, 2, 72), (1, 4, 1, 128), (520, 3, 1, 128)])
def test_gradients_are_as_near_as_their_types(n, h, hk, d, dtype):
    # dq and dk come from ds rounded to 16 bits, and are rounded: two independent errors of one size, sqrt(2) times
    # what rounding the 64-bit result costs.  6 % more for all else, weights and delta among it.
    # Where ds is 0 (one key), fp32 remains: dp and delta are sums of d products, each off by (d + 8) 2^-24 of their
    # magnitudes' sum, so ds is off by at most p E, E = 2 (d + 8) 2^-24 max_ij sum |dy_i v_j|.  As a row's p sum to 1, a
    # row of dq is then off by scale E max |k_j|, and all of dk by scale E max |q_i| a row of queries.
    q, k, v, dy = (normal(60 + i, 2, n, m, d, dtype=dtype) for i, m in enumerate((h, hk, hk, h)))
    want = stack([ref.attention(q[b], k[b], v[b], dy[b], True, d ** -0.5) for b in range(2)])
    ts = [leaf(t) for t in (q, k, v)]
    got = torch.autograd.grad(blocks().attention(*ts, causal=True), ts, dy.cuda())
    norms = {name: t.double().norm(dim=-1).max() for name, t in (("q", q), ("k", k), ("v", v), ("dy", dy))}
    rows, E = 2 * n * h, 2 * (d + 8) * 2.0 ** -24 * norms["dy"] * norms["v"]
    left = {"dq": rows ** 0.5 * d ** -0.5 * E * norms["k"], "dk": rows * d ** -0.5 * E * norms["q"]}
    for name, t in zip(("dq", "dk"), got):
        value = want[name][0]
        rounding = (value.to(dtype).double() - value).norm()
        assert (t.cpu().double() - value).norm() <= 1.06 * 2 ** 0.5 * rounding + left[name], name


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("scale,spread", [(2.0 ** -64, 1.0), (2.0 ** 64, 2.0 ** -32)])
def test_largest_and_smallest_scales(scale, spread, dtype):
    # (fp16 does not hold such inputs and gradients)
    run_batch(1, 150, 150, 2, 1, 64, dtype, True, scale=scale, spread=spread, seed=10)
    run_batch(1, 3, 600, 2, 1, 64, dtype, False, scale=scale, spread=spread, seed=11)


def test_scales_out_of_range_are_refused():
    q = torch.zeros(1, 2, 1, 8, device="cuda")
    for scale in (2.0 ** -65, 2.0 ** 65):
        with pytest.raises(ValueError):
            blocks().attention(q, q, q, scale=scale)


def test_one_tensor_for_all_and_shared_batches():
    # q, k and v one tensor, whose gradient is the sum; keys that all sequences share (no stride between them)
    b = blocks()
    x, dy = normal(1, 2, 70, 3, 64), normal(2, 2, 70, 3, 64)
    want = stack([ref.attention(x[i], x[i], x[i], dy[i], True, 0.125) for i in range(2)])
    t = leaf(x)
    (g,) = torch.autograd.grad(b.attention(t, t, t, causal=True), t, dy.cuda())
    value = sum(want[n][0] for n in ("dq", "dk", "dv"))
    bound = sum(want[n][1] for n in ("dq", "dk", "dv")) + 2 * 2.0 ** -24 * value.abs()   # and two sums in fp32
    ref.within(g, (value, bound), "one tensor")
    k = normal(3, 1, 70, 3, 64)
    want = stack([ref.attention(x[i], k[0], k[0], None, False, 0.125) for i in range(2)])
    shared = k.cuda().expand(2, 70, 3, 64)
    ref.within(b.attention(x.cuda(), shared, shared), want["y"], "shared keys")


def test_lengths_and_offsets_beyond_the_tokens():
    # taken to the tokens' ends
    b = blocks()
    q, k = normal(1, 3, 4, 2, 64, dtype=BF).cuda(), normal(2, 3, 50, 2, 64, dtype=BF).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    assert torch.equal(b.attention(q, k, k, causal=True, key_lengths=i32(-3, 51, 2 ** 31 - 1)),
                       b.attention(q, k, k, causal=True, key_lengths=i32(0, 50, 50)))
    x = normal(3, 64, 2, 64, dtype=BF).cuda()
    for bad, good in (((-5, 40, 1000), (0, 40, 64)), ((64, 2 ** 31 - 1), (64, 64)), ((-2 ** 31, -1, 3), (0, 0, 3))):
        t, u = x.clone().requires_grad_(), x.clone().requires_grad_()
        y, z = b.attention(t, t, t, offsets=i32(*bad)), b.attention(u, u, u, offsets=i32(*good))
        assert torch.equal(y, z)
        y.sum().backward()
        z.sum().backward()
        assert torch.equal(t.grad, u.grad)
