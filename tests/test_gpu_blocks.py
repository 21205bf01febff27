"""Attention, layer norm and dropout as they are used: captured in graphs, on
other streams, one after another with the dense operators, and in the example."""
import os
import sys

import pytest
import torch

import blocks_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def ops():
    from differentiable_gaussian_splatting_pdr_amd import blocks, dense
    return blocks, dense


def normal(seed, *shape, scale=1.0, dtype=FP):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def leaf(t):
    return t.detach().cuda().requires_grad_()


def int32(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# each: (the tensors that it differentiates, what it computes of them)
def batched(dtype):
    b, _ = ops()
    return [leaf(normal(i, 2, 200, h, 64, dtype=dtype)) for i, h in enumerate((4, 2, 2))], \
        lambda q, k, v: b.attention(q, k, v, causal=True)


def few_keys_split(dtype):
    # few queries, whose keys' gradients and whose own sums are put together of parts
    b, _ = ops()
    return [leaf(normal(i, 1, n, h, 128, dtype=dtype)) for i, (n, h) in enumerate(((3, 4), (2500, 1), (2500, 1)))], \
        lambda q, k, v: b.attention(q, k, v, causal=True)


def packed(dtype):
    b, _ = ops()
    at = int32(2, 2, 90, 300)
    return [leaf(normal(i, 310, h, 40, dtype=dtype)) for i, h in enumerate((6, 3, 3))], \
        lambda q, k, v: b.attention(q, k, v, causal=True, offsets=at)


def filled_cache(dtype):
    b, _ = ops()
    lengths = int32(0, 777, 31)
    return [leaf(normal(i, 3, n, h, 64, dtype=dtype)) for i, (n, h) in enumerate(((2, 8), (800, 2), (800, 2)))], \
        lambda q, k, v: b.attention(q, k, v, causal=True, key_lengths=lengths)


def norm(cols):
    def make(dtype):
        b, _ = ops()
        return [leaf(normal(i, *s, dtype=dtype)) for i, s in enumerate(((700, cols), (cols,), (cols,)))], b.layer_norm
    return make


def drop(dtype):
    b, _ = ops()
    return [leaf(normal(i, 300, 130, dtype=dtype)) for i in range(2)], \
        lambda x, r: b.dropout(x, 0.3, 7, offset=2, residual=r)


OPERATORS = [batched, few_keys_split, packed, filled_cache, norm(136), norm(20000), drop]
NAMES = ["batched", "few", "packed", "cache", "norm", "long norm", "dropout"]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("make", OPERATORS, ids=NAMES)
def test_captured_in_a_graph(make, dtype):
    leaves, f = make(dtype)
    dy = torch.randn(leaves[0].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(5)).to(dtype)

    def step():
        y = f(*leaves)
        return (y.detach(), *torch.autograd.grad(y, leaves, dy))

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
            for i, t in enumerate(leaves):
                t.copy_(normal(20 + 5 * k + i, *t.shape))
        eager = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, c in zip(eager, out):
            assert torch.equal(a, c), k


def test_graphs_that_share_memory():
    # two captured passes with one pool, replayed in turn: no workspace of one is the other's input
    b, _ = ops()
    q, k, v = (normal(i, 2, n, h, 64, dtype=BF).cuda() for i, (n, h) in enumerate(((1, 8), (3000, 2), (3000, 2))))
    few = lambda: b.attention(q, k, v, causal=True)  # noqa: E731
    many = lambda: b.attention(k, v, k, causal=True)  # noqa: E731
    want = [f() for f in (few, many)]
    graphs, outs = [], []
    for f in (few, many):
        f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(f())
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
            torch.cuda.synchronize()
            few()
    for a, c in zip(want, outs):
        assert torch.equal(a, c)


def test_replays_draw_anew_from_a_seed_in_memory():
    b, _ = ops()
    seed = torch.tensor([5], device="cuda")
    x = leaf(normal(1, 64, 96))

    def step():
        y = b.dropout(x, 0.5, seed)
        return y.detach(), torch.autograd.grad(y, x, torch.ones_like(y))[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = step()
    seen = []
    for k in (5, 6, 2 ** 40 + 1):
        seed.fill_(k)
        graph.replay()
        torch.cuda.synchronize()
        with torch.no_grad():
            want = b.dropout(x, 0.5, k)
        assert torch.equal(y, want)
        keep = ref.kept(k, 0, 0, x.numel(), 0.5).view(x.shape)
        assert torch.equal(g.cpu(), keep * 2.0)
        seen.append(y.clone())
    assert not torch.equal(seen[0], seen[1])


@pytest.mark.parametrize("make", OPERATORS, ids=NAMES)
def test_two_streams_at_once(make):
    # two passes in flight, each with its own workspaces
    leaves, f = make(BF)
    others = [(t.detach() * 0.5).requires_grad_() for t in leaves]
    dy = torch.ones_like(leaves[0])

    def step(ts):
        y = f(*ts)
        return (y.detach(), *torch.autograd.grad(y, ts, dy))

    want = step(leaves), step(others)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(side):
            first = step(others)
        second = step(leaves)
        torch.cuda.synchronize()
        for got, ok in zip((second, first), want):
            assert all(torch.equal(a, c) for a, c in zip(got, ok))


@pytest.mark.parametrize("make", OPERATORS, ids=NAMES)
def test_gradients_twice_from_one_graph(make):
    leaves, f = make(HF)
    y = f(*leaves)
    dy = torch.ones_like(y)
    first = torch.autograd.grad(y, leaves, dy, retain_graph=True)
    ops()[0].layer_norm(normal(9, 4000, 64).cuda())   # something else in the memory that was freed
    second = torch.autograd.grad(y, leaves, dy)
    assert all(torch.equal(a, c) for a, c in zip(first, second))


def transformer(x, weights, seed, heads, kv_heads, product, attend, normalise, gated, drop):
    """Two blocks as a model has them."""
    for n in range(2):
        g1, b1, w_qkv, w_mix, g2, b2, w_in, w_out = weights[8 * n:8 * n + 8]
        d = w_mix.shape[1] // heads
        qkv = product(normalise(x, g1, b1), w_qkv).unflatten(-1, (heads + 2 * kv_heads, d))
        q, k, v = qkv.split((heads, kv_heads, kv_heads), dim=-2)
        x = drop(product(attend(q, k, v).flatten(-2), w_mix), seed, 2 * n, x)
        x = drop(gated(normalise(x, g2, b2), w_in, w_out), seed, 2 * n + 1, x)
    return x


def plain64(lengths, p):
    """The operators in 64 bits; `noise` after each, relative to what it returns."""
    def attend(q, k, v, noise):
        out, at = [], 0
        for n in lengths:
            qs, ks, vs = (t[at:at + n].transpose(0, 1) for t in (q, k, v))
            g = qs.shape[0] // ks.shape[0]
            s = qs @ ks.repeat_interleave(g, 0).transpose(1, 2) * qs.shape[-1] ** -0.5
            s = s.masked_fill(~torch.ones(n, n, dtype=torch.bool).tril(), -torch.inf)
            out.append((torch.softmax(s, -1) @ vs.repeat_interleave(g, 0)).transpose(0, 1))
            at += n
        return noise(torch.cat(out))

    def normalise(x, w, b, noise):
        return noise(torch.nn.functional.layer_norm(x, x.shape[-1:], w, b, 1e-5))

    def gated(x, w_in, w_out, noise):
        a, c = (x @ w_in.T).chunk(2, -1)
        return noise(noise(torch.nn.functional.silu(a) * c) @ w_out.T)

    def drop(x, seed, offset, residual, noise):
        keep = ref.kept(seed, offset, 0, x.numel(), p).view(x.shape)
        return noise(x * keep / (1 - p) + residual)

    def run(noise):
        return dict(product=lambda x, w: noise(x @ w.T), attend=lambda *a: attend(*a, noise),
                    normalise=lambda *a: normalise(*a, noise), gated=lambda *a: gated(*a, noise),
                    drop=lambda *a: drop(*a, noise))
    return run


class Noise(torch.autograd.Function):
    """x (1 + e u), and the same of its gradient, with u of random signs."""

    @staticmethod
    def forward(ctx, x, e, g):
        ctx.e, ctx.g = e, g
        return x + e * x.abs().mean() * (torch.randint(0, 2, x.shape, generator=g) * 2 - 1)

    @staticmethod
    def backward(ctx, dy):
        return dy + ctx.e * dy.abs().mean() * (torch.randint(0, 2, dy.shape, generator=ctx.g) * 2 - 1), None, None


def test_transformer_blocks():
    # the operators together, forward and backward, in packed sequences: fp32 against 64 bits.  An operator's results
    # are off by at most (n + 8) 2^-24 of the magnitudes that are summed (n = 128 terms here), which are up to
    # sqrt(n) times the results' mean.  The tolerance is 4 times what errors of that size and random signs after
    # each operator do to the 64-bit results, as the largest of three draws.
    b, dense = ops()
    lengths, heads, kv_heads, d, hidden, p = (37, 0, 1, 90), 4, 2, 32, 96, 0.25
    width, T = heads * d, 128
    shapes = [(width,), (width,), ((heads + 2 * kv_heads) * d, width), (width, width),
              (width,), (width,), (2 * hidden, width), (width, hidden)] * 2
    weights = [normal(i, *s, scale=s[-1] ** -0.5) + (1.0 if i % 4 == 0 and len(s) == 1 else 0.0) for i, s in enumerate(shapes)]
    x, dy, seed = normal(50, T, width), normal(51, T, width), 11

    def in64(noise):
        ts = [t.double().requires_grad_() for t in (x, *weights)]
        y = transformer(ts[0], ts[1:], seed, heads, kv_heads, **plain64(lengths, p)(noise))
        return [y.detach(), *torch.autograd.grad(y, ts, dy.double())]

    want = in64(lambda t: t)
    e = 136 * 2.0 ** -24 * 128 ** 0.5
    off = [0.0] * len(want)
    for draw in range(3):
        g = torch.Generator().manual_seed(draw)
        got = in64(lambda t: Noise.apply(t, e, g))
        off = [max(o, float((a - c).norm())) for o, a, c in zip(off, got, want)]

    ts = [leaf(t) for t in (x, *weights)]
    at = int32(0, 37, 37, 38, 128)
    y = transformer(ts[0], ts[1:], seed, heads, kv_heads, dense.linear,
                    lambda q, k, v: b.attention(q, k, v, causal=True, offsets=at), b.layer_norm,
                    lambda t, w_in, w_out: dense.gated_mlp(t, w_in, w_out),
                    lambda t, s, offset, residual: b.dropout(t, p, s, offset=offset, residual=residual))
    got = [y.detach(), *torch.autograd.grad(y, ts, dy.cuda())]
    for i, (a, c, o) in enumerate(zip(got, want, off)):
        assert float((a.cpu().double() - c).norm()) <= 4 * o, i


def example():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import fit_predictor
    return fit_predictor


def test_example_runs_with_attention():
    losses = example().train(steps=3, B=2, heads=4, kv_heads=2, dropout=0.1, width=128, hidden=160)
    assert len(losses) == 3 and all(v == v and v < float("inf") for v in losses)


@pytest.mark.parametrize("seed", [None, 3])
def test_example_gradients_against_differences(seed):
    # as far as the Gaussians' raw values, in fp32; a central difference's rounding and third order are
    # of the order of 1e-4 of the gradient's and the step's sizes
    torch.manual_seed(1)
    net = example().Predictor(16, 64, 48, 2, 4, 4, 16, 16, 3, dtype=FP, heads=4, kv_heads=2, p=0.25)
    x = normal(1, 2, 16, 16).cuda()
    way = normal(2, 2, 16, 8).cuda()
    f = lambda: (net.raw(x, seed).double() * way.view_as(net.raw(x, seed))).sum()  # noqa: E731
    params = dict(net.named_parameters())
    grads = dict(zip(params, torch.autograd.grad(f(), list(params.values()))))
    for i, (name, t) in enumerate(params.items()):
        assert grads[name].abs().sum() > 0, name
        u = normal(100 + i, *t.shape).cuda()
        u = u / u.norm()
        h = 2e-3
        with torch.no_grad():
            t.add_(u, alpha=h)
            up = f()
            t.add_(u, alpha=-2 * h)
            down = f()
            t.add_(u, alpha=h)
        got = (grads[name].double() * u.double()).sum()
        assert abs(got - (up - down) / (2 * h)) < 1e-3 * grads[name].double().norm() + 1e-2, name
