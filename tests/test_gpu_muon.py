"""The Muon optimiser on the GPU: updates against the formula in 64 bits."""
import pytest
import torch

import dense_ref as ref

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
NS = (3.4445, -4.7750, 2.0315)


def dense():
    from differentiable_gaussian_splatting_pdr_amd import dense as d
    return d


def normal(seed, *shape, scale=1.0, dtype=FP):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


# As in test_gpu_dense: iterates rounded three times a step.
def ortho_bound(m, n, dtype):
    plane = 2.0 ** -12 if dtype == BF else 2.0 ** -21
    return 5 * 3 * (plane + (m + n) * 2.0 ** -24) + ref.U[dtype]


@pytest.mark.parametrize("scale", [1e-30, 1e-10, 1e-7, 1.0, 1e6, 1e30])
@pytest.mark.parametrize("shape", [(40, 24), (16, 70)])
def test_update_in_fp16_does_not_see_the_gradients_scale(scale, shape):
    # the state is fp32, and so is what the orthogonalisation starts from
    d = dense()
    p = torch.zeros(*shape, device="cuda", requires_grad=True)
    g = normal(1, *shape, scale=scale)
    p.grad = g.cuda()
    d.Muon([p], lr=1.0, momentum=0.9, work_dtype=HF).step()
    u = ref.orthogonalize(1.9 * g.double(), 5, NS, 1e-7) * max(1, shape[0] / shape[1]) ** 0.5
    off = (p.detach().cpu().double() + u).norm() / max(u.norm(), 1e-300)
    # the update is a value of fp16: where eps makes it small, a multiple of the type's step
    assert off <= ortho_bound(*shape, HF) + 2.0 ** -25 * (shape[0] * shape[1]) ** 0.5 / max(u.norm(), 1e-300)


@pytest.mark.parametrize("scale", [1e-6, 6e4])
def test_fp16_weights_with_gradients_at_the_ends_of_their_range(scale):
    # momentum reaches 20 gradients: the fp32 state holds what fp16 does not
    d = dense()
    p = normal(1, 48, 32, dtype=HF).cuda().requires_grad_()
    want, buf = p.detach().cpu().double(), 0
    opt = d.Muon([p], lr=0.125, momentum=0.95)
    for k in range(4):
        g = (normal(2, 48, 32).clamp(-1, 1) * scale + 0.01 * scale * normal(3 + k, 48, 32).clamp(-1, 1)).to(HF)
        p.grad = g.cuda()
        opt.step()
        buf = 0.95 * buf + g.double()
        u = ref.orthogonalize(g.double() + 0.95 * buf, 5, NS, 1e-7) * (48 / 32) ** 0.5
        want = want - 0.125 * u
        off = p.detach().cpu().double() - want
        # p is rounded, and the update by its bound of the whole matrix's norm
        assert torch.isfinite(off).all()
        assert off.norm() <= (0.125 * ortho_bound(48, 32, HF) * u.norm() + 2.0 ** -11 * want.norm()), k
        want = p.detach().cpu().double()


@pytest.mark.parametrize("dtype", (BF, HF))
def test_16_bit_weights_follow_the_formula(dtype):
    d = dense()
    p = normal(9, 16, 32, dtype=dtype).cuda().requires_grad_()
    opt = d.Muon([p], lr=0.1, momentum=0.9, weight_decay=0.01)
    buf = 0
    for k in range(3):
        before = p.detach().cpu().double()
        g = normal(100 + k, 16, 32, dtype=dtype)
        p.grad = g.cuda()
        opt.step()
        buf = 0.9 * buf + g.double()
        u = ref.orthogonalize(g.double() + 0.9 * buf, 5, NS, 1e-7)
        decayed = before * (1 - 0.001)
        want = decayed - 0.1 * u
        off = (p.detach().cpu().double() - want).norm()
        # rounded: what enters the orthogonalisation (relative to a norm of 1;
        # for singular values above 0.07 of it, which these matrices have, the
        # five steps' polynomial has a derivative below 32 and a ratio to its
        # argument below 17), the orthogonalisation, and the weight after its
        # decay and its update
        most = 0.1 * (u.norm() * ortho_bound(16, 32, dtype) + 32 * ref.U[dtype]) + ref.U[dtype] * (
            decayed.norm() + want.norm())
        assert off <= most, (k, off / most)


@pytest.mark.parametrize("dtype", (BF, HF, FP))
@pytest.mark.parametrize("shape", [(33, 129), (129, 33), (2, 40, 17)])
def test_orthogonalize_of_fp32_to_another_type(shape, dtype):
    d = dense()
    g = normal(3, *shape, scale=1e-9)
    want = ref.orthogonalize(g, 5, NS, 0.0)
    got = d.orthogonalize(g.cuda(), eps=0.0, dtype=dtype)
    assert got.dtype == dtype
    assert ((got.cpu().double() - want).norm() / want.norm()).item() <= ortho_bound(*shape[-2:], dtype)
    part = g.cuda()[..., 1:, 3:20]
    assert torch.equal(d.orthogonalize(part, dtype=dtype), d.orthogonalize(part.contiguous(), dtype=dtype))
    for bad in (g.cuda().half(), g.cuda().bfloat16()):
        for to in (torch.float32, torch.float64, torch.bfloat16 if bad.dtype == HF else HF):
            with pytest.raises(ValueError):
                d.orthogonalize(bad, dtype=to)


@pytest.mark.parametrize("steps", [5, 6])
@pytest.mark.parametrize("m,n", [(300, 2000), (336, 7000), (1024, 1024), (2000, 300)])
def test_bf16_orthogonalisation_is_as_exact_as_its_roundings(m, n, steps):
    # The error is that of rounding X, A and B once each step to fp16 under the
    # documented scales, and the result to bf16, in an fp64 chain; sums in fp32
    # add about (m + n)^(1/2) 2^-24 a step, their roundings' signs being
    # independent.  Which way a value rounds where sums differ moves the error
    # of a matrix by a few parts in a hundred: 1.1 times.
    a, b, c = NS
    g = torch.randn(m, n, device="cuda", generator=torch.Generator("cuda").manual_seed(m + n)).to(BF)
    want = ref.orthogonalize(g, steps, NS, 1e-7)

    def rounded(v, shift):
        return (v * 2.0 ** shift).to(HF).double() * 2.0 ** -shift
    x = g.double().t() if m > n else g.double()
    x = rounded(x / (x.pow(2).sum().sqrt() + 1e-7), 12)
    for k in range(steps):
        p = rounded(x @ x.t(), 10)
        x = a * x + rounded(b * p + c * (p @ p), 10) @ x
        x = rounded(x, 12) if k + 1 < steps else x.to(BF).double()
    x = x.t() if m > n else x
    norm = want.norm()
    allowed = 1.1 * ((x - want).norm() / norm) + steps * (m + n) ** 0.5 * 2.0 ** -24
    off = (dense().orthogonalize(g, steps=steps).double() - want).norm() / norm
    print("%dx%d, %d steps: %.2e, allowed %.2e" % (m, n, steps, off, allowed))
    assert off <= allowed
