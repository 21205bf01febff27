"""The dense operators at the ends of what their arguments allow."""
import ctypes

import pytest
import torch

from differentiable_gaussian_splatting_pdr_amd import _lib

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [2 ** 31 - 257, 2 ** 31 - 262144 + 1])
def test_bias_gradient_of_as_many_rows_as_there_may_be(M):
    # the last workgroup's rows would end past 2^31
    dy = torch.zeros(M, dtype=torch.bfloat16, device="cuda")
    dy[-300:] = 1
    dy[5] = 2
    db = torch.full((1,), -1, dtype=torch.bfloat16, device="cuda")
    a = _lib.pdr_linear(fmt=2, out_fmt=2, M=M, N=1, K=0, dy=dy.data_ptr(), lddy=1, dbias=db.data_ptr())
    size = _lib.lib().pdr_linear_backward_workspace_bytes(ctypes.byref(a))
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    assert _lib.lib().pdr_linear_backward(ctypes.byref(a), ws.data_ptr(), size,
                                          torch.cuda.current_stream().cuda_stream) == 0
    assert db.item() == 302   # a value of bf16


def test_rows_far_apart():
    # rows 2^22 + 64 values apart: a narrow view of a wide tensor
    from differentiable_gaussian_splatting_pdr_amd import dense
    wide = torch.zeros(5, (1 << 22) + 64, dtype=torch.bfloat16, device="cuda")
    near = torch.randn(5, 40, device="cuda", generator=torch.Generator("cuda").manual_seed(1)).to(torch.bfloat16)
    wide[:, 8:48] = near
    x = wide[:, 8:48]
    w = near[:3].contiguous()
    assert torch.equal(dense.linear(x, w), dense.linear(near, w))
    assert torch.equal(dense.linear(near, x), dense.linear(near, near))
    assert torch.equal(dense.linear(near, near[:, :40], residual=x[:, :5]),
                       dense.linear(near, near[:, :40], residual=near[:, :5]))
    y = dense.gated_mlp(x, near[:4], near[:, :2].contiguous())
    assert torch.equal(y, dense.gated_mlp(near, near[:4], near[:, :2].contiguous()))
    assert torch.equal(dense.orthogonalize(x), dense.orthogonalize(near))
    # a gradient with such rows
    v = near.clone().requires_grad_()
    (want,) = torch.autograd.grad(dense.linear(v, near.repeat(8, 1)), v, near)
    (got,) = torch.autograd.grad(dense.linear(v, near.repeat(8, 1)), v, x)
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("c,steps", [((0.0, 30.0, 25.0), 1), ((7.0, 0.0, 0.0), 2), ((0.0, -80.0, 80.0), 1), ((100.0, 0.0, 0.0), 1)])
def test_coefficients_at_the_end_of_the_iterates_range(c, steps, dtype):
    # one singular value, at 1 or in the middle, so that one entry holds it all
    from differentiable_gaussian_splatting_pdr_amd import PdrError, dense
    for other in (0.0, 1.0):
        g = torch.zeros(24, 40, dtype=dtype, device="cuda")
        g[2, 3], g[5, 7] = 1, other
        x = 2 ** -0.5 if other else 1.0
        for _ in range(steps):
            x = c[0] * x + (c[1] + c[2] * x * x) * x ** 3
        want = torch.zeros(24, 40, dtype=torch.float64)
        want[2, 3] = x
        want[5, 7] = x * other
        got = dense.orthogonalize(g, steps, c, 0.0).cpu().double()
        # powers of two and sums of two terms: each iterate rounded three times a step to 2^-12 of itself, of terms up to 80
        assert (got - want).abs().max() <= 80 * (steps + 1) * 3 * 2.0 ** -12 + 2.0 ** -8 * abs(x)
    for bad, n in (((0.0, 40.0, 40.0), 1), ((100.0, 0.0, 0.0), 2), ((2.0, 1.0, 1.0), 3)):
        with pytest.raises(PdrError):
            dense.orthogonalize(g, n, bad)


def test_more_rows_than_a_launch_of_small_tiles_holds():
    from differentiable_gaussian_splatting_pdr_amd import dense
    M = 2 ** 30 + 100001
    x = torch.zeros(M, 8, dtype=torch.bfloat16, device="cuda")
    w = torch.arange(1, 9, dtype=torch.bfloat16, device="cuda")[None]
    at = torch.tensor([0, 1, 63, 64, 2 ** 30 - 1, 2 ** 30, 2 ** 30 + 65536, M - 129, M - 2, M - 1], device="cuda")
    x[at] = torch.arange(1, 11, dtype=torch.bfloat16, device="cuda")[:, None]
    y = dense.linear(x, w)
    # 36 times the row's value, rounded to bf16
    assert torch.equal(y[at, 0], (36.0 * torch.arange(1, 11, device="cuda")).to(torch.bfloat16))
    assert y.count_nonzero() == 10


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gated_offsets_beyond_31_bits(dtype):
    # 2.3e9 gate and up sums, 1.15e9 values of h: the last rows, and their gradients
    import dense_ref as ref
    from differentiable_gaussian_splatting_pdr_amd import dense
    from test_gpu_dense_range import plain_product
    M, D, F, O = 280_003, 16, 4104, 8
    gen = torch.Generator("cuda").manual_seed(1)
    x, wi, wo = (torch.randn(*s, device="cuda", generator=gen).mul_(k).to(dtype).requires_grad_()
                 for s, k in (((M, D), 1.0), ((2 * F, D), D ** -0.5), ((O, F), F ** -0.5)))
    y = dense.gated_mlp(x, wi, wo)
    at = torch.tensor([0, 1, 131071, 131072, 261633, 261634, 262143, 262144, M - 130, M - 2, M - 1], device="cuda")
    dy = torch.zeros_like(y)
    dy[at] = torch.randn(len(at), O, device="cuda", generator=gen).to(dtype)
    gx, gi, go = torch.autograd.grad(y, (x, wi, wo), dy)
    keep = ref.product
    try:
        ref.product = plain_product if dtype == torch.float32 else keep
        want = ref.gated(*(t.detach() for t in (x[at], wi, wo)), None, "silu", dy[at])
    finally:
        ref.product = keep
    # the weights' gradients sum 280000 rows, all but eleven of them zero
    for k, t in (("y", y[at]), ("dx", gx[at]), ("dw_in", gi), ("dw_out", go)):
        value, bound = want[k]
        assert ((t.double() - value).abs() <= bound).all(), k
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[at] = False
    assert not gx[others].any()


def test_fp32_offsets_beyond_31_bits():
    # planes of 2.25e9 values each
    import dense_ref as ref
    from differentiable_gaussian_splatting_pdr_amd import dense
    from test_gpu_dense_range import plain_product
    M, K, N = 1_100_003, 2048, 16
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.randn(M, K, device="cuda", generator=gen).requires_grad_()
    w = (torch.randn(N, K, device="cuda", generator=gen) * K ** -0.5).requires_grad_()
    y = dense.linear(x, w)
    at = torch.tensor([0, 1, 524287, 524288, 1048575, 1048576, M - 130, M - 2, M - 1], device="cuda")
    dy = torch.zeros_like(y)
    dy[at] = torch.randn(len(at), N, device="cuda", generator=gen)
    gx, gw = torch.autograd.grad(y, (x, w), dy)
    keep = ref.product
    try:
        ref.product = plain_product
        want = ref.linear(x.detach()[at], w.detach(), None, None, "none", dy[at], torch.float32)
    finally:
        ref.product = keep
    for k, t in (("y", y[at]), ("dx", gx[at]), ("dw", gw)):
        value, bound = want[k]
        assert ((t.double() - value).abs() <= bound).all(), k
    others = torch.ones(M, dtype=torch.bool, device="cuda")
    others[at] = False
    assert not gx[others].any()
