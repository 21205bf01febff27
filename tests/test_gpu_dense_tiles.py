"""Every product kernel of the dense operators against fp64 on the GPU, with the
worst-case bounds of dense_ref, at the sizes of dense_sizes."""
import pytest
import torch

import dense_ref as ref
import dense_sizes as sizes
from test_gpu_dense_range import plain_product

pytestmark = pytest.mark.gpu


def dense():
    from differentiable_gaussian_splatting_pdr_amd import dense as d
    return d


def normal(seed, *shape, scale=1.0, dtype=torch.float32):
    g = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def within(got, want, what):
    value, bound = want
    got = got.detach().double()
    assert got.shape == value.shape and torch.isfinite(got).all(), what
    worst = ((got - value).abs() / bound).max().item()
    assert worst <= 1.0, "%s: %.3g times its bound" % (what, worst)


@pytest.mark.parametrize("dtype,out,M,K,N,act,residual", sizes.LINEAR)
def test_linear(dtype, out, M, K, N, act, residual, monkeypatch):
    if dtype == torch.float32:
        monkeypatch.setattr(ref, "product", plain_product)
    x, w = normal(1, M, K, dtype=dtype), normal(2, N, K, scale=K ** -0.5, dtype=dtype)
    b, dy = normal(3, N, dtype=dtype), normal(4, M, N, dtype=out)
    r = normal(5, M, N, dtype=out) if residual else None
    want = ref.linear(x, w, b, r, act, dy, out)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    y = dense().linear(x, w, b, residual=r, activation=act, out_dtype=out)
    within(y, want["y"], "y")
    for k, g in zip(("dx", "dw", "db"), torch.autograd.grad(y, leaves, dy)):
        within(g, want[k], k)


@pytest.mark.parametrize("dtype,M,D,F,O", sizes.GATED)
def test_gated(dtype, M, D, F, O, monkeypatch):
    if dtype == torch.float32:
        monkeypatch.setattr(ref, "product", plain_product)
    x, r, dy = normal(1, M, D, dtype=dtype), normal(2, M, O, dtype=dtype), normal(3, M, O, dtype=dtype)
    wi, wo = normal(4, 2 * F, D, scale=D ** -0.5, dtype=dtype), normal(5, O, F, scale=F ** -0.5, dtype=dtype)
    want = ref.gated(x, wi, wo, r, "silu", dy)
    leaves = [t.requires_grad_() for t in (x, wi, wo)]
    y = dense().gated_mlp(x, wi, wo, residual=r)
    within(y, want["y"], "y")
    for k, g in zip(("dx", "dw_in", "dw_out"), torch.autograd.grad(y, leaves, dy)):
        within(g, want[k], k)


@pytest.mark.parametrize("dtype,batch,m,n", sizes.ORTHOGONALIZE)
def test_orthogonalize(dtype, batch, m, n):
    # two steps take every product; the bound is test_gpu_dense's: iterates
    # rounded three times a step, a relative error that grows by the steps' count
    g = normal(m + n, batch, m, n, dtype=dtype)
    want = ref.orthogonalize(g, 2, (3.4445, -4.7750, 2.0315), 1e-7)
    got = dense().orthogonalize(g, steps=2).double()
    plane = 2.0 ** -12 if dtype == torch.bfloat16 else 2.0 ** -21
    off = ((got - want).norm(dim=(-2, -1)) / want.norm(dim=(-2, -1))).max().item()
    assert off <= 2 * 3 * (plane + (m + n) * 2.0 ** -24) + ref.U[dtype], off
