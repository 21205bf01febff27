"""A query's result and gradient are a function of what it sees alone, to the last bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = (torch.bfloat16, torch.float16, torch.float32)


def normal(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def run(q, k, v, dy):
    from differentiable_gaussian_splatting_pdr_amd import blocks
    q = q.detach().requires_grad_()
    y = blocks.attention(q, k, v, causal=True)
    return y.detach(), torch.autograd.grad(y, q, dy)[0]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("nq,nk,h,hk,d", [(30, 300, 4, 4, 64), (90, 1200, 2, 1, 128), (150, 150, 256, 256, 64), (140, 333, 256, 256, 128)])
def test_rows_beside_it_do_not_matter(nq, nk, h, hk, d, dtype):
    # the last two sizes take 128 rows to a workgroup
    q, k, v, dy = (normal(i, 1, n, m, d, dtype=dtype) for i, (n, m) in enumerate(((nq, h), (nk, hk), (nk, hk), (nq, h))))
    clean = run(q, k, v, dy)
    for row in (nq - 1, nq // 2):
        # one row's scores grow by far more, and with them its maximum
        x = q.clone()
        x[:, row] *= 48
        keep = [i for i in range(nq) if i != row]
        for got, want in zip(run(x, k, v, dy), clean):
            assert torch.equal(got[:, keep], want[:, keep])
        # a key that only later rows see
        x = k.clone()
        x[:, row + nk - nq] *= 48
        for got, want in zip(run(q, x, v, dy), clean):
            assert torch.equal(got[:, :row], want[:, :row])
