"""Gradients where some of what attention reads is not finite."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = (torch.bfloat16, torch.float16, torch.float32)


def normal(seed, *shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def attention(*a, **kw):
    from differentiable_gaussian_splatting_pdr_amd import blocks
    return blocks.attention(*a, **kw)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("queries", [4, 700])   # one part of the rows, and several
def test_keys_behind_a_length_have_no_gradient(queries, d, causal, dtype):
    # whatever queries and incoming gradients hold
    lengths = [130, 0, 300, 77]
    q, dy = normal(1, 4, queries, 2, d, dtype=dtype), normal(2, 4, queries, 2, d, dtype=dtype)
    k, v = normal(3, 4, 300, 1, d, dtype=dtype), normal(4, 4, 300, 1, d, dtype=dtype)
    q[:, queries // 2, 0, 3] = float("nan")
    dy[:, queries - 1, 1, 5] = float("inf")
    ts = [t.requires_grad_() for t in (q, k, v)]
    y = attention(*ts, causal=causal, key_lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    _, dk, dv = torch.autograd.grad(y, ts, dy)
    for b, n in enumerate(lengths):
        assert not dk[b, n:].any() and not dv[b, n:].any()
        if n:
            assert not torch.isfinite(dv[b, :n]).all()
