"""Attention whose many small weights add up to what counts."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = (torch.bfloat16, torch.float16, torch.float32)
N, D = 65536, 8
CALLS = pytest.mark.parametrize("queries,heads", [(1, 1), (1, 8), (129, 128)])   # the last: 128 rows to a workgroup
GAPS = pytest.mark.parametrize("gap", [12.0, 17.0, 20.5])
PLACES = pytest.mark.parametrize("at", [0, 3, 40000, 65535])


def blocks():
    from differentiable_gaussian_splatting_pdr_amd import blocks as b
    return b


def one_large_key(queries, heads, at, gap, dtype):
    """(result, the others' weights' sum relative to the large one): key `at` has a score of 0 and a value of
    (1, 0, ..), the others, with (0, 1, ..), a score of -gap."""
    q = torch.zeros(1, queries, heads, D, dtype=dtype, device="cuda")
    q[..., 0] = 1.0
    k, v = (torch.zeros(1, N, 1, D, dtype=dtype, device="cuda") for _ in range(2))
    k[..., 0] = -gap
    k[:, at, :, 0] = 0.0
    v[..., 1] = 1.0
    v[:, at, :, 0], v[:, at, :, 1] = 1.0, 0.0
    kv = 1 if queries == 1 else heads
    y = blocks().attention(q, k.expand(1, N, kv, D), v.expand(1, N, kv, D), scale=1.0)
    return y.double(), (N - 1) * math.exp(-gap)


@pytest.mark.parametrize("dtype", TYPES)
@GAPS
@PLACES
@CALLS
def test_sum_of_many_small_weights(queries, heads, at, gap, dtype):
    # The large key's share is 1 / (1 + small), and its weight no product's sum: what it is off by is the sum of the
    # weights (at most N / 64 tiles follow one another, and 32 weights in each: 1.1 2^10 2^-25), their exponents
    # (scores of up to 20.5 times log2(e) in fp32, 30 2^-23; exp2 2^-21) and its rounding.
    y, small = one_large_key(queries, heads, at, gap, dtype)
    want = 1 / (1 + small)
    assert ((y[..., 0] - want).abs() <= want * (1.1 * 2.0 ** -15 + 2.0 ** -17 + torch.finfo(dtype).eps / 2)).all()


@GAPS
@PLACES
@CALLS
def test_values_of_many_small_weights_in_fp16(queries, heads, at, gap):
    # The others' share is small / (1 + small).  Their weights are all alike, so it is off by one weight's and its own
    # rounding to fp16 (2^-11 each), what the above says of the sum, the products' sum (N / 16 steps follow one
    # another, of 2^-25 each), and by N times half a weight's smallest step, which is 2^-37 of the largest.
    y, small = one_large_key(queries, heads, at, gap, torch.float16)
    want = small / (1 + small)
    bound = want * (2 * 2.0 ** -11 + 1.1 * 2.0 ** -15 + 2.0 ** -17 + 2.0 ** -13) + N * 2.0 ** -37
    assert ((y[..., 1] - want).abs() <= bound).all()
