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
