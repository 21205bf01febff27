"""Sizes that attention, layer norm and dropout take and refuse, and what follows from
sizes alone, without a GPU."""
import ctypes

import pytest

from differentiable_gaussian_splatting_pdr_amd import _lib

FAKE = 0x10000  # 256-byte aligned, never dereferenced on these paths
MOST_COLS = 1 << 30


def norm(cols, rows=1):
    a = _lib.pdr_layer_norm(fmt=2, rows=rows, cols=cols, eps=1e-5)
    for name in ("x", "weight", "bias", "y", "stats", "dy", "dx", "dweight", "dbias"):
        setattr(a, name, FAKE)
    for name in ("ldx", "ldy", "lddy", "lddx"):
        setattr(a, name, cols)
    return a


def size(name, a):
    return getattr(_lib.lib(), name + "_workspace_bytes")(ctypes.byref(a))


@pytest.mark.parametrize("name", ["pdr_layer_norm_forward", "pdr_layer_norm_backward"])
@pytest.mark.parametrize("cols", [MOST_COLS + 1, (1 << 31) - 2048, (1 << 31) - 2047, (1 << 31) - 257])
def test_rows_longer_than_the_loops_count_are_refused(name, cols):
    # the kernels go over a long row in steps of 2048 columns, which a whole number of 32 bits has to hold
    a = norm(cols)
    assert size(name, a) == _lib.PDR_ERR_INVALID_ARG
    assert getattr(_lib.lib(), name)(ctypes.byref(a), FAKE, 1 << 50, None) == _lib.PDR_ERR_INVALID_ARG


def test_the_longest_row_is_taken():
    assert size("pdr_layer_norm_forward", norm(MOST_COLS)) == 0
    assert size("pdr_layer_norm_backward", norm(MOST_COLS)) > 0
