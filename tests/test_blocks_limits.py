"""Sizes that attention, layer norm and dropout take and refuse, and what follows from
sizes alone, without a GPU."""
import ctypes
import os
import subprocess

import pytest
import torch

import test_gpu_attention_wide
from differentiable_gaussian_splatting_pdr_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
RULE = os.path.join(ROOT, "differentiable_gaussian_splatting_pdr_amd", "csrc", "attention_plan.hpp")
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


def test_sizes_take_the_kernels_of_128_rows(tmp_path):
    """Every call of test_gpu_attention_wide takes the larger workgroups; one sequence of it, the smaller."""
    formats = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
    calls = list(test_gpu_attention_wide.calls())
    lines = []
    for dtype, causal, batch, queries, keys, heads, kv_heads, dim, packed in calls:
        per = 4 if dtype == torch.float32 else 8
        lines.append("{%d, %d, %d, %d, %d, %d, %d, %d, %d}," % (formats[dtype], causal, batch, heads, kv_heads, (dim + per - 1) // per * per,
                                                              queries, keys, packed))
    src, exe = tmp_path / "rows.cpp", tmp_path / "rows"
    src.write_text('''
#include <stdio.h>
#include "attention_plan.hpp"
static const long long calls[][9] = {
%s
};
int main() {
  for (const auto &c : calls) {
    pdr_attention p = {};
    p.fmt = (int)c[0], p.causal = (int)c[1], p.batch = c[2], p.heads = c[3], p.kv_heads = c[4], p.dim = c[5];
    p.q_rows = c[6], p.k_rows = c[7];
    static const int offsets = 0;
    if (c[8]) p.q_offsets = p.k_offsets = &offsets;
    const int few = pdr::attend::takes_few(p);
    p.q_rows = p.q_offsets ? p.q_rows / p.batch : p.q_rows;
    p.batch = 1, p.heads /= p.kv_heads, p.kv_heads = 1;
    printf("%%d %%d\\n", few, pdr::attend::takes_few(p));
  }
}
''' % "\n".join(lines))
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", os.path.dirname(RULE), str(src),
                    "-o", str(exe)], check=True)
    said = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")[:-1]
    assert len(said) == len(calls)
    for call, line in zip(calls, said):
        assert line == "0 1", call
