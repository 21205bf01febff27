"""Host-side checks of the blocks' C ABI (no GPU): names, struct layouts,
workspace sizes, and refusals before anything is enqueued."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from differentiable_gaussian_splatting_pdr_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pdr_blocks.h")
FAKE = 0x10000  # 256-byte aligned, never dereferenced on these paths
STRUCTS = ("pdr_attention", "pdr_layer_norm", "pdr_dropout_args")


def test_names():
    declared = sorted(set(re.findall(r"\b(pdr_\w+)\s*\(", re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S))))
    assert declared == sorted(_lib.EXPORTED_BLOCKS)
    for f in declared:
        assert hasattr(_lib.lib(), f)


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pdr_blocks.h"', "int main(void) {"]
    for name in STRUCTS:
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for f, _ in getattr(_lib, name)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f))
    lines.append("return 0; }")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    said = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name in STRUCTS:
        cls = getattr(_lib, name)
        assert int(said[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(said[name + "." + f]) == getattr(cls, f).offset, f


def made(cls, fields, more):
    a = cls()
    for k, v in {**fields, **more}.items():
        setattr(a, k, v)
    return a


def attention(**kw):
    c = dict(fmt=2, causal=1, batch=2, heads=8, kv_heads=2, dim=64, q_rows=100, k_rows=120, scale=0.125, lse=FAKE)
    for t, h, n in (("q", 8, 100), ("k", 2, 120), ("v", 2, 120), ("o", 8, 100), ("dy", 8, 100), ("dq", 8, 100), ("dk", 2, 120),
                    ("dv", 2, 120)):
        c.update({t: FAKE, t + "_row": h * 64, t + "_head": 64, t + "_batch": n * h * 64})
    return made(_lib.pdr_attention, c, kw)


def norm(**kw):
    return made(_lib.pdr_layer_norm, dict(fmt=2, rows=20, cols=64, eps=1e-5, x=FAKE, ldx=64, weight=FAKE, bias=FAKE, y=FAKE, ldy=64,
                                          stats=FAKE, dy=FAKE, lddy=64, dx=FAKE, lddx=64, dweight=FAKE, dbias=FAKE), kw)


def dropout(**kw):
    return made(_lib.pdr_dropout_args, dict(fmt=0, rows=20, cols=64, p=0.5, seed=1, x=FAKE, ldx=64, res=FAKE, ldr=64, y=FAKE, ldy=64), kw)


def size(name, a):
    return getattr(_lib.lib(), name + "_workspace_bytes")(ctypes.byref(a))


def refused(name, a):
    assert size(name, a) == -1
    assert getattr(_lib.lib(), name)(ctypes.byref(a), FAKE, 1 << 40, None) == -1


ATTENTION_BAD = [dict(fmt=3), dict(fmt=-1), dict(batch=-1), dict(q_rows=-1), dict(k_rows=1 << 31), dict(heads=0), dict(kv_heads=0),
                 dict(heads=7), dict(heads=-8), dict(dim=0), dict(dim=60), dict(dim=136), dict(scale=0.0), dict(scale=-1.0),
                 dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=FAKE + 8),
                 dict(k_row=127), dict(v_head=4), dict(q_batch=-64), dict(o_row=-512), dict(k_row=(1 << 22) + 8), dict(q_head=(1 << 24) + 8),
                 dict(q_head=1 << 26), dict(q_offsets=FAKE), dict(k_offsets=FAKE), dict(key_lengths=FAKE + 2),
                 dict(q_offsets=FAKE, k_offsets=FAKE, key_lengths=FAKE), dict(q_offsets=FAKE, k_offsets=FAKE + 1), dict(lse=FAKE + 2),
                 dict(batch=1 << 20), dict(q_rows=1 << 26), dict(batch=1 << 22, q_rows=1), dict(fmt=0, dim=66)]


@pytest.mark.parametrize("kw", ATTENTION_BAD)
def test_attention_forward_refuses(kw):
    refused("pdr_attention_forward", attention(**kw))


@pytest.mark.parametrize("kw", ATTENTION_BAD + [dict(dy=None), dict(dy=FAKE + 4), dict(dy_row=3), dict(lse=None), dict(dk=None), dict(dv=None),
                                                dict(dq=FAKE + 2), dict(dk_row=4), dict(dv_head=-64), dict(k_rows=1 << 28)])
def test_attention_backward_refuses(kw):
    refused("pdr_attention_backward", attention(**kw))


NORM_BAD = [dict(fmt=4), dict(rows=-1), dict(cols=-1), dict(cols=1 << 31), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
            dict(x=None), dict(x=FAKE + 1), dict(ldx=63), dict(weight=FAKE + 1), dict(stats=FAKE + 4)]


@pytest.mark.parametrize("kw", NORM_BAD + [dict(y=None), dict(ldy=3), dict(bias=FAKE + 1)])
def test_norm_forward_refuses(kw):
    refused("pdr_layer_norm_forward", norm(**kw))


@pytest.mark.parametrize("kw", NORM_BAD + [dict(dy=None), dict(lddy=63), dict(stats=None), dict(dx=FAKE + 1), dict(lddx=5),
                                           dict(dweight=FAKE + 1), dict(dbias=FAKE + 1)])
def test_norm_backward_refuses(kw):
    refused("pdr_layer_norm_backward", norm(**kw))


@pytest.mark.parametrize("kw", [dict(fmt=3), dict(rows=-1), dict(cols=-1), dict(rows=1 << 30, cols=1 << 10), dict(p=-0.1), dict(p=1.5),
                                dict(p=float("nan")), dict(seed_at=FAKE + 4), dict(x=None), dict(x=FAKE + 2), dict(ldx=63), dict(y=None),
                                dict(ldy=1), dict(res=FAKE + 2), dict(ldr=63)])
def test_dropout_refuses(kw):
    refused("pdr_dropout", dropout(**kw))


def test_null_structs_and_workspaces():
    L = _lib.lib()
    calls = [n for n in _lib.EXPORTED_BLOCKS if not n.endswith("_workspace_bytes")]
    for name in calls:
        assert getattr(L, name + "_workspace_bytes")(None) == -1
        assert getattr(L, name)(None, FAKE, 1 << 30, None) == -1
    few = attention(q_rows=1, k_rows=5000)
    for name, a in (("pdr_attention_forward", few), ("pdr_attention_backward", attention()), ("pdr_layer_norm_backward", norm())):
        need = size(name, a)
        assert need > 0
        for ws, n in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
            assert getattr(L, name)(ctypes.byref(a), ws, n, None) == _lib.PDR_ERR_WORKSPACE


def test_workspace_bytes():
    # many queries keep nothing; two values a row in the backward, and parts' sums for dk and dv
    assert size("pdr_attention_forward", attention()) == 0
    assert size("pdr_attention_backward", attention(dk=None, dv=None)) == 2 * (2 * 100 * 8 * 4)
    assert size("pdr_attention_backward", attention()) >= 2 * (2 * 100 * 8 * 4)
    # few keys for many queries: sums of parts
    assert size("pdr_attention_backward", attention(q_rows=4096)) > 2 * (2 * 4096 * 8 * 4)
    assert size("pdr_attention_backward", attention(q_rows=4096, dk=None, dv=None)) == 2 * (2 * 4096 * 8 * 4)
    assert size("pdr_layer_norm_forward", norm()) == 0
    assert size("pdr_layer_norm_backward", norm(dweight=None, dbias=None)) == 0
    assert size("pdr_dropout", dropout()) == 0


@pytest.mark.parametrize("which", ["batch", "q_rows", "k_rows"])
@pytest.mark.parametrize("packed", [False, True])
def test_empty_attention_needs_no_pointers(which, packed):
    more = dict(q_offsets=FAKE, k_offsets=FAKE) if packed else {}
    gone = {"batch": ("q", "k", "v", "o", "dy", "dq"), "q_rows": ("q", "o", "dy", "dq", "lse"), "k_rows": ("k", "v")}[which]
    if packed and which == "batch":
        gone = ()   # tokens that no sequence has
    for q_rows in (1, 100):
        a = attention(**{"q_rows": q_rows, which: 0, **more}, **{g: None for g in gone})
        assert size("pdr_attention_forward", a) >= 0 and size("pdr_attention_backward", a) >= 0


def test_empty_rows_need_no_pointers():
    for kw in (dict(rows=0), dict(cols=0)):
        a = norm(**kw, x=None, y=None, dy=None, dx=None, stats=None)
        assert size("pdr_layer_norm_forward", a) == 0 and size("pdr_layer_norm_backward", a) == 0
        assert size("pdr_dropout", dropout(**kw, x=None, y=None)) == 0


def test_cpu_tensors_are_refused():
    code = r'''
import torch
from differentiable_gaussian_splatting_pdr_amd import blocks
x = torch.zeros(2, 4, 2, 8)
for f in (lambda: blocks.attention(x, x, x), lambda: blocks.layer_norm(x), lambda: blocks.dropout(x, 0.5, 1)):
    try:
        f()
    except ValueError as e:
        assert "ROCm device" in str(e)
    else:
        raise SystemExit("ran on the CPU")
print("refused")
'''
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("scale", [2.0 ** -65, 2.0 ** 65, 1e-30, 1e38])
def test_scales_out_of_range_are_refused(scale):
    # the backward's sums start from lse / scale, which has to stay in fp32's range
    for name in ("pdr_attention_forward", "pdr_attention_backward"):
        refused(name, attention(scale=scale))
        assert size(name, attention(scale=2.0 ** 64)) >= 0 and size(name, attention(scale=2.0 ** -64)) >= 0
