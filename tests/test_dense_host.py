"""Host-side checks of the dense operators' C ABI (no GPU): names, struct
layouts, workspace sizes, and refusals before anything is enqueued."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

from differentiable_gaussian_splatting_pdr_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "pdr_dense.h")
FAKE = 0x10000  # 256-byte aligned, never dereferenced on these paths


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_names():
    declared = sorted(set(re.findall(r"\b(pdr_\w+)\s*\(", header())))
    assert declared == sorted(_lib.EXPORTED_DENSE)
    for f in declared:
        assert hasattr(_lib.lib(), f)


def test_struct_layouts_match_the_header(tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "pdr_dense.h"', "int main(void) {"]
    for name in ("pdr_linear", "pdr_gated_mlp", "pdr_orthogonalize_args"):
        lines.append('printf("%s %%zu\\n", sizeof(%s));' % (name, name))
        for f, _ in getattr(_lib, name)._fields_:
            lines.append('printf("%s.%s %%zu\\n", offsetof(%s, %s));' % (name, f, name, f))
    lines.append("return 0; }")
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    said = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True,
                                                        check=True).stdout.splitlines())
    for name in ("pdr_linear", "pdr_gated_mlp", "pdr_orthogonalize_args"):
        cls = getattr(_lib, name)
        assert int(said[name]) == ctypes.sizeof(cls)
        for f, _ in cls._fields_:
            assert int(said[name + "." + f]) == getattr(cls, f).offset, f


def linear(**kw):
    a = _lib.pdr_linear()
    for k, v in dict(fmt=2, out_fmt=2, activation=0, M=64, N=32, K=128, x=FAKE, ldx=128, w=FAKE, ldw=128,
                     y=FAKE, ldy=32, dy=FAKE, lddy=32).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def gated(**kw):
    a = _lib.pdr_gated_mlp()
    for k, v in dict(fmt=2, activation=2, M=64, D=32, F=96, O=32, x=FAKE, ldx=32, w_in=FAKE, ld_in=32,
                     w_out=FAKE, ld_out=96, y=FAKE, ldy=32, h=FAKE, gu=FAKE, dy=FAKE, lddy=32, dx=FAKE,
                     lddx=32).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def ortho(**kw):
    a = _lib.pdr_orthogonalize_args()
    for k, v in dict(fmt=0, batch=2, m=10, n=20, g=FAKE, ldg=20, batch_g=200, x=FAKE, ldx=20, batch_x=200,
                     steps=5, a=3.4, b=-4.7, c=2.0, eps=1e-7).items():
        setattr(a, k, v)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def refused(name, a, code=-1):
    L = _lib.lib()
    size = getattr(L, name + "_workspace_bytes")(ctypes.byref(a))
    if code == -1:
        assert size == -1
    assert getattr(L, name)(ctypes.byref(a), None, 0, None) == code


BIG = 1 << 23
LINEAR_BAD = [dict(fmt=3), dict(fmt=-1), dict(out_fmt=1), dict(fmt=0, out_fmt=2, x=FAKE), dict(activation=4),
              dict(activation=-1), dict(M=-1), dict(N=1 << 31), dict(K=-5), dict(x=None), dict(w=None),
              dict(x=FAKE + 1), dict(ldx=127), dict(ldw=BIG), dict(slope=FAKE + 8)]


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(y=None), dict(ldy=31), dict(y=FAKE + 1), dict(res=FAKE, ldr=3),
                                             dict(res=FAKE + 1, ldr=32), dict(bias=FAKE + 1)])
def test_linear_forward_refuses(kw):
    refused("pdr_linear_forward", linear(**kw))


@pytest.mark.parametrize("kw", LINEAR_BAD + [dict(dy=None), dict(lddy=31), dict(dx=FAKE, lddx=100),
                                             dict(dw=FAKE, lddw=5), dict(dw=FAKE + 1, lddw=128),
                                             dict(dbias=FAKE + 1), dict(activation=2)])
def test_linear_backward_refuses(kw):
    refused("pdr_linear_backward", linear(**kw))


GATED_BAD = [dict(fmt=5), dict(activation=9), dict(M=-1), dict(D=-1), dict(F=-1), dict(O=-1), dict(x=None),
             dict(w_in=None), dict(w_out=None), dict(ldx=31), dict(ld_in=31), dict(ld_out=95), dict(h=None),
             dict(h=FAKE + 8), dict(gu=FAKE + 4), dict(F=1 << 22)]


@pytest.mark.parametrize("kw", GATED_BAD + [dict(y=None), dict(ldy=31), dict(res=FAKE, ldr=31)])
def test_gated_forward_refuses(kw):
    refused("pdr_gated_mlp_forward", gated(**kw))


@pytest.mark.parametrize("kw", GATED_BAD + [dict(dy=None), dict(lddy=3), dict(lddx=31), dict(gu=None),
                                            dict(dw_in=FAKE, ldd_in=3), dict(dw_out=FAKE, ldd_out=95)])
def test_gated_backward_refuses(kw):
    refused("pdr_gated_mlp_backward", gated(**kw))


@pytest.mark.parametrize("kw", [dict(fmt=7), dict(batch=-1), dict(batch=65536), dict(m=-1), dict(n=-1), dict(g=None),
                                dict(x=None), dict(ldg=19), dict(ldx=19), dict(steps=-1), dict(a=float("inf")),
                                dict(b=float("nan")), dict(eps=-1.0), dict(eps=float("nan")), dict(m=BIG),
                                dict(g=FAKE + 2)])
def test_orthogonalize_refuses(kw):
    refused("pdr_orthogonalize", ortho(**kw))


def test_null_structs_and_workspaces():
    L = _lib.lib()
    for name in ("pdr_linear_forward", "pdr_linear_backward", "pdr_gated_mlp_forward", "pdr_gated_mlp_backward",
                 "pdr_orthogonalize"):
        assert getattr(L, name + "_workspace_bytes")(None) == -1
        assert getattr(L, name)(None, FAKE, 1 << 30, None) == -1
    a = ortho()
    need = L.pdr_orthogonalize_workspace_bytes(ctypes.byref(a))
    assert need > 0
    for ws, size in ((None, need), (FAKE, need - 1), (FAKE + 16, need)):
        assert L.pdr_orthogonalize(ctypes.byref(a), ws, size, None) == _lib.PDR_ERR_WORKSPACE


def test_workspace_bytes():
    L = _lib.lib()
    # in place: rows on 16 bytes, a multiple of 8 long, results enough to fill the card
    a = linear(M=8192, N=2048, K=128, ldy=2048)
    assert L.pdr_linear_forward_workspace_bytes(ctypes.byref(a)) == 0
    # a row that is not a multiple of 8 long: both operands are copied to padded rows
    b = linear(M=8192, N=2048, K=125, ldy=2048)
    assert L.pdr_linear_forward_workspace_bytes(ctypes.byref(b)) == (8192 + 2048) * 128 * 2
    assert _lib.pdr_dense_kept_ld(0) == 0 and _lib.pdr_dense_kept_ld(1) == 8 and _lib.pdr_dense_kept_ld(16) == 16
    with pytest.raises(_lib.PdrError):
        _lib.pdr_dense_kept_ld(-1)


@pytest.mark.parametrize("which", ["M", "N", "K", "D", "F", "O", "m", "n", "batch"])
def test_empty_lengths_need_no_pointers(which):
    """Lengths of 0 are sized like any other (no matrix is looked at)."""
    L = _lib.lib()
    for fmt in (0, 1, 2):
        if which in "MNK":
            for act in (0, 3):
                a = linear(fmt=fmt, out_fmt=fmt, activation=act, slope=FAKE, dx=FAKE, lddx=128, dw=FAKE, lddw=128,
                           dbias=FAKE, **{which: 0})
                assert L.pdr_linear_forward_workspace_bytes(ctypes.byref(a)) >= 0
                assert L.pdr_linear_backward_workspace_bytes(ctypes.byref(a)) >= 0
        if which in "MDFO":
            a = gated(fmt=fmt, dw_in=FAKE, ldd_in=32, dw_out=FAKE, ldd_out=96, **{which: 0})
            assert L.pdr_gated_mlp_forward_workspace_bytes(ctypes.byref(a)) >= 0
            assert L.pdr_gated_mlp_backward_workspace_bytes(ctypes.byref(a)) >= 0
        if which in ("m", "n", "batch"):
            a = ortho(fmt=fmt, **{which: 0})
            assert L.pdr_orthogonalize_workspace_bytes(ctypes.byref(a)) >= 0


def test_cpu_tensors_are_refused():
    code = r'''
import torch
from differentiable_gaussian_splatting_pdr_amd import dense
x = torch.zeros(4, 8)
for f in (lambda: dense.linear(x, x), lambda: dense.gated_mlp(x, x, x), lambda: dense.orthogonalize(x)):
    try:
        f()
    except ValueError as e:
        assert "ROCm device" in str(e)
    else:
        raise SystemExit("ran on the CPU")
try:
    dense.Muon([torch.zeros(3, requires_grad=True)])
except ValueError:
    print("refused")
'''
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "refused" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("name,M,F", [("forward", 1 << 21, 1 << 13), ("forward", 3 << 19, 10921), ("backward", 1 << 20, 1 << 13),
                                      ("backward", 3 << 19, 5461)])
def test_gated_kept_values_beyond_the_passes_index_are_refused(name, M, F):
    """fp32 layouts of h and [dg | du] count 8 values in 31 bits; 16-bit ones are read in place."""
    L = _lib.lib()
    size = getattr(L, "pdr_gated_mlp_%s_workspace_bytes" % name)
    sizes = dict(M=M, F=F, D=8, ldx=8, ld_in=8, lddx=8, O=8, ldy=8, lddy=8, ld_out=F)
    assert size(ctypes.byref(gated(fmt=0, **sizes))) == -1
    assert size(ctypes.byref(gated(fmt=2, **sizes))) >= 0
    assert size(ctypes.byref(gated(fmt=0, **{**sizes, "M": M // 2}))) >= 0


# What the iterates reach from singular values in [0, 1], and whether fp16 holds it under the fixed scales.
COEFFICIENTS = [((3.4445, -4.7750, 2.0315), 5, True), ((3.4445, -4.7750, 2.0315), 100, True), ((2.0, -1.5, 0.5), 12, True),
                ((15 / 8, -10 / 8, 3 / 8), 30, True), ((1.5, -0.5, 0.0), 30, True), ((1.0, 0.0, 0.0), 9, True),
                ((0.0, 30.0, 25.0), 1, True), ((0.0, 40.0, 40.0), 1, False), ((0.0, -80.0, 80.0), 1, True),
                ((0.0, -300.0, 300.0), 1, False), ((100.0, 0.0, 0.0), 1, True), ((100.0, 0.0, 0.0), 2, False),
                ((1.1, 0.0, 0.0), 21, True), ((1.1, 0.0, 0.0), 40, False), ((2.0, 1.0, 1.0), 2, False), ((1e30, 0.0, 0.0), 1, True),
                ((1e30, 1e30, 1e30), 0, True), ((7.0, 0.0, 0.0), 2, True), ((0.0, 0.0, 3e38), 1, False)]


@pytest.mark.parametrize("c,steps,held", COEFFICIENTS)
def test_coefficients_that_leave_the_iterates_range_are_refused(c, steps, held):
    a = ortho(steps=steps, a=c[0], b=c[1], c=c[2])
    size = _lib.lib().pdr_orthogonalize_workspace_bytes(ctypes.byref(a))
    assert size > 0 if held else size == -1


FMT = {"torch.float32": 0, "torch.float16": 1, "torch.bfloat16": 2}
ACT = {"none": 0, "silu": 2, "gelu": 3}
TILES = [(64, 1), (64, 4), (128, 1), (128, 2), (256, 1)]


def test_struct_layout_of_a_product_matches_the_header(tmp_path):
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "pdr_dense.h"\nint main(void) {\n'
                   'printf("%zu", sizeof(pdr_dense_product));\n'
                   + "\n".join('printf(" %%zu", offsetof(pdr_dense_product, %s));' % f
                               for f, _ in _lib.pdr_dense_product._fields_) + "\nreturn 0; }\n")
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)],
                   check=True)
    said = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(v) for v in said] == [ctypes.sizeof(_lib.pdr_dense_product)] + [
        getattr(_lib.pdr_dense_product, f).offset for f, _ in _lib.pdr_dense_product._fields_]


def test_sizes_take_every_product_kernel():
    """The sizes of test_gpu_dense_tiles reach each kernel that a product may run in."""
    import dense_sizes as sizes
    kernels, epilogues, cut = set(), set(), set()

    def note(p, columns):
        whole = columns is None or columns % 8 == 0   # rows that begin on 16 bytes
        kernels.add((p.fmt, p.a_mc, p.b_mc, p.epilogue, p.tile, p.groups, whole))
        cut.add((p.a_mc, p.b_mc, p.epilogue, p.parts > 1, whole))

    for dtype, out, M, K, N, act, residual in sizes.LINEAR:
        c = dict(fmt=FMT[str(dtype)], out_fmt=FMT[str(out)], activation=ACT[act], M=M, N=N, K=K, ldx=K, ldw=K, bias=FAKE,
                 ldy=N, slope=FAKE, lddy=N, dx=FAKE, lddx=K, dw=FAKE, lddw=K, dbias=FAKE)
        forward, = _lib.dense_products(linear(res=FAKE if residual else None, ldr=N, **c))
        dx, dw = _lib.dense_products(linear(**c), True)
        for p, n in ((forward, N), (dx, K), (dw, K)):
            note(p, n)
        epilogues.add((forward.tile, forward.groups, act != "none", residual, str(out) == "torch.float32", N % 8 == 0))
    for dtype, M, D, F, O in sizes.GATED:
        c = dict(fmt=FMT[str(dtype)], M=M, D=D, F=F, O=O, ldx=D, ld_in=D, ld_out=F, ldy=O, lddy=O, lddx=D, dw_in=FAKE,
                 ldd_in=D, dw_out=FAKE, ldd_out=F)
        both, down = _lib.dense_products(gated(res=FAKE, ldr=O, **c))
        dwo, dgu, dx, dwi = _lib.dense_products(gated(**c), True)
        for p, n in ((both, None), (down, O), (dwo, F), (dgu, None), (dx, D), (dwi, D)):
            note(p, n)
    for fmt in (1, 2):
        for a_mc, b_mc, epilogue in ((0, 0, 0), (0, 1, 0), (1, 1, 0), (0, 0, 1), (0, 1, 2)):
            for tile, groups in TILES:
                for whole in (True, False) if epilogue == 0 else (True,):
                    assert (fmt, a_mc, b_mc, epilogue, tile, groups, whole) in kernels
    for tile, groups in TILES:
        for key in [(act, res, wide, whole) for act in (0, 1) for res in (0, 1) for wide in (0, 1) for whole in (0, 1)]:
            assert (tile, groups, *map(bool, key)) in epilogues
    for a_mc, b_mc, epilogue, whole in ((0, 0, 0, 0), (0, 0, 0, 1), (0, 1, 0, 0), (0, 1, 0, 1), (1, 1, 0, 0), (1, 1, 0, 1),
                                        (0, 1, 2, 1)):
        for parts in (True, False):
            assert (a_mc, b_mc, epilogue, parts, bool(whole)) in cut

    steps, last = set(), set()
    for dtype, batch, m, n in sizes.ORTHOGONALIZE:
        fmt = FMT[str(dtype)]
        made = _lib.dense_products(ortho(fmt=fmt, batch=batch, m=m, n=n, ldg=n, batch_g=m * n, ldx=n, batch_x=m * n, steps=2))
        assert len(made) == 6
        steps.update((p.a_mc, p.b_mc, p.tile, p.groups, p.lower) for p in made)
        last.add((made[5].b_mc, made[5].tile, fmt, n % 8 == 0))
    for tile, groups in TILES:
        for a_mc, b_mc, lower in ((0, 0, 0), (0, 0, 1), (0, 1, 0), (1, 1, 0), (1, 1, 1)):
            assert (a_mc, b_mc, tile, groups, lower) in steps
    assert {(b, f, w) for b, _, f, w in last} == {(b, f, w) for b in (0, 1) for f in (0, 1, 2) for w in (True, False)}


@pytest.mark.parametrize("M,N,K", [(2 ** 31 - 257, 1, 8), (2 ** 30 + 100001, 1, 8), (2 ** 31 - 257, 8, 8), (2 ** 31 - 257, 7, 8),
                                   (8, 8, 2 ** 31 - 257), (1 << 22, 4088, 8), (4096, 1 << 21, 8)])
def test_launches_hold_their_threads(M, N, K):
    """A launch has fewer than 2^32 threads along its first axis."""
    # dw of (N x K outputs) sums over M rows: the third length is the sum's in one direction or the other
    for act, fmt in ((0, 2), (3, 2), (0, 0)):
        if K < 1 << 22:
            made = _lib.dense_products(linear(fmt=fmt, out_fmt=fmt, activation=act, M=M, N=N, K=K, ldx=K, ldw=K, ldy=N))
        else:
            made = _lib.dense_products(linear(fmt=fmt, out_fmt=fmt, M=K, N=N, K=M, ldx=M, ldw=M, lddy=N, dw=FAKE, lddw=M), True)
        for p in made:
            tiles = ((p.M + p.tile - 1) // p.tile) * ((p.N + p.tile - 1) // p.tile)
            assert tiles * 256 * p.groups < 2 ** 32 and p.parts < 65536
            assert p.parts == 1 or p.M * p.N < 2 ** 31
