"""The int8 products' plan and order of tiles, from csrc/int8_plan.h compiled by the host's C++ compiler."""
import ctypes as C
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "mxfp8_precision_numerics_amd", "csrc")
FEW, WIDE, MIDDLE, LARGE = range(4)
SHIM = """
#include "int8_plan.h"
extern "C" {
int plan(int64_t M, int64_t cols, int64_t K, int64_t G, int swiglu, int64_t* blocks, int* rows) {
    const mxq::Int8Plan p = mxq::int8_plan(M, cols, K, G, swiglu != 0);
    *blocks = p.blocks;
    *rows = p.rows;
    return p.kind;
}
int form(int64_t M, int64_t cols, int64_t K, int64_t G, int swiglu) {       // wide: few blocks of B; middle: the longer ring
    const mxq::Int8Plan p = mxq::int8_plan(M, cols, K, G, swiglu != 0);
    return p.kind == mxq::INT8_WIDE ? p.wide <= 4 : p.kind == mxq::INT8_MIDDLE ? p.deep : 0;
}
int groups(int64_t most) { return mxq::large_groups(most); }
int tiles(int64_t row_tiles, int tiles_n, int most) { return mxq::large_tiles(row_tiles, tiles_n, most); }
int tile(int b, int T) { return mxq::large_tile(b, T); }
}
"""


def load(folder):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SHIM)
    r = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", CSRC, src, "-o", lib],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lib = C.CDLL(lib)
    lib.plan.argtypes = [C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_int, C.POINTER(C.c_int64), C.POINTER(C.c_int)]
    lib.form.argtypes = [C.c_int64, C.c_int64, C.c_int64, C.c_int64, C.c_int]
    lib.groups.argtypes = [C.c_int64]
    lib.tiles.argtypes = [C.c_int64, C.c_int, C.c_int]
    return lib


def plan(lib, M, cols, K, G=0, swiglu=False):
    """(kernel, workgroups or tiles, rows of A in a tile) of one call with `cols` output columns."""
    blocks, rows = C.c_int64(), C.c_int()
    kind = lib.plan(M, cols, K, G, 1 if swiglu else 0, C.byref(blocks), C.byref(rows))
    return kind, blocks.value, rows.value


def variant(lib, M, cols, K, G=0, swiglu=False, aligned=True):
    """The kernel's form that takes a call: all that tells the compiled ones apart. aligned: 16-byte rows of the output."""
    kind, _, rows = plan(lib, M, cols, K, G, swiglu)
    form = bool(lib.form(M, cols, K, G, 1 if swiglu else 0))
    if kind == LARGE:
        return "large", G > 0, swiglu, aligned and cols % 8 == 0
    if kind == MIDDLE:
        return "middle", form, G > 0, swiglu
    if kind == WIDE:
        return "wide", rows, form, swiglu
    return "few", rows, G > 0, swiglu
