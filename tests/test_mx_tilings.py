"""Which tiling an MXFP4 product runs on: the sizes of tests/mx_tilings.py reach the kernels that they are listed under,
and between them every kernel. The rule is host code, built here with g++."""

import ctypes
import os
import shutil
import subprocess

import pytest

from tests import mx_tilings as mt

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp8_fine_grained_fp8bq_amd", "csrc")
SOURCE = """
#include "mxfp4_tiling.h"
extern "C" void pick(int mode, int groups, long m, long n, long chunks, int* tiling, int* deep) {
  const fp8bq::MxPick p = fp8bq::mx_pick((fp8bq::MxMode)mode, groups, m, n, chunks);
  *tiling = p.tiling;
  *deep = p.deep;
}
extern "C" void tile(int i, int* bm, int* bn) {
  *bm = fp8bq::kTilings[i].bm;
  *bn = fp8bq::kTilings[i].bn;
}
"""


@pytest.fixture(scope="module")
def rule(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("tiling")
    (d / "rule.cpp").write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I" + CSRC, str(d / "rule.cpp"), "-o", str(d / "rule.so")],
                   check=True)
    lib = ctypes.CDLL(str(d / "rule.so"))
    lib.pick.argtypes = [ctypes.c_int, ctypes.c_int] + [ctypes.c_long] * 3 + [ctypes.POINTER(ctypes.c_int)] * 2

    def name(mode, groups, m, n, k):
        i, deep = ctypes.c_int(), ctypes.c_int()
        lib.pick(mode, groups, m, n, -(-k // 256), ctypes.byref(i), ctypes.byref(deep))
        found = [t for t, v in mt.TILINGS.items() if v[0] == i.value]
        return found[0] if len(found) == 1 or deep.value else found[1]

    name.lib = lib
    return name


def test_tile_sizes(rule):
    for t, (i, bm, bn, _) in mt.TILINGS.items():
        a, b = ctypes.c_int(), ctypes.c_int()
        rule.lib.tile(i, ctypes.byref(a), ctypes.byref(b))
        assert (a.value, b.value) == (bm, bn), t


@pytest.mark.parametrize("tiling,several,m,n,k", mt.DENSE)
def test_dense(rule, tiling, several, m, n, k):
    assert rule(0, 1, m, n, k) == tiling
    if tiling != "stream":
        assert (mt.tiles(tiling, [m], n) > mt.workgroups(0, tiling)) == several


@pytest.mark.parametrize("tiling,several,m,n,k,counts", mt.ROWS)
def test_rows(rule, tiling, several, m, n, k, counts):
    assert sum(counts) < m and rule(1, len(counts), m, n, k) == tiling
    if tiling != "stream":
        assert (mt.tiles(tiling, counts, n) > mt.workgroups(1, tiling)) == several


@pytest.mark.parametrize("tiling,several,m,n,counts", mt.WGRAD)
def test_weight_gradients(rule, tiling, several, m, n, counts):
    assert rule(2, len(counts), m, n, mt.padded(counts, 256)[-1] + 256) == tiling
    if tiling != "stream":
        assert (mt.tiles(tiling, [m], n, len(counts)) > mt.workgroups(2, tiling)) == several


@pytest.mark.parametrize("tiling,m,n", mt.WGRAD_FEW)
def test_weight_gradients_of_few_experts(rule, tiling, m, n):
    assert rule(2, 4, m, n, 1024) == tiling


@pytest.mark.parametrize("table", ["DENSE", "ROWS", "WGRAD"])
def test_every_kernel_is_reached(table):
    rows = getattr(mt, table)
    assert {r[0] for r in rows} == set(mt.TILINGS)
    # more tiles than workgroups wherever the rule allows it (dense and gradients of 128 x 128 with loading waves are
    # chosen for one tile per workgroup or fewer)
    once = {"stream"} | ({"128x128 deep"} if table != "ROWS" else set())
    assert {r[0] for r in rows if r[1]} == set(mt.TILINGS) - once
