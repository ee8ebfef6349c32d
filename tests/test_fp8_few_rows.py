"""The few-rows kernel's launches and forms (CPU: host arithmetic on the sizes, compiled here)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.conftest import ROOT
from tests.few_rows_shapes import PASSES, SCATTERED, SIXTEEN

SOURCE = r"""
#include "fp8_plan.h"
extern "C" int tile(int64_t t, int64_t k, int64_t n, int e, int grouped) {
  return q4::fp8_plan(q4::FP8_Y, t, k, n, e, grouped).tile;
}
extern "C" int fits(int64_t t, int64_t k, int64_t n, int e, int grouped) {
  return q4::fp8_fits(q4::FP8_Y, t, k, n, e, grouped);
}
extern "C" int search(int64_t t, int64_t n, int64_t e) { return q4::fp8_rows_search(t, n, e); }
extern "C" int64_t grid(int64_t t, int64_t n, int64_t e) { return q4::fp8_rows_grid(t, n, e); }
extern "C" int sixteen(int64_t t, int e, int grouped) { return q4::fp8_rows_sixteen(t, e, grouped); }
"""
MOST = 1 << 23   # workgroups of a launch


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, out = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int4_group_quantized_g128_amd", "csrc"), str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    i64, i32 = ctypes.c_int64, ctypes.c_int
    lib.tile.argtypes = lib.fits.argtypes = [i64, i64, i64, i32, i32]
    lib.search.argtypes = lib.grid.argtypes = [i64, i64, i64]
    lib.sixteen.argtypes = [i64, i32, i32]
    lib.grid.restype = i64
    return lib


def test_experts_without_rows_get_no_workgroups(plan):
    """One token's 8 of 256 experts: as many workgroups as the rows can need, not one per expert and
    16 columns."""
    assert plan.grid(8, 4096, 256) == 8 * 256
    assert plan.grid(2, 4096, 1024) == 2 * 256
    for t, k, n, e in [s[:4] for s in SCATTERED]:
        assert plan.tile(t, k, n, e, 1) == 0 and plan.search(t, n, e), (t, k, n, e)
    # where most have rows, or one has all, nothing is searched for
    assert plan.grid(300, 4096, 300) == 300 * 256 and not plan.search(300, 4096, 300)
    assert plan.grid(1, 16384, 1) == 1024 and not plan.search(1, 16384, 1)


def test_launches_fit(plan):
    rng = random.Random(5)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    seen = set()
    for _ in range(20000):
        t, k, n, e = log(1, 1 << 20), log(1, 1024) * 16, log(1, 1 << 20), log(1, 4096)
        if plan.tile(t, k, n, e, 1) == 0:
            assert plan.fits(t, k, n, e, 1)
            grid = plan.grid(t, n, e)
            assert min(t, e) * -(-n // 16) <= grid < MOST
            seen.add(plan.search(t, n, e))
    assert seen == {0, 1}


def test_shapes_take_both_passes(plan):
    for counts, *t, k, n, rows in PASSES:
        t, e, grouped = (t[0], 1, 0) if counts is None else (sum(counts), len(counts), 1)
        assert plan.tile(t, k, n, e, grouped) == 0, (counts, t, k, n)
        assert plan.sixteen(t, e, grouped) == (rows == 16), (counts, t, k, n)
    for many in (16, 64):   # more rows than a pass, of one matrix or expert
        assert any(max(c[0] or [c[1]]) > c[-1] for c in PASSES if c[-1] == many)


def test_up_to_sixteen_rows_take_passes_of_sixteen(plan):
    for t, k, n, counts in SIXTEEN:
        assert plan.tile(t, k, n, len(counts or [0]), int(counts is not None)) == 0
    rng = random.Random(6)
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(20000):
        t, k, n = rng.randint(1, 16), log(1, 1 << 16) * 16, log(1, 1 << 20)
        for e, grouped in ((1, 0), (log(1, 4096), 1)):
            assert plan.tile(t, k, n, e, grouped) == 0 and plan.sixteen(t, e, grouped)
            assert plan.fits(t, k, n, e, grouped)
