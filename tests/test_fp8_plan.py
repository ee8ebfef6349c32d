"""The shapes of the e4m3 products' GPU tests take every kernel, tile and K split (CPU: the plan is
host arithmetic, compiled here on its own), and every plan stays within the launch limits."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.conftest import ROOT
from tests.fp8_shapes import DENSE, DENSE_BACKWARD, GROUPED, GROUPED_BACKWARD

SOURCE = r"""
#include <initializer_list>
#include "fp8_plan.h"
extern "C" void plan(int mode, int64_t t, int64_t k, int64_t n, int e, int grouped, int* out) {
  const q4::Plan p = q4::fp8_plan(q4::Fp8Mode(mode), t, k, n, e, grouped);
  out[0] = p.tile, out[1] = p.ksplit, out[2] = q4::fp8_fits(q4::Fp8Mode(mode), t, k, n, e, grouped);
}
"""
Y, DX, DW = 0, 1, 2


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
    lib.plan.argtypes = [ctypes.c_int] + [ctypes.c_int64] * 3 + [ctypes.c_int] * 2 + [ctypes.c_void_p]

    def query(mode, t, k, n, e=1, grouped=False):
        """-> (tile, K slices, whether it fits); tile 0 is the few-rows kernel."""
        r = (ctypes.c_int * 3)()
        lib.plan(mode, t, k, n, e, int(grouped), r)
        return r[0], r[1], bool(r[2])

    return query


def seen(plans):
    return {(tile, split > 1) for tile, split, _ in plans}


def sampled(rng):
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    return log(1, 8192), log(1, 1024) * 16, log(1, 1024) * 16


@pytest.mark.parametrize("mode", [Y, DX, DW])
def test_dense_shapes_take_every_plan(plan, mode):
    shapes = DENSE if mode == Y else DENSE_BACKWARD
    got = seen(plan(mode, t, k, n) for t, k, n in shapes)
    rng = random.Random(1)
    assert got >= seen(plan(mode, *sampled(rng)) for _ in range(4000))


@pytest.mark.parametrize("mode", [Y, DX, DW])
def test_grouped_shapes_take_every_plan(plan, mode):
    shapes = GROUPED if mode == Y else GROUPED_BACKWARD
    got = seen(plan(mode, sum(c), k, n, len(c), True) for c, k, n in shapes)
    rng = random.Random(2)
    want = set()
    for _ in range(4000):
        t, k, n = sampled(rng)
        want |= seen([plan(mode, t, k, n, rng.randint(1, 64), True)])
    assert got >= want


def test_plans_fit(plan):
    rng = random.Random(3)
    for _ in range(4000):
        t, k, n = sampled(rng)
        for mode in (Y, DX, DW):
            for e, grouped in ((1, False), (rng.randint(1, 4096), True)):
                if mode == DW and e * n * k > 1 << 36:
                    continue
                tile, split, fits = plan(mode, t, k, n, e, grouped)
                assert fits and tile in (0, 64, 128, 256) and (tile or mode == Y)
                assert split == 1 or not grouped
