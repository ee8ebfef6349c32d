"""The shapes of the dense products' GPU tests take every kernel, tile and K split that
ordinary sizes can take (CPU: the plan is host arithmetic, compiled here on its own)."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = r"""
#include "dense_plan.h"
#include <initializer_list>
extern "C" {
#define ENTRY(name)                                                              \
  void name(int64_t t, int64_t a, int64_t b, int* out) {                         \
    const q4::Plan p = q4::name##_plan(t, a, b);                                 \
    out[0] = p.tile, out[1] = p.ksplit;                                          \
  }
ENTRY(int8) ENTRY(swiglu) ENTRY(dx) ENTRY(dw)
}
"""


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

    def query(product, t, a, b):
        """-> (tile, whether K is split); tile 0 is the few-rows kernel."""
        f = getattr(lib, product)
        f.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_void_p]
        r = (ctypes.c_int * 2)()
        f(t, a, b, r)
        return r[0], r[1] > 1

    return query


def sampled(rng, product):
    """Sizes of the operator's ordinary range, spread over their logarithm."""
    log = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    t = log(1, 8192)
    if product == "int8":
        return t, log(4, 1024) * 16, log(16, 16384)
    return t, log(8, 1024) * 8, log(8, 1024) * 8


@pytest.mark.parametrize("product", ["int8", "swiglu", "dx", "dw"])
def test_gpu_shapes_take_every_plan(plan, product):
    from tests.test_gpu_dense_paths import INT8_SHAPES, SWIGLU_SHAPES
    rng = random.Random(product)
    reachable = {plan(product, *sampled(rng, product)) for _ in range(20000)}
    assert len(reachable) >= 6
    tested = {plan(product, *s) for s in (INT8_SHAPES if product == "int8" else SWIGLU_SHAPES)}
    assert reachable <= tested, sorted(reachable - tested)


def test_equal_bits_shapes_take_every_plan(plan):
    from tests.test_gpu_dense_paths import EQUAL_BITS
    taken = {plan("int8", t, k, n) for rows, k, n in EQUAL_BITS for t in rows}
    assert taken == {(0, False)} | {(tile, split) for tile in (64, 128, 256) for split in (False, True)}
