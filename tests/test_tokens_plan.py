"""Which workgroups sort tokens by expert (CPU: host arithmetic, compiled here)."""
import ctypes
import os
import shutil
import subprocess

import pytest

from tests.conftest import ROOT

SOURCE = r"""
#include "tokens_plan.h"
extern "C" int by_waves(int64_t t, int k, int64_t bytes) { return q4::dispatch_by_waves(t, k, bytes); }
"""


@pytest.fixture(scope="module")
def by_waves(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if not cxx:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    src, out = d / "plan.cpp", d / "plan.so"
    src.write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-O2", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "int4_group_quantized_g128_amd", "csrc"), str(src), "-o", str(out)], check=True)
    lib = ctypes.CDLL(str(out))
    lib.by_waves.argtypes = [ctypes.c_int64, ctypes.c_int, ctypes.c_int64]
    return lib.by_waves


def test_few_tokens_go_by_workgroups(by_waves):
    """Whatever their width: by waves 16 tokens of 256 take twice as long."""
    for t in (1, 16, 300, 1500):
        for k in (1, 2, 8):
            assert not any(by_waves(t, k, b) for b in (32, 512, 1024, 4096, 14336))


def test_many_tokens_by_width(by_waves):
    for t in (1792, 2000, 4096, 1 << 20):
        assert by_waves(t, 2, 4096) and by_waves(t, 8, 1024) and by_waves(t, 64, 2)
        assert not by_waves(t, 2, 4098) and not by_waves(t, 8, 1026) and not by_waves(t, 65, 2)
