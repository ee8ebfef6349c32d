"""The large tiles' panels start at LDS addresses that their transposing reads allow (CPU: the device
code's declarations as the compiler's front end lays them down)."""
import os
import re
import subprocess

import pytest

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def declared(tmp_path_factory):
    """-> (kernel, LDS variable, alignment) of every __shared__ variable of the e4m3 products."""
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    if not os.path.exists(hipcc):
        pytest.skip("no hipcc")
    out = tmp_path_factory.mktemp("lds") / "fp8.ll"
    subprocess.run([hipcc, "--offload-arch=gfx950", "-O3", "-std=c++17", "--cuda-device-only", "-S", "-emit-llvm",
                    "-Xclang", "-disable-llvm-passes", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                    "-o", str(out), os.path.join(ROOT, "int4_group_quantized_g128_amd", "csrc", "fp8.hip")],
                   check=True, capture_output=True)
    found = []
    for line in out.read_text().splitlines():
        m = re.match(r"@(\S+) = .*addrspace\(3\) global .*align (\d+)", line)
        if m:
            kernel, name = re.search(r"\d(k_[a-z0-9_]+?)I.*E\d([a-z]+)$", m.group(1)).groups()
            found.append((kernel, name, int(m.group(2))))
    return found


def test_panels_of_the_large_tiles(declared):
    """Columns 16, 32 and 48 on are read by flipping bits 4 and 5 of an address."""
    panels = [align for kernel, name, align in declared if kernel == "k_fp8_big" and name == "mem"]
    assert len(panels) == 6 and all(align % 64 == 0 for align in panels), panels   # y, dx, dW by 128 and 256
