"""The binding on a torch without the private device and stream calls."""
import subprocess
import sys

import pytest
import torch

from tests.conftest import ROOT
from tests.helpers import require_gpu


def test_import_without_private_torch_calls():
    code = ("import torch\n"
            "for name in ('_cuda_getDevice', '_cuda_getCurrentRawStream'):\n"
            "    if hasattr(torch._C, name):\n"
            "        delattr(torch._C, name)\n"
            "from int4_group_quantized_g128_amd import _lib\n"
            "assert _lib._current_device is torch.cuda.current_device\n"
            "assert _lib._raw_stream is _lib._public_raw_stream\n")
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert res.returncode == 0, res.stderr


@pytest.mark.gpu
def test_public_calls_give_the_current_stream(monkeypatch):
    require_gpu()
    from int4_group_quantized_g128_amd import _lib
    side = torch.cuda.Stream()
    for s in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(s):
            assert _lib._raw_stream(0) == _lib._public_raw_stream(0) == s.cuda_stream
    x = torch.randn(5, 264, device="cuda")
    w = torch.ones(264, device="cuda")
    want = _lib.block_norm_forward(x, w_pre=w)[1]
    monkeypatch.setattr(_lib, "_current_device", torch.cuda.current_device)
    monkeypatch.setattr(_lib, "_raw_stream", _lib._public_raw_stream)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = _lib.block_norm_forward(x, w_pre=w)[1]
    side.synchronize()
    assert torch.equal(got, want)
