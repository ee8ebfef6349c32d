"""The token order and the e4m3 products record no autograd graph, and say so."""
import pytest
import torch

from tests.helpers import require_gpu

NAMES = ["moe_dispatch_forward", "moe_dispatch_backward", "moe_combine_forward", "moe_combine_backward",
         "quantize_fp8_tokens", "quantize_fp8_blocks", "fp8_linear_forward", "fp8_linear_backward"]


@pytest.mark.parametrize("name", NAMES)
def test_said(name):
    import int4_group_quantized_g128_amd as lib
    assert "autograd graph" in " ".join(getattr(lib, name).__doc__.split())


@pytest.mark.gpu
def test_no_graph():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    leaf = lambda *s: torch.ones(s, device="cuda").requires_grad_()
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    x, w = leaf(4, 64), leaf(4, 2)
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, 1)
    q, s, qc, sc = lib.quantize_fp8_tokens(leaf(8, 64), columns=True, offsets=offsets)
    wq, ws = lib.quantize_fp8_blocks(leaf(1, 32, 64))
    y = lib.fp8_linear_forward(q, s, wq, ws, offsets=offsets)
    dy = torch.ones(8, 32, dtype=torch.bfloat16, device="cuda").requires_grad_()
    outs = [xp, q, s, qc, sc, wq, ws, y, lib.moe_combine_forward(leaf(8, 64), inv, w, add=x),
            *lib.moe_combine_backward(x, leaf(8, 64), inv, w), lib.moe_dispatch_backward(leaf(8, 64), inv),
            *lib.fp8_linear_backward(dy, qc, sc, wq, ws, offsets=offsets)]
    assert not any(v.requires_grad for v in outs)
