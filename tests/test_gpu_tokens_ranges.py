"""GPU tests of the token order where its launches change: one range of slots or several, tokens by
workgroups or by waves.  Rows and codes are compared bit for bit."""
import pytest
import torch

from tests.test_gpu_tokens import ALL_TYPES, gen_of, ids_of, lib, order_ref  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,k", [(1791, 1), (1792, 1), (2047, 1), (2048, 1), (2049, 1), (1791, 2), (1793, 2), (1795, 64),
                                 (1800, 65), (300, 6), (342, 6), (4, 512), (5, 512)])
@pytest.mark.parametrize("h", [16, 512, 2064])
@pytest.mark.parametrize("dt", ALL_TYPES)
def test_ranges(lib, t, k, h, dt):  # noqa: F811
    g = gen_of(t + k + h)
    ids = ids_of(g, t, k, 40)
    x = torch.randn(t, h, generator=g, device="cuda").to(dt)
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, 24, first=8,
                                                      out=torch.full((t * k, h), 77.0, dtype=dt, device="cuda"))
    ref = order_ref(ids, 8, 24)
    assert offsets.tolist() == ref[0] and perm.tolist() == ref[1] and inv.flatten().tolist() == ref[2]
    total = ref[0][-1]
    tok = perm[:total].long() // k
    assert torch.equal(xp[:total], x[tok]) and (xp[total:] == 77).all()
    q, s, o2, p2, i2 = lib.moe_dispatch_forward(x, ids, 24, first=8, quantize=True)
    assert torch.equal(o2, offsets) and torch.equal(p2, perm) and torch.equal(i2, inv)
    tq, ts = lib.quantize_fp8_tokens(x)
    assert torch.equal(q[:total].view(torch.uint8), tq.view(torch.uint8)[tok]) and torch.equal(s[:, :total], ts[:, tok])
