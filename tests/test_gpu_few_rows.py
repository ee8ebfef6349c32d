"""GPU tests of the e4m3 product's few-rows kernel, bit for bit (operands whose products and sums are
exact in fp32, as in the products' other tests)."""
import pytest
import torch

from tests.few_rows_shapes import PASSES, SCATTERED
from tests.helpers import require_gpu
from tests.test_gpu_fp8 import E4M3, TYPES, assert_equal, by_expert, ceil, gen_of, halves, offsets_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


@pytest.mark.parametrize("t,k,n,e,held", SCATTERED)
@pytest.mark.parametrize("dt", TYPES)
def test_scattered_experts(lib, t, k, n, e, held, dt):
    """Few rows at a few of many experts; the codes and scales of the others are NaN."""
    g = gen_of(t + n)
    x = halves(g, t, k) / 64
    q, s = lib.quantize_fp8_tokens(x)
    wq = torch.full((e, n, k), 0x7f, dtype=torch.uint8, device="cuda").view(E4M3)
    ws = torch.full((e, ceil(n), ceil(k)), torch.nan, device="cuda")
    w = {z: halves(g, n, k) / 64 for z in held}
    for z, v in w.items():
        wq[z], ws[z] = lib.quantize_fp8_blocks(v)
    counts = [held.get(z, 0) for z in range(e)]
    total = sum(counts)
    assert total <= t
    off = offsets_of(counts)
    y = torch.full((t, n), 9.0, dtype=dt, device="cuda")
    lib.fp8_linear_forward(q, s, wq, ws, offsets=off, out_dtype=dt, out=y)
    for z, v in w.items():
        r = slice(int(off[z]), int(off[z + 1]))
        assert_equal(y[r], x[r].double() @ v.double().T, f"expert {z}")
    assert (y[total:] == 9).all()


@pytest.mark.parametrize("shape", PASSES, ids=str)
@pytest.mark.parametrize("dt", TYPES)
def test_passes(lib, shape, dt):
    counts, k, n = shape[0], shape[-3], shape[-2]
    t, e = (shape[1], 1) if counts is None else (sum(counts), len(counts))
    g = gen_of(t + k + n)
    x = halves(g, t, k) / 64
    w = torch.stack([halves(g, n, k) / 64 for _ in range(e)])
    q, s = lib.quantize_fp8_tokens(x)
    if counts is None:
        y = lib.fp8_linear_forward(q, s, *lib.quantize_fp8_blocks(w[0]), out_dtype=dt)
        return assert_equal(y, x.double() @ w[0].double().T, "y")
    y = lib.fp8_linear_forward(q, s, *lib.quantize_fp8_blocks(w), offsets=offsets_of(counts), out_dtype=dt)
    for z, (r, one) in enumerate(by_expert(counts, 0, lambda z, r: (r, x[r].double() @ w[z].double().T))):
        assert_equal(y[r], one, f"expert {z}")
