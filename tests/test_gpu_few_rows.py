"""GPU tests of the e4m3 product's few-rows kernel, bit for bit (operands whose products and sums are
exact in fp32, as in the products' other tests)."""
import pytest
import torch

from tests.few_rows_shapes import PASSES, SCATTERED, SIXTEEN, SIXTY_FOUR
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


def beside_large(g, t, n, k):
    """x [t, k] and w [n, k] whose codes are their values: in each eight of the summed index one product
    of +-448^2 and seven of at most 4 in steps of 1 / 4; the large ones cancel within each group of 128.  Every
    sum in any order is a multiple of 1 / 4 below 2^22, exact in fp32; one that drops what is 2^-13
    below an eight's largest loses nearly all of the result."""
    small = lambda rows: torch.randint(1, 5, (rows, k), generator=g, device="cuda") * 0.5 * (
        torch.randint(0, 2, (rows, k), generator=g, device="cuda") * 2.0 - 1)
    x, w = small(t), small(n)
    eights = torch.arange(k // 8, device="cuda")
    at = eights * 8 + torch.randint(0, 8, (k // 8,), generator=g, device="cuda")
    sign = torch.randint(0, 2, (k // 8,), generator=g, device="cuda") * 2.0 - 1
    x[:, at], w[:, at] = 448 * sign, 448 * sign * (1 - 2.0 * (eights % 2))
    return x, w


@pytest.mark.parametrize("t,k,n,counts", SIXTEEN + SIXTY_FOUR)
@pytest.mark.parametrize("dt", TYPES)
def test_small_products_beside_large_ones(lib, t, k, n, counts, dt):
    """Up to 16 rows, and whatever else the few-rows kernel takes, are multiplied without the narrow matrix
    instructions' loss."""
    g = gen_of(t + k + n)
    x, w = beside_large(g, t, n, k)
    q, s = lib.quantize_fp8_tokens(x)
    assert (s == 1).all()
    if counts is None:
        return assert_equal(lib.fp8_linear_forward(q, s, *lib.quantize_fp8_blocks(w), out_dtype=dt),
                            x.double() @ w.double().T, "y")
    scale = [2.0 ** (z % 3) for z in range(len(counts))]   # experts that differ
    wq, ws = lib.quantize_fp8_blocks(torch.stack([w * v for v in scale]))
    y = lib.fp8_linear_forward(q, s, wq, ws, offsets=offsets_of(counts), out_dtype=dt)
    at = 0
    for c, v in zip(counts, scale):
        assert_equal(y[at:at + c], x[at:at + c].double() @ w.double().T * v, "y of an expert")
        at += c
    assert at <= t


def test_searched_runs_in_a_graph(lib):
    """A captured product finds the runs of the offsets that it meets at each replay."""
    t, k, n, e = 8, 2064, 1040, 300
    g = gen_of(2)
    x, w = halves(g, t, k) / 64, torch.stack([halves(g, n, k) / 64 for _ in range(e)])
    q, s = lib.quantize_fp8_tokens(x)
    wq, ws = lib.quantize_fp8_blocks(w)
    off = offsets_of([0] * e)
    y = torch.empty(t, n, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.fp8_linear_forward(q, s, wq, ws, offsets=off, out=y)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.fp8_linear_forward(q, s, wq, ws, offsets=off, out=y)
    for held in ({0: 8}, {299: 1}, {}, {z: 1 for z in range(60, 68)}, {255: 3, 256: 5}, {0: 8}):
        off.copy_(offsets_of([held.get(z, 0) for z in range(e)]))
        y.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.full_like(y, 9)
        lib.fp8_linear_forward(q, s, wq, ws, offsets=off, out=want)
        assert torch.equal(y, want)
        at = 0
        for z, c in sorted(held.items()):
            assert_equal(y[at:at + c], x[at:at + c].double() @ w[z].double().T, f"expert {z}")
            at += c
        assert (y[at:] == 9).all()


def test_searched_runs_of_offsets_not_ascending(lib):
    """More runs than there can be with ascending offsets: nothing outside the result is written."""
    t, k, n, e = 6, 1040, 520, 256
    q, s = lib.quantize_fp8_tokens(torch.ones(t, k, device="cuda"))
    wq, ws = lib.quantize_fp8_blocks(torch.ones(e, n, k, device="cuda"))
    for off in ([0, t] * (e // 2) + [0], [t] + [0] * (e - 1) + [2 ** 31 - 1], [-5, 2 ** 31 - 1] * (e // 2) + [3],
                list(range(e, -1, -1))):
        buf = torch.full((t * n + 128,), -3.0, dtype=torch.bfloat16, device="cuda")
        y = buf[64:64 + t * n].view(t, n)
        lib.fp8_linear_forward(q, s, wq, ws, offsets=torch.tensor(off, dtype=torch.int32, device="cuda"), out=y)
        assert (buf[:64] == -3).all() and (buf[64 + t * n:] == -3).all()
        assert ((y == -3) | (y == k)).all()
