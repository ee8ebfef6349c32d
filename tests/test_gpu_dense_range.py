"""The gated projection's gradients where dg = dh u sig(g) (1 + g (1 - sig(g))) and du = dh silu(g)
leave the range of fp16 while the gradients themselves are within it.

dg and du are matrix-core operands of 16 bits.  In fp16 each token's row (for dx) and each
column (for dw_gate, dw_up) carries a power of two that puts its largest magnitude into
[2^14, 2^15): an element is off by half a step of the type, hs |v|, or by 2^-25 of the scaled
value, at most 2^-39 of that largest magnitude.  Other roundings as in test_gpu_dense.py."""
import pytest
import torch

from tests.helpers import require_gpu
from tests.test_gpu_dense import U, gen_of, half_step, randn, swiglu_grads, tiny, within

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8, 8), (5, 72, 40), (33, 512, 520), (130, 1000, 1032), (300, 264, 4104), (1300, 72, 4360),
          (2200, 2568, 640)]
DT = torch.float16


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


def powers(gen, n, lo, hi):
    return torch.exp2(torch.randint(lo, hi + 1, (n,), generator=gen, device="cuda").double()).float()


def inputs(t, h, i, kind):
    """dh, x, w_gate, w_up, gu with dg and du up to 2^24 ("large"), below 2^-24 ("small"), or rows
    and columns of magnitudes 2^32 apart ("mixed")."""
    g = gen_of(t + h + i)
    dh, x = randn(g, t, i), randn(g, t, h)
    wg, wu = randn(g, i, h, std=h ** -0.5), randn(g, i, h, std=h ** -0.5)
    gu = randn(g, t, 2, i)
    if kind == "large":
        dh, gu, x, wg, wu = dh * 2.0 ** 11, gu * 2.0 ** 7, x * 2.0 ** -14, wg * 2.0 ** -12, wu * 2.0 ** -12
    elif kind == "small":
        dh, gu, x, wg, wu = dh * 2.0 ** -13, gu * 2.0 ** -13, x * 2.0 ** 9, wg * 2.0 ** 9, wu * 2.0 ** 9
    else:
        dh = dh * powers(g, t, -11, 11)[:, None]
        gu = gu * powers(g, i, -10, 6)
        x, wg, wu = x * 2.0 ** -10, wg * 2.0 ** -9, wu * 2.0 ** -9
    return dh.to(DT), x.to(DT), wg.to(DT), wu.to(DT), gu


def reference(dh, x, wg, wu, gu):
    """64-bit gradients, each with its tolerance."""
    d, xd, gd, ud = dh.double(), x.double(), wg.double(), wu.double()
    g, u = gu[:, 0].double(), gu[:, 1].double()
    t, i = g.shape
    dg, du, rx, rg, ru = swiglu_grads(d, xd, gd, ud, g, u)
    hs = half_step(DT)
    # dg, du: 8 fp32 operations on terms up to |dh u| (1 + |g|), one rounding to fp16
    eg = 32 * U * (d * u).abs() * (1 + g.abs()) + hs * dg.abs() * (1 + hs)
    eu = 32 * U * (d * g).abs() + hs * du.abs() * (1 + hs)
    low = 2.0 ** -39
    row = torch.maximum(dg.abs().amax(1), du.abs().amax(1))[:, None] * low
    er, fr = eg + row, eu + row
    ag, au = dg.abs() + er, du.abs() + fr
    tol = er @ gd.abs() + fr @ ud.abs() + 4 * i * U * (ag @ gd.abs() + au @ ud.abs())
    out = [(rx, tol + hs * (rx.abs() + tol) + tiny(DT))]
    for r, v, e in ((rg, dg, eg), (ru, du, eu)):
        e = e + v.abs().amax(0) * low
        tol = e.T @ xd.abs() + 2 * t * U * ((v.abs() + e).T @ xd.abs())
        out.append((r, tol + hs * (r.abs() + tol) + tiny(DT)))
    return dg, du, out


@pytest.mark.parametrize("kind", ["large", "small", "mixed"])
@pytest.mark.parametrize("t,h,i", SHAPES)
def test_fp16_gradients_outside_the_operands_range(lib, t, h, i, kind):
    args = inputs(t, h, i, kind)
    dg, du, ref = reference(*args)
    top = max(dg.abs().max(), du.abs().max())
    if kind != "small":
        assert t * i < 1000 or top > 65504
    else:
        assert top < 2.0 ** -15
    got = lib.swiglu_linear_backward(*args)
    for name, v, (r, tol) in zip(("dx", "dw_gate", "dw_up"), got, ref):
        assert r.abs().max() < 60000, "the gradients themselves are within fp16"
        within(v, r, tol, name)


def test_fp16_gradients_nonfinite_entries_stay_in_their_row_and_column(lib):
    """An infinite or NaN dh spoils its token's dx and its column of the weight gradients; all
    other results are as close as without it."""
    for bad in (float("inf"), float("nan")):
        for t, h, i in ((70, 136, 72), (300, 264, 520)):
            dh, x, wg, wu, gu = inputs(t, h, i, "mixed")
            row, col = t // 2, i - 3
            dh[row, col] = bad
            got = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
            dh[row, col] = 0
            _, _, ref = reference(dh, x, wg, wu, gu)
            for v, (r, tol), at in zip(got, ref, (row, col, col)):
                assert not torch.isfinite(v[at]).any()
                keep = [k for k in range(v.shape[0]) if k != at]
                within(v[keep], r[keep], tol[keep])


def test_fp16_gradients_of_zero_rows_and_columns(lib):
    """A token without gradient (padding) and a column without: exact zeros there."""
    dh, x, wg, wu, gu = inputs(130, 72, 264, "large")
    dh[7:50] = 0
    dh[:, 100:140] = 0
    dx, dwg, dwu = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
    assert not dx[7:50].any() and not dwg[100:140].any() and not dwu[100:140].any()
    _, _, ref = reference(dh, x, wg, wu, gu)
    for v, (r, tol) in zip((dx, dwg, dwu), ref):
        within(v, r, tol)


def test_fp16_gradients_captured(lib):
    """The fp16 backward pass in a graph, replayed with other gradients and eager work between."""
    dh, x, wg, wu, gu = inputs(130, 264, 1032, "mixed")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        lib.swiglu_linear_backward(dh, x, wg, wu, gu)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
    for rep in range(4):
        dh.copy_((randn(gen_of(rep), *dh.shape) * 2.0 ** (4 * rep - 8)).to(DT))
        graph.replay()
        torch.cuda.synchronize()
        want = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), rep


def test_fp16_gradients_offsets_past_32_bits(lib):
    """More than 2^31 elements of dh, all rows but the last ones zero: the weight gradients are
    those of the last rows, and so are their dx."""
    t, h, i, tail = 270000, 8, 8192, 100
    few = inputs(tail, h, i, "mixed")
    dh, x, gu = (torch.zeros(t, *v.shape[1:], dtype=v.dtype, device="cuda") for v in (few[0], few[1], few[4]))
    dh[-tail:], x[-tail:], gu[-tail:] = few[0], few[1], few[4]
    _, _, ref = reference(*few)
    dx, dwg, dwu = lib.swiglu_linear_backward(dh, x, few[2], few[3], gu)
    assert not dx[:-tail].any()
    # (the weight gradients' sums run over the zero rows too, which adds no rounding)
    for v, (r, tol) in zip((dx[-tail:], dwg, dwu), ref):
        within(v, r, tol)
