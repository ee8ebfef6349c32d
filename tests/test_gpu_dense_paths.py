"""Every kernel, tile and K split of the dense products (test_dense_plan.py checks that the
shapes below take them all) against 64 bits, for equal bits, repeated and guarded."""
import pytest
import torch

import tests.test_gpu_dense as base
from tests.helpers import require_gpu
from tests.test_gpu_dense import ALL_TYPES, TYPES, U, codes, gen_of, half_step, randn, swiglu_inputs, tiny, within

pytestmark = pytest.mark.gpu

# t, k, n: few rows (one and two fragments a wave), then tiles of 64, 128 and 256, each with K whole and split
INT8_SHAPES = [(5, 144, 33), (9, 208, 7001), (333, 1040, 1001), (20, 3328, 19), (204, 1664, 12738), (71, 8144, 8283),
               (778, 64, 7681), (131, 7152, 5544), (5472, 6944, 133)]
# t, h, i: forward 64 whole and split, 128 whole and split, 256 whole and split, ...
SWIGLU_SHAPES = [(5, 72, 40), (9, 72, 3600), (21, 64, 72), (17, 1712, 72), (201, 792, 6848), (66, 3680, 4352),
                 (471, 64, 6216), (146, 3968, 2936),
                 # ... dx 128 whole and split, 256 whole (and dw 128 split), 256 split,
                 (464, 6168, 64), (70, 6168, 2392), (2761, 4392, 72), (130, 5912, 3464),
                 # ... dw 64 split, 256 whole and split
                 (2241, 72, 64), (65, 6472, 920), (2626, 2336, 848)]
# row counts that take every plan at one k, n (odd; a multiple of 8)
EQUAL_BITS = [((1, 5, 17, 130, 200, 400, 700, 1700), 7264, 4835), ((1, 17, 130, 200, 400, 700, 1700), 7264, 4840)]


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,k,n", INT8_SHAPES)
def test_int8_linear(lib, t, k, n, dt):
    base.test_int8_linear(lib, t, k, n, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", SWIGLU_SHAPES)
def test_swiglu_linear_forward(lib, t, h, i, dt):
    base.test_swiglu_linear_forward(lib, t, h, i, dt)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", SWIGLU_SHAPES)
def test_swiglu_linear_backward(lib, t, h, i, dt):
    base.test_swiglu_linear_backward(lib, t, h, i, dt)


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("rows,k,n", EQUAL_BITS)
def test_int8_linear_equal_bits_on_every_plan(lib, rows, k, n, dt):
    """A row's result does not depend on the rows beside it, with and without a bias, and is
    what the definition gives in fp32: one rounding of the INT32 sum, one of the scales'
    product, one of the product of both with the bias added."""
    g = gen_of(k + n)
    q, wq = codes(g, max(rows), k), codes(g, n, k)
    s, ws = torch.rand(max(rows), generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    acc = q.double() @ wq.double().T   # exact: below 2^53
    for bias in (None, randn(g, n, std=1e4)):
        full = lib.int8_linear_forward(q, s, wq, ws, bias=bias, out_dtype=dt)
        # sum and scales' product have 24 bits each, so their product is exact in fp64; adding the
        # bias there rounds once more before fp32 does, which is off by one step at most
        want = acc.float().double() * (s[:, None] * ws).double() + (0 if bias is None else bias.double())
        exact = want.float()
        if bias is None:
            assert torch.equal(full, exact.to(dt))
        else:
            same = full == exact.to(dt)   # (infinities of fp16 among them)
            off = (full.double() - exact.to(dt).double()).abs()
            assert (same | (off <= torch.finfo(dt).eps * want.abs() * (1 + 2.0 ** -7) + tiny(dt))).all()
            assert same.double().mean() > 0.999
        for t in rows:
            got = lib.int8_linear_forward(q[:t], s[:t], wq, ws, bias=bias, out_dtype=dt)
            assert torch.equal(got, full[:t]), (t, bias is not None)


@pytest.mark.parametrize("t,k,n", [(130, 144, 257 + e) for e in range(8)] +
                         [(778, 64, 7680 + e) for e in (0, 4, 1)] + [(204, 1664, 12736 + e) for e in (0, 4, 2)])
def test_int8_linear_every_row_end(lib, t, k, n):
    """Rows that end anywhere in a lane's eight columns, stored in vectors of 8 and 4 or singly as
    the row length allows, between guards."""
    r = lib._lib.raw
    g = gen_of(n)
    q, wq = codes(g, t, k), codes(g, n, k)
    s, ws = torch.rand(t, generator=g, device="cuda") * 1e-3, torch.rand(n, generator=g, device="cuda") * 1e-3
    want = ((q.double() @ wq.double().T).float().double() * (s[:, None] * ws).double()).float()
    for dt in ALL_TYPES:
        b = base.Guarded()
        y = b.new(t, n, dtype=dt)
        nbytes = r.int8_linear_workspace_bytes(t, k, n)
        work = b.new(max(nbytes, 16), dtype=torch.uint8)
        assert r.int8_linear_forward(base.ptr(q), base.ptr(s), t, k, base.ptr(wq), base.ptr(ws), n, None,
                                     lib._lib._DT[dt], base.ptr(y), base.ptr(work), nbytes, base.stream()) == 0
        b.check()
        assert torch.equal(y, want.to(dt))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", [(17, 1712, 72), (66, 3680, 4352), (146, 3968, 2936), (70, 6168, 2392),
                                   (130, 5912, 3464), (2241, 72, 64), (2761, 4392, 72), (2626, 2336, 848)])
def test_split_products_repeat_and_write_only_their_outputs(lib, t, h, i, dt):
    r, code = lib._lib.raw, lib._lib._DT[dt]
    x, wg, wu, dh = swiglu_inputs(t, h, i, dt, 4)
    ptr, stream = base.ptr, base.stream
    ref, gu_ref = lib.swiglu_linear_forward(x, wg, wu, save=True)
    grads = lib.swiglu_linear_backward(dh, x, wg, wu, gu_ref)
    for fill in (0, 0xFF):   # a workspace of zeros and of NaN
        b = base.Guarded()
        out, gu = b.new(t, i, dtype=dt), b.new(t, 2, i, dtype=torch.float32)
        nbytes = r.swiglu_linear_workspace_bytes(t, h, i)
        work = b.new(max(nbytes, 16), dtype=torch.uint8).fill_(fill)
        assert r.swiglu_linear_forward(ptr(x), ptr(wg), ptr(wu), t, h, i, code, ptr(out), ptr(gu), ptr(work), nbytes,
                                       stream()) == 0
        dx, dwg, dwu = b.new(t, h, dtype=dt), b.new(i, h, dtype=dt), b.new(i, h, dtype=dt)
        nbytes = r.swiglu_linear_backward_workspace_bytes(t, h, i)
        work = b.new(nbytes, dtype=torch.uint8).fill_(fill)
        assert r.swiglu_linear_backward(ptr(dh), ptr(x), ptr(wg), ptr(wu), ptr(gu), t, h, i, code, ptr(dx), ptr(dwg),
                                        ptr(dwu), ptr(work), nbytes, stream()) == 0
        b.check()
        assert torch.equal(out, ref) and torch.equal(gu, gu_ref)
        assert all(torch.equal(a, c) for a, c in zip((dx, dwg, dwu), grads))


@pytest.mark.parametrize("t,k,n", [(20, 3328, 19), (71, 8144, 8283), (131, 7152, 5544)])
def test_split_int8_products_repeat_and_write_only_their_output(lib, t, k, n):
    r = lib._lib.raw
    g = gen_of(t + n)
    q, wq = codes(g, t, k), codes(g, n, k)
    s, ws = torch.rand(t, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    for dt in ALL_TYPES:
        ref = lib.int8_linear_forward(q, s, wq, ws, out_dtype=dt)
        for fill in (0, 0xFF):
            b = base.Guarded()
            y = b.new(t, n, dtype=dt)
            nbytes = r.int8_linear_workspace_bytes(t, k, n)
            assert nbytes > 0
            work = b.new(nbytes, dtype=torch.uint8).fill_(fill)
            assert r.int8_linear_forward(base.ptr(q), base.ptr(s), t, k, base.ptr(wq), base.ptr(ws), n, None,
                                         lib._lib._DT[dt], base.ptr(y), base.ptr(work), nbytes, base.stream()) == 0
            b.check()
            assert torch.equal(y, ref)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", [(70, 136, 72), (130, 264, 520), (17, 1712, 72)])
def test_swiglu_linear_gradient_along_itself(lib, t, h, i, dt):
    """Forward and backward pass against differences of the 64-bit loss sum(dh h) along the sign
    of its own gradient (by automatic differentiation), where the difference is the sum of the
    gradient's magnitudes, and against that gradient element by element.

    A gradient entry carries one rounding of the result (half a step of it), one of dg and du
    (half a step of every term of its sum) and fp32 sums of h, then of i or t terms:
    |dg| <= 1.1 |dh u|, |du| <= |dh g|."""
    x, wg, wu, dh = swiglu_inputs(t, h, i, dt, 2)
    _, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
    grads = [v.double() for v in lib.swiglu_linear_backward(dh, x, wg, wu, gu)]
    p = [v.double().requires_grad_() for v in (x, wg, wu)]
    d = dh.double()

    def loss(x, wg, wu):
        g = x @ wg.T
        return (d * (g * torch.sigmoid(g)) * (x @ wu.T)).sum()

    auto = torch.autograd.grad(loss(*p), p)
    p = [v.detach() for v in p]
    xa, ga, ua = (v.abs() for v in p)
    # g and u carry 2 h u of their sums' magnitudes, so do dg and du of theirs (|sig''| < 1)
    eg, eu = 2 * h * U * (xa @ ga.T), 2 * h * U * (xa @ ua.T)
    g, u = (p[0] @ p[1].T).abs(), (p[0] @ p[2].T).abs()
    ag, au = 1.1 * d.abs() * u, d.abs() * g
    hs = half_step(dt)
    fg = hs * ag + d.abs() * (1.1 * eu + u * eg) + 32 * U * d.abs() * u * (1 + g) + tiny(dt)
    fu = hs * au + d.abs() * 1.1 * eg + 32 * U * au + tiny(dt)
    n = max(i, t) * 4 * U
    tols = [(fg + n * ag) @ ga + (fu + n * au) @ ua, (fg + n * ag).T @ xa, (fu + n * au).T @ xa]
    e = 1e-5
    for j, name in enumerate(("dx", "dw_gate", "dw_up")):
        tol = 1.01 * (tols[j] + hs * (auto[j].abs() + tols[j])) + tiny(dt)
        within(grads[j], auto[j], tol, name)
        v = torch.sign(auto[j])
        plus, minus = list(p), list(p)
        plus[j], minus[j] = p[j] + e * v, p[j] - e * v
        diff = (loss(*plus) - loss(*minus)) / (2 * e)
        assert tol.sum() < 0.25 * diff, "the tolerance is well below what it measures"
        # (the differences' own error: e^2 and 2^-53 / e of the loss's terms)
        assert abs((grads[j] * v).sum() - diff) <= tol.sum() + 1e-6 * diff, name
