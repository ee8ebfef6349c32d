"""GPU tests of the token order: rows sorted by expert and back, with weights, and gradients.

Copies are compared bit for bit.  A sum of k fp32 terms w y is off by at most (k + 1) half steps of
2^-24 of the sum of their magnitudes; a dot product of h terms by (h + 64) of them (fused
multiplications, then the join); then the result is rounded once to its type."""
import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
ALL_TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def order_ref(ids, first, e):
    """Stable order on the host: offsets, perm, inv as lists."""
    flat = [i - first if 0 <= i - first < e else e for i in ids.flatten().tolist()]
    slots = sorted((s for s in range(len(flat)) if flat[s] < e), key=lambda s: (flat[s], s))
    offsets = [sum(1 for f in flat if f < x) for x in range(e + 1)] if len(flat) * e < 10 ** 6 else None
    if offsets is None:
        count = torch.bincount(torch.tensor(flat), minlength=e + 1)[:e]
        offsets = [0] + torch.cumsum(count, 0).tolist()
    perm = slots + [-1] * (len(flat) - len(slots))
    inv = [-1] * len(flat)
    for p, s in enumerate(slots):
        inv[s] = p
    return offsets, perm, inv


def close(got, ref, terms, n, what):
    """got against ref (64 bits), a sum of n terms of magnitudes `terms` in all."""
    eps = torch.finfo(got.dtype).eps / 2
    tol = terms * n * U
    tol = tol + (ref.abs() + tol) * eps + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    over = ((got.double() - ref).abs() - tol).max().item() if got.numel() else -1.0
    assert over <= 0, f"{what}: {over:.3e} over the tolerance"


# (t, h, k, ids drawn from [0, all), first, held)
CASES = [(1, 64, 1, 1, 0, 1), (1, 7168, 8, 256, 0, 256), (3, 33, 2, 5, 1, 3), (64, 2048, 8, 256, 64, 32),
         (65, 1, 4, 4096, 0, 4096), (511, 100, 8, 40, 0, 40), (512, 72, 8, 16, 0, 16), (513, 72, 8, 16, 4, 9),
         (777, 1001, 6, 40, 8, 24), (1500, 16, 3, 300, 0, 300), (4097, 130, 1, 7, 0, 7), (2500, 264, 2, 8, 3, 1),
         (2, 40, 600, 64, 0, 64), (3, 48, 2500, 64, 8, 40), (9000, 24, 2, 8, 7, 5), (300, 2056, 20, 32, 0, 32)]


def ids_of(g, t, k, n):
    return torch.randint(0, n, (t, k), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("t,h,k,n,first,held", CASES)
@pytest.mark.parametrize("dt", ALL_TYPES)
def test_order_and_gradients(lib, t, h, k, n, first, held, dt):
    """Every operator on one order; rows that no slot has hold NaN in the inputs and a mark in the
    outputs, which neither reaches nor leaves."""
    g = gen_of(t + h + k)
    ids = ids_of(g, t, k, n)
    p = t * k
    x = torch.randn(t, h, generator=g, device="cuda").to(dt)
    out = torch.full((p, h), 77.0, dtype=dt, device="cuda")
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, held, first=first, out=out)
    assert xp is out
    ref = order_ref(ids, first, held)
    assert offsets.tolist() == ref[0] and perm.tolist() == ref[1] and inv.flatten().tolist() == ref[2]
    total = ref[0][-1]
    slots = perm[:total].long()
    assert torch.equal(xp[:total], x[slots // k]) and (xp[total:] == 77).all()

    y = torch.randn(p, h, generator=g, device="cuda").to(dt)
    dxp = torch.randn(p, h, generator=g, device="cuda").to(dt)
    y[total:], dxp[total:] = float("nan"), float("nan")
    w = torch.rand(t, k, generator=g, device="cuda")
    w[torch.rand(t, k, generator=g, device="cuda") < 0.1] = 0
    add, dout = (torch.randn(t, h, generator=g, device="cuda").to(dt) for _ in range(2))

    def back(rows, terms=False):
        v = rows.double().abs() if terms else rows.double()
        return torch.zeros(t, h, dtype=torch.float64, device="cuda").index_add_(0, slots // k, v)

    ws = w.flatten()[slots, None].double()
    close(lib.moe_dispatch_backward(dxp, inv), back(dxp[:total]), back(dxp[:total], True), k + 1, "dx")
    wy = y[:total].double() * ws
    close(lib.moe_combine_forward(y, inv, w), back(wy), back(wy, True), k + 1, "out")
    close(lib.moe_combine_forward(y, inv, w, add=add), back(wy) + add.double(), back(wy, True) + add.double().abs(),
          k + 2, "out + add")
    close(lib.moe_combine_forward(y, inv), back(y[:total]), back(y[:total], True), k + 1, "out of ones")
    mark = torch.full((p, h), 55.0, dtype=dt, device="cuda")
    dy, dw = lib.moe_combine_backward(dout, y, inv, w, out=mark)
    assert dy is mark and (dy[total:] == 55).all()
    d = dout[slots // k].double()
    close(dy[:total], d * ws, torch.zeros_like(d), 0, "dy")
    if total:
        full, mag = (torch.zeros(p, dtype=torch.float64, device="cuda") for _ in range(2))
        full[slots], mag[slots] = (d * y[:total].double()).sum(1), (d * y[:total].double()).abs().sum(1)
        close(dw.flatten(), full, mag, h + 64, "dw")
    assert not dw.flatten()[inv.flatten() < 0].any()
    dy1, none = lib.moe_combine_backward(dout, y, inv)
    assert none is None and torch.equal(dy1[:total], dout[slots // k])


@pytest.mark.parametrize("t,h,k,n,first,held", [c for c in CASES if c[1] % 16 == 0])
@pytest.mark.parametrize("dt", ALL_TYPES)
def test_codes_in_order(lib, t, h, k, n, first, held, dt):
    """The sorted codes are the tokens' own codes in that order."""
    g = gen_of(t + h)
    x = (torch.randn(t, h, generator=g, device="cuda") * 3).to(dt)
    x[:, h // 3] *= 30
    ids = ids_of(g, t, k, n)
    q, s, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, held, first=first, quantize=True)
    xp, o2, p2, i2 = lib.moe_dispatch_forward(x, ids, held, first=first)
    assert torch.equal(offsets, o2) and torch.equal(perm, p2) and torch.equal(inv, i2)
    total = int(offsets[-1])
    tq, ts = lib.quantize_fp8_tokens(x)
    tok = perm[:total].long() // k
    assert torch.equal(q[:total].view(torch.uint8), tq.view(torch.uint8)[tok]) and torch.equal(s[:, :total], ts[:, tok])


def test_none_held_and_none_sent(lib):
    ids = torch.full((5, 3), 9, dtype=torch.int32, device="cuda")
    ids[0, 0], ids[1, 1] = -1, 2 ** 31 - 1
    x = torch.ones(5, 64, device="cuda")
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, 4)
    assert not offsets.any() and (perm == -1).all() and (inv == -1).all()
    y = torch.full((15, 64), float("nan"), device="cuda")
    assert not lib.moe_combine_forward(y, inv, torch.ones(5, 3, device="cuda")).any()
    assert not lib.moe_dispatch_backward(y, inv).any()
    assert not lib.moe_combine_backward(x, y, inv, torch.ones(5, 3, device="cuda"))[1].any()
    e = torch.zeros(0, 64, device="cuda")
    xp, offsets, perm, inv = lib.moe_dispatch_forward(e, ids[:0], 4)
    assert xp.shape == (0, 64) and not offsets.any() and perm.shape == (0,) and inv.shape == (0, 3)
    assert lib.moe_combine_forward(xp, inv).shape == (0, 64)
    dy, dw = lib.moe_combine_backward(e, xp, inv, torch.zeros(0, 3, device="cuda"))
    assert dy.shape == (0, 64) and dw.shape == (0, 3)


def test_inv_outside(lib):
    """Values of inv outside the rows count as dropped."""
    inv = torch.tensor([[0, -1], [4, 2], [-7, 2 ** 31 - 1]], dtype=torch.int32, device="cuda")
    y = torch.arange(6.0, device="cuda")[:, None].repeat(1, 40) + 1
    out = lib.moe_combine_forward(y, inv)
    assert torch.equal(out[:, 0], torch.tensor([1.0, 8.0, 0.0], device="cuda"))
    dy = torch.full_like(y, 3.0)
    dw = lib.moe_combine_backward(torch.ones(3, 40, device="cuda"), y, inv, torch.ones(3, 2, device="cuda"), out=dy)[1]
    assert dw.tolist() == [[40.0, 0.0], [200.0, 120.0], [0.0, 0.0]]
    assert dy[:, 0].tolist() == [1.0, 3.0, 1.0, 3.0, 1.0, 3.0]


def test_same_order_as_permute(lib):
    """With every expert held the order is moe_permute's."""
    for t, k, e in ((64, 8, 256), (1000, 8, 40), (6000, 2, 8)):
        ids = ids_of(gen_of(t), t, k, e)
        counts, offsets, perm, inv = lib.moe_permute(ids, e)
        got = lib.moe_dispatch_forward(torch.ones(t, 8, device="cuda"), ids, e)[1:]
        assert torch.equal(got[0], offsets) and torch.equal(got[1], perm) and torch.equal(got[2].flatten(), inv.flatten())


def test_rows_past_32_bits(lib):
    """Sorted rows past 2^32 bytes."""
    t, k, h = 70000, 8, 4104
    ids = ids_of(gen_of(1), t, k, 16)
    x = (torch.arange(t, device="cuda") % 251).to(torch.bfloat16)[:, None].repeat(1, h)
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, 16)
    assert xp.numel() * 2 > 2 ** 32
    tok = perm.long() // k
    assert torch.equal(xp[:, 0], x[tok, 0]) and torch.equal(xp[:, -1], x[tok, -1])
    for a in range(0, t * k, 40000):
        assert torch.equal(xp[a:a + 40000], x[tok[a:a + 40000]])
    out = lib.moe_dispatch_backward(xp, inv)
    assert torch.equal(out, (x.float() * 8).to(torch.bfloat16))
    dy, dw = lib.moe_combine_backward(x, xp, inv, torch.ones(t, k, device="cuda"), out=xp.clone())
    assert torch.equal(dy, xp)
    del dy, xp
    ref = (x[:, 0].double() ** 2 * h)[:, None].expand(t, k)
    assert ((dw.double() - ref).abs() <= ref * (h + 64) * U).all()


def test_gradients_against_differences(lib):
    """The operators are linear: sums along a direction agree with the gradients."""
    g = gen_of(7)
    t, k, h = 50, 4, 96
    ids = ids_of(g, t, k, 12)
    x, dirx, dout = (torch.randn(t, h, generator=g, device="cuda") for _ in range(3))
    w, dirw = (torch.randn(t, k, generator=g, device="cuda") for _ in range(2))

    def f(xv, wv):
        xp, _, _, inv = lib.moe_dispatch_forward(xv, ids, 9, first=2, out=torch.zeros(t * k, h, device="cuda"))
        return lib.moe_combine_forward(xp, inv, wv), xp, inv

    out, xp, inv = f(x, w)
    dyp, dw = lib.moe_combine_backward(dout, xp, inv, w, out=torch.zeros_like(xp))
    dx = lib.moe_dispatch_backward(dyp, inv)
    for got, d, along in ((dx, dirx, f(dirx, w)[0]), (dw, dirw, f(x, dirw)[0])):
        lhs, rhs = (dout.double() * along.double()).sum(), (got.double() * d.double()).sum()
        scale = (dout.double() * along.double()).abs().sum() + (got.double() * d.double()).abs().sum()
        assert (lhs - rhs).abs() <= scale * (h + 64) * 2 * U


def test_equal_bits(lib):
    g = gen_of(8)
    for t in (40, 3000):
        ids = ids_of(g, t, 8, 32)
        y = torch.randn(t * 8, 520, generator=g, device="cuda").bfloat16()
        w = torch.rand(t, 8, generator=g, device="cuda")
        dout = torch.randn(t, 520, generator=g, device="cuda").bfloat16()
        inv = lib.moe_dispatch_forward(dout, ids, 32)[3]
        one = lib.moe_combine_forward(y, inv, w), *lib.moe_combine_backward(dout, y, inv, w)
        for _ in range(3):
            two = lib.moe_combine_forward(y, inv, w), *lib.moe_combine_backward(dout, y, inv, w)
            assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_experts_outside(lib):
    """Experts that 32 bits do not hold are refused, not wrapped."""
    x, ids = torch.ones(3, 16, device="cuda"), torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    for n, first in ((0, 0), (4097, 0), (2 ** 32 + 4, 0), (4, -1), (4, 2 ** 32), (4, 2 ** 31 - 4)):
        with pytest.raises(ValueError):
            lib.moe_dispatch_forward(x, ids, n, first=first)
    ids[0, 0] = -2 ** 31
    ids[1, 1] = 2 ** 31 - 2
    assert lib.moe_dispatch_forward(x, ids, 4, first=2 ** 31 - 5)[1].tolist() == [0, 0, 0, 0, 1]


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("h", [7, 64, 513])
def test_rows_keep_their_bits(lib, dt, h):
    """Rows are copied bit by bit: every 16-bit pattern, NaNs of either kind in fp32, whole vectors
    and what is left of a row."""
    bits = torch.int32 if dt is torch.float32 else torch.int16
    n = -(-65536 // h) * h
    v = torch.arange(n, device="cuda") % 65536
    v = (v << 16 | 0x7fa00001).to(torch.int32) if dt is torch.float32 else v.to(torch.int16)
    x = v.view(dt).view(-1, h)
    ids = ids_of(gen_of(h), x.shape[0], 2, 5)
    xp, offsets, perm, inv = lib.moe_dispatch_forward(x, ids, 5)
    assert torch.equal(xp.view(bits), x.view(bits)[perm.long() // 2])
