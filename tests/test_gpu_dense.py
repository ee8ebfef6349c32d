"""GPU tests of the dense operators against plain computations in 64 bits.

Tolerances count roundings.  u = 2^-24 is half a step of fp32, h = finfo(dtype).eps / 2 half
a step of the stored type.  A sum of K fp32 terms (exact products) is off by at most
2 K u sum|terms| (the factor 2 for the matrix core's own rounding of partial sums)."""
import pytest
import torch

from tests.helpers import require_gpu

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = [torch.bfloat16, torch.float16]
ALL_TYPES = TYPES + [torch.float32]


@pytest.fixture(scope="module")
def lib():
    require_gpu()
    import int4_group_quantized_g128_amd as lib
    return lib


def half_step(dt):
    return torch.finfo(dt).eps / 2


def tiny(dt):
    """Half a step at the bottom of the type's range (fp16 subnormals)."""
    return torch.finfo(dt).smallest_normal * torch.finfo(dt).eps


def randn(gen, *shape, std=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * std


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def within(got, ref, tol, what=""):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    worst = ((got - ref).abs() - tol).max().item() if got.numel() else -1.0
    assert worst <= 0, f"{what}: {worst:.3e} over the tolerance"


# ------------------------------------------------------------------ INT8 linear
def codes(gen, rows, k):
    return torch.randint(-128, 128, (rows, k), generator=gen, device="cuda", dtype=torch.int8)


def int8_ref(q, s, wq, ws, bias):
    y = (q.double() @ wq.double().T) * (s.double()[:, None] * ws.double())
    return y if bias is None else y + bias.double()


@pytest.mark.parametrize("t,k,n", [(1, 16, 1), (1, 2048, 2048), (3, 144, 33), (16, 1040, 130), (17, 272, 64),
                                   (40, 4096, 100), (64, 512, 17), (65, 2048, 96), (130, 48, 257), (333, 1040, 1001),
                                   (1000, 640, 2050), (2100, 384, 1100), (3500, 272, 4100), (3500, 400, 4101), (7, 80, 14400), (8, 80, 14400),
                                   (16, 144, 14401)])
@pytest.mark.parametrize("dt", ALL_TYPES)
def test_int8_linear(lib, t, k, n, dt):
    g = gen_of(t + k + n)
    q, wq = codes(g, t, k), codes(g, n, k)
    s, ws = torch.rand(t, generator=g, device="cuda") * 0.01, torch.rand(n, generator=g, device="cuda") * 0.001
    for bias in (None, randn(g, n)):
        y = lib.int8_linear_forward(q, s, wq, ws, bias=bias, out_dtype=dt)
        assert y.shape == (t, n) and y.dtype == dt
        ref = int8_ref(q, s, wq, ws, bias)
        # the sum to fp32, the product of the scales, their product, the bias: 4 roundings
        mag = int8_ref(q, s, wq, ws, None).abs() + (0 if bias is None else bias.double().abs())
        within(y, ref, 4 * U * mag + half_step(dt) * ref.abs() * (1 + 8 * U) + 4 * U * half_step(dt) * mag + tiny(dt),
               f"bias={bias is not None}")


def test_int8_linear_extreme_codes_and_zero_scales(lib):
    """Every product 2^14 over the largest K: the INT32 sums reach 2^31 - 2^18; a zero scale
    gives zeros, a NaN scale only its own row or column."""
    k = 131072 - 16
    for t in (2, 70):
        q = torch.full((t, k), -128, dtype=torch.int8, device="cuda")
        wq = torch.full((5, k), -128, dtype=torch.int8, device="cuda")
        s = torch.ones(t, device="cuda")
        ws = torch.tensor([1.0, 0.0, 0.5, float("nan"), 2.0], device="cuda")
        s[1] = float("nan")
        y = lib.int8_linear_forward(q, s, wq, ws, out_dtype=torch.float32)
        assert torch.isnan(y[1]).all() and torch.isnan(y[:, 3]).all()
        keep = [i for i in range(t) if i != 1]
        total = float(k) * 2 ** 14
        within(y[keep][:, [0, 1, 2, 4]], torch.tensor([total, 0.0, total / 2, total * 2], device="cuda").double().expand(t - 1, 4),
               3 * U * 2 * total)


def test_int8_linear_same_bits_on_every_path(lib):
    """The same rows in batches that take the few-rows kernel, the split tiles and the whole
    tiles: exact sums, so equal bits."""
    g = gen_of(5)
    q, wq = codes(g, 3000, 1040), codes(g, 1500, 1040)
    s, ws = torch.rand(3000, generator=g, device="cuda"), torch.rand(1500, generator=g, device="cuda")
    full = lib.int8_linear_forward(q, s, wq, ws, out_dtype=torch.float32)
    for t in (1, 20, 64, 65, 200, 700):
        assert torch.equal(lib.int8_linear_forward(q[:t], s[:t], wq, ws, out_dtype=torch.float32), full[:t]), t


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("n,k", [(1, 16), (37, 272), (64, 2048)])
def test_quantize_int8_channel(lib, dt, n, k):
    g = gen_of(n + k)
    w = randn(g, n, k, std=0.02).to(dt)
    w[0] = 0
    q, s = lib.quantize_int8_channel(w)
    wf = w.float().cpu()
    sr = wf.abs().amax(1) / 127
    qr = torch.where(sr[:, None] > 0, wf / sr[:, None], torch.zeros(())).round().clamp(-127, 127).to(torch.int8)
    assert torch.equal(s.cpu(), sr) and torch.equal(q.cpu(), qr)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.quantize_int8_channel(w, flags=flags)
    assert flags.item() == 0
    w[n - 1, k - 1] = float("nan")
    lib.quantize_int8_channel(w, flags=flags)
    assert flags.item() == 1


# ------------------------------------------------------------------ gated projection
SWIGLU_SHAPES = [(1, 8, 8), (1, 2048, 1024), (5, 72, 40), (16, 1000, 136), (17, 64, 24), (33, 512, 200),
                 (64, 136, 72), (65, 72, 264), (130, 1000, 136), (300, 264, 520), (1030, 136, 1288),
                 (1300, 72, 4360), (3600, 3592, 264), (200, 2568, 2560),   # the large tiles: forward, dx, dw
                 (7, 72, 7200), (9, 72, 7200)]   # rows and tiles of a wide projection


def swiglu_inputs(t, h, i, dt, seed=0):
    g = gen_of(t + h + i + seed)
    return (randn(g, t, h).to(dt), randn(g, i, h, std=h ** -0.5).to(dt), randn(g, i, h, std=h ** -0.5).to(dt),
            randn(g, t, i).to(dt))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", SWIGLU_SHAPES)
def test_swiglu_linear_forward(lib, t, h, i, dt):
    x, wg, wu, _ = swiglu_inputs(t, h, i, dt)
    out, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
    assert torch.equal(lib.swiglu_linear_forward(x, wg, wu), out)
    xd, gd, ud = x.double(), wg.double(), wu.double()
    g, u = xd @ gd.T, xd @ ud.T
    dg, du = 2 * h * U * (xd.abs() @ gd.abs().T), 2 * h * U * (xd.abs() @ ud.abs().T)
    hs = half_step(dt)
    within(gu[:, 0], g, dg, "g")
    within(gu[:, 1], u, du, "u")
    sig = torch.sigmoid(g)
    ref = g * sig * u
    # |silu'| < 1.1; e^-g through exp2: (|g| + 4) roundings, then 4 more operations
    tol = 1.1 * dg * (u.abs() + du) + (g * sig).abs() * du + (g.abs() + 8) * 2 * U * ref.abs()
    within(out, ref, tol + hs * (ref.abs() + tol) + tiny(dt), "h")


def swiglu_grads(dh, x, wg, wu, g, u):
    sig = torch.sigmoid(g)
    dg = dh * u * sig * (1 + g * (1 - sig))
    du = dh * g * sig
    return dg, du, dg @ wg + du @ wu, dg.T @ x, du.T @ x


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("t,h,i", SWIGLU_SHAPES)
def test_swiglu_linear_backward(lib, t, h, i, dt):
    x, wg, wu, dh = swiglu_inputs(t, h, i, dt, 1)
    gu = torch.stack((randn(gen_of(7), t, i), randn(gen_of(8), t, i)), 1)
    dx, dwg, dwu = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
    xd, gd, ud, d = x.double(), wg.double(), wu.double(), dh.double()
    g, u = gu[:, 0].double(), gu[:, 1].double()
    dg, du, rx, rg, ru = swiglu_grads(d, xd, gd, ud, g, u)
    hs = half_step(dt)
    # dg, du: 8 fp32 operations on terms up to |dh u| (1 + |g|), then one rounding to dt
    eg = 32 * U * (d * u).abs() * (1 + g.abs()) + hs * dg.abs() * (1 + hs) + tiny(dt)
    eu = 32 * U * (d * g).abs() + hs * du.abs() * (1 + hs) + tiny(dt)
    ag, au = dg.abs() + eg, du.abs() + eu
    tol = eg @ gd.abs() + eu @ ud.abs() + 4 * i * U * (ag @ gd.abs() + au @ ud.abs())
    within(dx, rx, tol + hs * (rx.abs() + tol) + tiny(dt), "dx")
    for got, ref, e, a in ((dwg, rg, eg, ag), (dwu, ru, eu, au)):
        tol = e.T @ xd.abs() + 2 * t * U * (a.T @ xd.abs())
        within(got, ref, tol + hs * (ref.abs() + tol) + tiny(dt), "dw")


@pytest.mark.parametrize("dt", TYPES)
def test_swiglu_linear_gradient_against_differences(lib, dt):
    """<grad, d> against (L(p + e d) - L(p - e d)) / 2e of the 64-bit loss L = sum dh h, for a
    direction in each of x, w_gate and w_up.  The gradients carry roundings of dg, du and of
    the result: 2 half steps, taken at full size against the absolute values of the sum."""
    t, h, i = 70, 136, 72
    x, wg, wu, dh = swiglu_inputs(t, h, i, dt, 2)
    _, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
    grads = [v.double() for v in lib.swiglu_linear_backward(dh, x, wg, wu, gu)]
    p = [x.double(), wg.double(), wu.double()]
    d = dh.double()

    def loss(x, wg, wu):
        g = x @ wg.T
        return (d * g * torch.sigmoid(g) * (x @ wu.T)).sum()

    g, u = p[0] @ p[1].T, p[0] @ p[2].T
    ag, au = (d * u).abs() * (1 + g.abs()), (d * g).abs() + d.abs()
    mags = [ag @ p[1].abs() + au @ p[2].abs(), ag.T @ p[0].abs(), au.T @ p[0].abs()]
    e = 1e-5
    for j in range(3):
        v = torch.sign(randn(gen_of(j + 20), *p[j].shape)).double()
        plus, minus = [list(p), list(p)]
        plus[j], minus[j] = p[j] + e * v, p[j] - e * v
        diff = (loss(*plus) - loss(*minus)) / (2 * e)
        tol = 2.1 * half_step(dt) * mags[j].sum() + 1e-6 * mags[j].sum()
        assert abs((grads[j] * v).sum() - diff) <= tol


def test_swiglu_linear_no_tokens(lib):
    for dt in TYPES:
        x, wg, wu, dh = swiglu_inputs(0, 64, 40, dt)
        out, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
        assert out.shape == (0, 40) and gu.shape == (0, 2, 40)
        dx, dwg, dwu = lib.swiglu_linear_backward(dh, x, wg, wu, gu)
        assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()


def test_swiglu_linear_far_gates(lib):
    """Gate products far from zero: silu is 0 or the identity there, its gradient 0 or 1."""
    for dt in TYPES:
        x = torch.zeros(128, 8, dtype=dt, device="cuda")
        x[:, 0] = 1
        wg = torch.zeros(16, 8, dtype=dt, device="cuda")
        wg[:8, 0], wg[8:, 0] = -300.0, 300.0
        wu = torch.zeros(16, 8, dtype=dt, device="cuda")
        wu[:, 0] = 2.0
        out, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
        assert (out[:, :8] == 0).all() and (out[:, 8:] == 600).all()
        one = torch.ones_like(out)
        dx, dwg, dwu = lib.swiglu_linear_backward(one, x, wg, wu, gu)
        assert (dwg[:8, 0] == 0).all() and (dwg[8:, 0] == 256).all()
        assert (dwu[:8, 0] == 0).all() and (dwu[8:, 0] == 38400).all()
        assert torch.isfinite(dx).all()


# ------------------------------------------------------------------ block norms
GATES = ["none", "channel", "token", "element"]


def norm_inputs(t, c, dt, gate, seed=0):
    g = gen_of(t + c + seed)
    res, y = randn(g, t, c).to(dt), randn(g, t, c, std=0.5).to(dt)
    w_post, w_pre = (1 + randn(g, c, std=0.2)).to(dt), (1 + randn(g, c, std=0.2)).to(dt)
    shape = {"none": None, "channel": (c,), "token": (t, 1), "element": (t, c)}[gate]
    gv = None if shape is None else randn(g, *shape).to(dt)
    return dict(res=res, y=y, w_post=w_post, gate=gv, w_pre=w_pre)


def rstd64(v, eps):
    return ((v * v).mean(1, keepdim=True) + eps).rsqrt()


class Ref:
    """The operator in 64 bits, with the absolute values its rounding errors scale with."""

    def __init__(self, res, y=None, w_post=None, gate=None, alpha=1.0, w_pre=None, eps=1e-6):
        d = lambda v: None if v is None else v.double()
        self.res, y, self.w_post, gate, self.w_pre = d(res), d(y), d(w_post), d(gate), d(w_pre)
        self.alpha, self.gate = alpha, torch.ones((), dtype=torch.float64, device="cuda") if gate is None else gate
        self.has_y = y is not None
        self.r = self.res
        self.rabs = self.res.abs()
        if self.has_y:
            self.rs_y = rstd64(y, eps) if w_post is not None else torch.ones_like(y[:, :1])
            self.yh = y * self.rs_y
            self.p = self.yh * self.w_post if w_post is not None else y
            self.r = self.res + alpha * self.gate * self.p
            self.rabs = self.rabs + (alpha * self.gate * self.p).abs()
        self.rs = rstd64(self.r, eps)
        # relative error of rstd: 16 terms per thread, 10 tree steps, the mean, root and
        # quotient: 32 roundings, and the rounding of r itself
        self.e_rs = 32 * U + 48 * U * self.rabs.norm(dim=1, keepdim=True) / self.r.norm(dim=1, keepdim=True).clamp_min(1e-300)
        if w_pre is not None:
            self.n = self.r * self.rs * self.w_pre


def norm_check(lib, kw, alpha=0.75, eps=1e-6):
    dt = kw["res"].dtype
    r, n = lib.block_norm_forward(alpha=alpha, eps=eps, **kw)
    f = Ref(alpha=alpha, eps=eps, **kw)
    hs = half_step(dt)
    e_r = 48 * U * f.rabs
    within(r, f.r, e_r + hs * (f.r.abs() + e_r) + tiny(dt), "r")
    if kw.get("w_pre") is None:
        assert n is None
        return f
    e_n = (f.w_pre * f.rs).abs() * e_r * (1 + f.e_rs) + (f.e_rs + 4 * U) * f.n.abs()
    within(n, f.n, e_n + hs * (f.n.abs() + e_n) + tiny(dt), "n")
    return f


NORM_SHAPES = [(1, 1), (3, 7), (1, 2048), (5, 129), (4, 512), (7, 520), (9, 1024), (2, 1537), (6, 2048), (3, 4096),
               (2, 4104), (3, 7168), (2, 8191), (2, 16384), (600, 64), (1100, 2056), (1023, 1032),
               (1025, 1032)]


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,c", NORM_SHAPES)
def test_block_norm_forward(lib, t, c, dt):
    for gate in GATES:
        norm_check(lib, norm_inputs(t, c, dt, gate))


@pytest.mark.parametrize("dt", ALL_TYPES)
def test_block_norm_forward_parts(lib, dt):
    """Each part alone: norm before only, plain residual add, norm after only, no post norm."""
    for t, c in ((5, 520), (3, 7168), (4, 77)):
        kw = norm_inputs(t, c, dt, "token")
        for keep in (("res", "w_pre"), ("res", "y"), ("res", "y", "w_post"), ("res", "y", "w_pre"),
                     ("res", "y", "gate"), ("res", "y", "w_post", "w_pre")):
            f = norm_check(lib, {k: kw[k] for k in keep})
            if "y" not in keep:
                assert lib.block_norm_forward(kw["res"], w_pre=kw["w_pre"])[0] is kw["res"]


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,c", NORM_SHAPES)
def test_block_norm_codes(lib, t, c, dt):
    """q s stands for n to half a code step, plus the error of n and of the scale."""
    kw = norm_inputs(t, c, dt, "channel", 3)
    r, q, s = lib.block_norm_forward(alpha=0.5, quantize=True, **kw)
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    f = Ref(alpha=0.5, **kw)
    e_n = (f.w_pre * f.rs).abs() * 48 * U * f.rabs * (1 + f.e_rs) + (f.e_rs + 4 * U) * f.n.abs()
    amax, e_max = f.n.abs().amax(1), e_n.amax(1)
    within(s, amax / 127, e_max / 127 + 2 * U * amax)
    sd = s.double()[:, None]
    within(q.double() * sd, f.n, 0.5 * sd * (1 + 4 * U) + e_n + 2 * U * f.n.abs())
    assert (q.abs().amax(1) == 127).all()


def test_block_norm_zero_and_nonfinite_rows(lib):
    for dt in ALL_TYPES:
        x = randn(gen_of(1), 5, 264).to(dt)
        x[1] = 0
        x[2, 5] = float("nan")
        x[3, 7] = float("inf")
        w = torch.ones(264, dtype=dt, device="cuda")
        _, n = lib.block_norm_forward(x, w_pre=w)
        assert (n[1] == 0).all() and torch.isnan(n[2]).all() and torch.isnan(n[3, 7])
        _, q, s = lib.block_norm_forward(x, w_pre=w, quantize=True)
        assert s[1] == 0 and torch.isnan(s[2]) and torch.isnan(s[3]) and not q[1:4].any()
        ok = [0, 4]
        assert torch.equal(n[ok], lib.block_norm_forward(x[ok].contiguous(), w_pre=w)[1])


def test_block_norm_in_place_residual(lib):
    """The residual stream may be updated in place through the C entry point."""
    import ctypes
    L = lib._lib
    for t, c in ((3, 520), (4, 7168)):
        kw = norm_inputs(t, c, torch.bfloat16, "channel")
        want, n_want = lib.block_norm_forward(**kw)
        d = L._norm_desc(kw["res"], kw["y"], kw["w_post"], kw["gate"], 1.0, kw["w_pre"], 1e-6)
        n = torch.empty_like(want)
        rc = L.raw.block_norm_forward(ctypes.byref(d), kw["res"].data_ptr(), n.data_ptr(), None, None,
                                      torch.cuda.current_stream().cuda_stream)
        assert rc == 0 and torch.equal(kw["res"], want) and torch.equal(n, n_want)


def norm_grads(f, dr, dn, y, gate_kind):
    """64-bit gradients and, beside each, the absolute values its roundings scale with."""
    mean = lambda v: v.mean(1, keepdim=True)
    d = torch.zeros_like(f.res) if dr is None else dr.double()
    da = d.abs()
    out = {}
    if f.w_pre is not None:
        dnd = dn.double()
        rh, rha = f.r * f.rs, f.rabs * f.rs
        wd = f.w_pre * dnd
        d = d + f.rs * (wd - rh * mean(wd * rh))
        da = da + f.rs * (wd.abs() + rha * mean(wd.abs() * rha))
        out["w_pre"] = ((dnd * rh).sum(0), (dnd.abs() * rha).sum(0))
    out["res"] = (d, da)
    if not f.has_y:
        return out
    e, ea = f.alpha * d, abs(f.alpha) * da
    ep, epa = e * f.p, ea * f.p.abs()
    if gate_kind == "channel":
        out["gate"] = (ep.sum(0), epa.sum(0))
    elif gate_kind == "token":
        out["gate"] = (ep.sum(1, keepdim=True), epa.sum(1, keepdim=True))
    elif gate_kind == "element":
        out["gate"] = (ep, epa)
    dp, dpa = e * f.gate, ea * f.gate.abs()
    if f.w_post is None:
        out["y"] = (dp, dpa)
        return out
    wd, wda = f.w_post * dp, (f.w_post * dpa).abs()
    out["y"] = (f.rs_y * (wd - f.yh * mean(wd * f.yh)), f.rs_y * (wda + f.yh.abs() * mean(wda * f.yh.abs())))
    out["w_post"] = ((dp * f.yh).sum(0), (dpa * f.yh.abs()).sum(0))
    return out


def grad_check(lib, kw, gate, dr, dn, alpha=0.75):
    got = lib.block_norm_backward(dr, dn, alpha=alpha, **kw)
    f = Ref(alpha=alpha, **kw)
    ref = norm_grads(f, dr, dn, kw.get("y"), gate)
    # rstd twice in every term (32 + 48 |rabs| / |r| roundings each), sums over the row (32)
    # and over the rows (rows / groups + groups / 16 + 16 <= 64), a dozen products
    c = 3 * float((f.e_rs / U).max()) + 192
    for name in ("res", "y", "w_post", "w_pre", "gate"):
        if name not in ref:
            assert got[name] is None, name
            continue
        v, mag = ref[name]
        tol = c * U * mag
        if got[name].dtype != torch.float32:
            tol = tol + half_step(got[name].dtype) * (v.abs() + tol) + tiny(got[name].dtype)
        assert got[name].shape == v.shape, name
        within(got[name], v, tol + 1e-37, name)


@pytest.mark.parametrize("dt", ALL_TYPES)
@pytest.mark.parametrize("t,c", NORM_SHAPES)
def test_block_norm_backward(lib, t, c, dt):
    g = gen_of(t + 2 * c)
    dr, dn = randn(g, t, c).to(dt), randn(g, t, c).to(dt)
    for gate in GATES:
        grad_check(lib, norm_inputs(t, c, dt, gate, 5), gate, dr, dn)


@pytest.mark.parametrize("dt", ALL_TYPES)
def test_block_norm_backward_parts(lib, dt):
    for t, c in ((5, 520), (3, 7168), (4, 77)):
        kw = norm_inputs(t, c, dt, "channel", 6)
        g = gen_of(c)
        dr, dn = randn(g, t, c).to(dt), randn(g, t, c).to(dt)
        for keep in (("res", "w_pre"), ("res", "y"), ("res", "y", "w_post"), ("res", "y", "w_pre"),
                     ("res", "y", "gate"), ("res", "y", "w_post", "w_pre")):
            sub = {k: kw[k] for k in keep}
            gate = "channel" if "gate" in keep else "none"
            for r in (dr, None):
                grad_check(lib, sub, gate, r, dn if "w_pre" in keep else None)


def test_block_norm_gradient_against_differences(lib):
    """Directional derivatives of the 64-bit loss sum(dr r + dn n) against the fp32 gradients."""
    t, c, e = 6, 200, 1e-5
    for gate in GATES:
        kw = norm_inputs(t, c, torch.float32, gate, 9)
        g = gen_of(11)
        dr, dn = randn(g, t, c), randn(g, t, c)
        got = lib.block_norm_backward(dr, dn, alpha=0.75, **kw)
        f = Ref(alpha=0.75, **kw)
        mags = norm_grads(f, dr, dn, kw["y"], gate)

        def loss(**p):
            f = Ref(alpha=0.75, **p)
            return (dr.double() * f.r + dn.double() * f.n).sum()

        base = {k: None if v is None else v.double() for k, v in kw.items()}
        for name in base:
            if base[name] is None:
                continue
            v = torch.sign(randn(g, *base[name].shape)).double()
            diff = (loss(**{**base, name: base[name] + e * v}) - loss(**{**base, name: base[name] - e * v})) / (2 * e)
            total = mags[name][1].sum()
            # the fp32 gradient's roundings, and the differences' own: e^2 and 2^-53 / e
            assert abs((got[name].double() * v).sum() - diff) <= (512 * U + 1e-7) * total, name


def test_block_norm_no_rows(lib):
    for dt in ALL_TYPES:
        kw = norm_inputs(0, 40, dt, "channel")
        r, n = lib.block_norm_forward(**kw)
        assert r.shape == n.shape == (0, 40)
        got = lib.block_norm_backward(torch.empty_like(r), torch.empty_like(r), **kw)
        for name in ("w_post", "w_pre", "gate"):
            assert got[name].shape == (40,) and not got[name].any()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("t", [1, 16, 100, 700])
@pytest.mark.parametrize("dt", TYPES)
def test_int8_block(lib, t, dt):
    """Residual stream -> norm with INT8 codes -> INT8 product -> norm, gate, residual scale;
    each stage against 64 bits on the previous stage's own output."""
    c, n = 1040, 1040
    g = gen_of(t)
    res = randn(g, t, c).to(dt)
    w_pre, w_post = (1 + randn(g, c, std=0.1)).to(dt), (1 + randn(g, n, std=0.1)).to(dt)
    wq, ws = lib.quantize_int8_channel(randn(g, n, c, std=0.02))
    gate = torch.sigmoid(randn(g, t, 1)).to(dt)
    _, q, s = lib.block_norm_forward(res, w_pre=w_pre, quantize=True)
    y = lib.int8_linear_forward(q, s, wq, ws, out_dtype=dt)
    ref = int8_ref(q, s, wq, ws, None)
    within(y, ref, (3 * U + half_step(dt) * (1 + 4 * U)) * ref.abs() + tiny(dt), "y")
    norm_check(lib, dict(res=res, y=y, w_post=w_post, gate=gate), alpha=0.5)
    # against the unquantised block: a code is off by at most half a step of amax / 127 in x
    # and in w, independent over k: |y - y0| <= sum_k (|x| sw / 2 + |w| sx / 2 + sx sw / 4)
    f = Ref(res=res, w_pre=w_pre)
    wd = wq.double() * ws.double()[:, None]
    y0 = f.n @ wd.T
    tol = (0.5 * s.double()[:, None] * (1 + 1e-4)) * wd.abs().sum(1) + half_step(dt) * 1.01 * y0.abs() + 1e-4 * (f.n.abs() @ wd.abs().T)
    within(y, y0, tol * 1.01 + tiny(dt), "block")


@pytest.mark.parametrize("dt", TYPES)
def test_training_block(lib, dt):
    """Norm -> gated projection -> down projection -> norm, gate, residual scale, with every
    gradient, against 64-bit automatic differentiation.  Each stored tensor on the way (n, h,
    y, dy, dh, dg, du, dn and the result) is rounded once: at most 9 half steps, and
    as much again for what the norms' Jacobians (norm at most 2 here) make of them."""
    t, c, i = 130, 264, 520
    g = gen_of(3)
    res = randn(g, t, c).to(dt)
    w_pre, w_post = (1 + randn(g, c, std=0.1)).to(dt), (1 + randn(g, c, std=0.1)).to(dt)
    wg, wu = randn(g, i, c, std=c ** -0.5).to(dt), randn(g, i, c, std=c ** -0.5).to(dt)
    wd = randn(g, c, i, std=i ** -0.5).to(dt)
    gate = torch.sigmoid(randn(g, c)).to(dt)
    dr = randn(g, t, c).to(dt)
    post = dict(w_post=w_post, gate=gate, alpha=0.5)
    _, n = lib.block_norm_forward(res, w_pre=w_pre)
    h, gu = lib.swiglu_linear_forward(n, wg, wu, save=True)
    y = (h.float() @ wd.float().T).to(dt)
    r, _ = lib.block_norm_forward(res, y=y, **post)
    g2 = lib.block_norm_backward(dr, None, res, y=y, **post)
    dh = (g2["y"].float() @ wd.float()).to(dt)
    dn, dwg, dwu = lib.swiglu_linear_backward(dh, n, wg, wu, gu)
    g1 = lib.block_norm_backward(g2["res"], dn, res, w_pre=w_pre)

    leaves = [v.double().requires_grad_() for v in (res, w_pre, wg, wu, w_post, gate)]
    R, A, G, W, B, K = leaves
    nn = R * rstd64(R, 1e-6) * A
    gg = nn @ G.T
    yy = (gg * torch.sigmoid(gg) * (nn @ W.T)) @ wd.double().T
    rr = R + 0.5 * K * (yy * rstd64(yy, 1e-6) * B)
    rr.backward(dr.double())
    tol = 18 * half_step(dt)
    for got, ref in ((r, rr.detach()), (g1["res"], R.grad), (g1["w_pre"], A.grad), (dwg, G.grad), (dwu, W.grad),
                     (g2["w_post"], B.grad), (g2["gate"], K.grad)):
        assert (got.double() - ref).norm() <= tol * ref.norm()


def test_results_repeat_bit_for_bit(lib):
    for dt in TYPES:
        x, wg, wu, dh = swiglu_inputs(130, 1000, 136, dt)
        _, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
        a, b = (lib.swiglu_linear_backward(dh, x, wg, wu, gu) for _ in range(2))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        kw = norm_inputs(1100, 520, dt, "channel")
        a, b = (lib.block_norm_backward(kw["y"], kw["res"], **kw) for _ in range(2))
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_on_a_side_stream(lib):
    """Calls on a stream other than the default one, ordered after their inputs there."""
    s = torch.cuda.Stream()
    x, wg, wu, dh = swiglu_inputs(130, 264, 136, torch.bfloat16)
    ref = lib.swiglu_linear_forward(x, wg, wu, save=True)
    ref_b = lib.swiglu_linear_backward(dh, x, wg, wu, ref[1])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        x2 = (x.float() * 1).to(x.dtype)
        got = lib.swiglu_linear_forward(x2, wg, wu, save=True)
        got_b = lib.swiglu_linear_backward(dh, x2, wg, wu, got[1])
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref + ref_b, got + got_b))


def test_captured_graphs(lib):
    """A training block and an INT8 block captured as two graphs, replayed in turn with eager
    work and new inputs between; every replay against the eager result."""
    dt = torch.bfloat16
    x, wg, wu, dh = swiglu_inputs(130, 1000, 136, dt)
    kw = norm_inputs(130, 1000, dt, "channel")
    wq, ws = lib.quantize_int8_channel(randn(gen_of(1), 1000, 1008, std=0.02))
    big = randn(gen_of(2), 130, 1008).to(dt)
    w_pre = torch.ones(1008, dtype=dt, device="cuda")

    def train():
        h, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
        g = lib.block_norm_backward(kw["y"], kw["res"], **kw)
        return (h,) + lib.swiglu_linear_backward(dh, x, wg, wu, gu) + tuple(g[k] for k in sorted(g))

    def serve():
        _, q, s = lib.block_norm_forward(big, w_pre=w_pre, quantize=True)
        return q, s, lib.int8_linear_forward(q, s, wq, ws)

    graphs = []
    for f in (train, serve):
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            f()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = f()
        graphs.append((f, g, out))
    for rep in range(4):
        gen = gen_of(100 + rep)
        x.copy_(randn(gen, *x.shape).to(dt))
        big.copy_(randn(gen, *big.shape).to(dt))
        kw["res"].copy_(randn(gen, *kw["res"].shape).to(dt))
        for _, g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for f, _, out in graphs:
            want = f()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(out, want)), rep


def test_binding_refusals(lib):
    bf = torch.bfloat16
    x = torch.zeros(4, 64, dtype=bf, device="cuda")
    w = torch.zeros(8, 64, dtype=bf, device="cuda")
    with pytest.raises(TypeError):
        lib.swiglu_linear_forward(x.float(), w, w)
    with pytest.raises(TypeError):
        lib.swiglu_linear_forward(x, w.half(), w)
    with pytest.raises(ValueError):
        lib.swiglu_linear_forward(x, w, w[:7].contiguous())
    with pytest.raises(ValueError):
        lib.swiglu_linear_forward(x.t(), w, w)
    with pytest.raises(ValueError):
        lib.swiglu_linear_backward(x, x, w, w, x)
    with pytest.raises(lib.Q4Error):
        lib.swiglu_linear_forward(torch.zeros(4, 12, dtype=bf, device="cuda"), torch.zeros(8, 12, dtype=bf, device="cuda"),
                                  torch.zeros(8, 12, dtype=bf, device="cuda"))
    q = torch.zeros(4, 64, dtype=torch.int8, device="cuda")
    s = torch.zeros(4, device="cuda")
    with pytest.raises(ValueError):
        lib.int8_linear_forward(q, s[:3].contiguous(), q, s)
    with pytest.raises(TypeError):
        lib.int8_linear_forward(q, s.double(), q, s)
    with pytest.raises(TypeError):
        lib.int8_linear_forward(q, s, q, s, out_dtype=torch.int32)
    with pytest.raises(lib.Q4Error):
        lib.int8_linear_forward(q[:, :8].contiguous(), s, q[:, :8].contiguous(), s)
    wv = torch.ones(64, dtype=bf, device="cuda")
    with pytest.raises(ValueError):
        lib.block_norm_forward(x)
    with pytest.raises(ValueError):
        lib.block_norm_forward(x, w_post=wv, w_pre=wv)
    with pytest.raises(ValueError):
        lib.block_norm_forward(x, y=x, gate=wv[:5].contiguous())
    with pytest.raises(TypeError):
        lib.block_norm_forward(x, w_pre=wv.float())
    with pytest.raises(ValueError):
        lib.block_norm_backward(x, None, x, w_pre=wv)
    with pytest.raises(lib.Q4Error):
        lib.block_norm_forward(x, w_pre=wv, eps=0.0)


# ------------------------------------------------------------------ buffers
class Guarded:
    """Buffers between filled guard regions; check() finds a write outside any of them."""
    PAD = 4096

    def __init__(self):
        self.bufs = []

    def new(self, *shape, dtype):
        n = 1
        for d in shape:
            n *= d
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((nbytes + 2 * self.PAD,), 0xA5, dtype=torch.uint8, device="cuda")
        self.bufs.append((raw, nbytes))
        return raw[self.PAD:self.PAD + nbytes].view(dtype).view(*shape)

    def check(self):
        for raw, nbytes in self.bufs:
            assert (raw[:self.PAD] == 0xA5).all() and (raw[self.PAD + nbytes:] == 0xA5).all()


def ptr(t):
    return None if t is None else t.data_ptr()


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("t,k,n", [(5, 48, 33), (70, 1040, 1001), (333, 272, 130), (3500, 80, 4101)])
def test_int8_linear_writes_only_its_output(lib, t, k, n):
    r = lib._lib.raw
    g = gen_of(t)
    q, wq = codes(g, t, k), codes(g, n, k)
    s, ws = torch.rand(t, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    for dt in ALL_TYPES:
        b = Guarded()
        y = b.new(t, n, dtype=dt)
        nbytes = r.int8_linear_workspace_bytes(t, k, n)
        work = b.new(nbytes, dtype=torch.uint8) if nbytes else None
        assert r.int8_linear_forward(ptr(q), ptr(s), t, k, ptr(wq), ptr(ws), n, None, lib._lib._DT[dt], ptr(y),
                                     ptr(work), nbytes, stream()) == 0
        b.check()
        assert torch.equal(y, lib.int8_linear_forward(q, s, wq, ws, out_dtype=dt))


@pytest.mark.parametrize("t,h,i", [(5, 40, 24), (70, 1000, 136), (300, 264, 520), (1300, 72, 4360), (200, 2568, 2560)])
def test_swiglu_linear_writes_only_its_outputs(lib, t, h, i):
    r, dt = lib._lib.raw, torch.bfloat16
    code = lib._lib._DT[dt]
    x, wg, wu, dh = swiglu_inputs(t, h, i, dt, 4)
    b = Guarded()
    out, gu = b.new(t, i, dtype=dt), b.new(t, 2, i, dtype=torch.float32)
    nbytes = r.swiglu_linear_workspace_bytes(t, h, i)
    work = b.new(nbytes, dtype=torch.uint8) if nbytes else None
    assert r.swiglu_linear_forward(ptr(x), ptr(wg), ptr(wu), t, h, i, code, ptr(out), ptr(gu), ptr(work), nbytes,
                                   stream()) == 0
    dx, dwg, dwu = b.new(t, h, dtype=dt), b.new(i, h, dtype=dt), b.new(i, h, dtype=dt)
    nbytes = r.swiglu_linear_backward_workspace_bytes(t, h, i)
    work = b.new(nbytes, dtype=torch.uint8)
    assert r.swiglu_linear_backward(ptr(dh), ptr(x), ptr(wg), ptr(wu), ptr(gu), t, h, i, code, ptr(dx), ptr(dwg),
                                    ptr(dwu), ptr(work), nbytes, stream()) == 0
    b.check()
    ref, gu_ref = lib.swiglu_linear_forward(x, wg, wu, save=True)
    assert torch.equal(out, ref) and torch.equal(gu, gu_ref)
    for a, c in zip((dx, dwg, dwu), lib.swiglu_linear_backward(dh, x, wg, wu, gu)):
        assert torch.equal(a, c)


@pytest.mark.parametrize("t,c", [(3, 7), (5, 1000), (70, 1001), (33, 4104), (9, 9000)])
def test_block_norm_writes_only_its_outputs(lib, t, c):
    import ctypes
    L = lib._lib
    for dt in ALL_TYPES:
        kw = norm_inputs(t, c, dt, "channel", 8)
        d = L._norm_desc(kw["res"], kw["y"], kw["w_post"], kw["gate"], 0.5, kw["w_pre"], 1e-6)
        b = Guarded()
        rr, n, q, s = b.new(t, c, dtype=dt), b.new(t, c, dtype=dt), b.new(t, c, dtype=torch.int8), b.new(t, dtype=torch.float32)
        assert L.raw.block_norm_forward(ctypes.byref(d), ptr(rr), ptr(n), None, None, stream()) == 0
        assert L.raw.block_norm_forward(ctypes.byref(d), ptr(rr), None, ptr(q), ptr(s), stream()) == 0
        dres, dy = b.new(t, c, dtype=dt), b.new(t, c, dtype=dt)
        dwo, dwi, dg = (b.new(c, dtype=torch.float32) for _ in range(3))
        nbytes = L.raw.block_norm_workspace_bytes(ctypes.byref(d))
        work = b.new(nbytes, dtype=torch.uint8)
        assert L.raw.block_norm_backward(ctypes.byref(d), ptr(kw["y"]), ptr(kw["res"]), ptr(dres), ptr(dy), ptr(dwo),
                                         ptr(dg), ptr(dwi), ptr(work), nbytes, stream()) == 0
        b.check()
        got = lib.block_norm_backward(kw["y"], kw["res"], alpha=0.5, **kw)
        for a, name in ((dres, "res"), (dy, "y"), (dwo, "w_post"), (dwi, "w_pre"), (dg, "gate")):
            assert torch.equal(a, got[name]), name


def test_two_streams_at_once(lib):
    """The same operators on two streams with work of their own in flight together."""
    x, wg, wu, dh = swiglu_inputs(300, 1000, 520, torch.bfloat16, 6)
    kw = norm_inputs(700, 2048, torch.bfloat16, "channel")

    def work():
        h, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
        g = lib.block_norm_backward(kw["y"], kw["res"], **kw)
        return (h,) + lib.swiglu_linear_backward(dh, x, wg, wu, gu) + tuple(g[k] for k in sorted(g))

    ref = work()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(work())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))


def test_offsets_past_32_bits(lib):
    """Outputs of more than 2^31 elements: the last rows against a call on them alone."""
    bf = torch.bfloat16
    g = gen_of(12)
    t, n, tail = 200000, 12288, 100
    q, wq = codes(g, t, 16), codes(g, n, 16)
    s, ws = torch.rand(t, generator=g, device="cuda"), torch.rand(n, generator=g, device="cuda")
    y = lib.int8_linear_forward(q, s, wq, ws)
    assert torch.equal(y[-tail:], lib.int8_linear_forward(q[-tail:].contiguous(), s[-tail:].contiguous(), wq, ws))
    del y
    t, h, i = 150000, 8, 8192
    x, wg, wu = randn(g, t, h).to(bf), randn(g, i, h).to(bf), randn(g, i, h).to(bf)
    out, gu = lib.swiglu_linear_forward(x, wg, wu, save=True)
    xt = x[-tail:].double()
    gd, ud = xt @ wg.double().T, xt @ wu.double().T
    within(gu[-tail:, 0], gd, 2 * h * U * (xt.abs() @ wg.double().abs().T), "g")
    within(gu[-tail:, 1], ud, 2 * h * U * (xt.abs() @ wu.double().abs().T), "u")
    dx, dwg, dwu = lib.swiglu_linear_backward(out, x, wg, wu, gu)
    dh = out[-tail:].double()
    dg, du, rx, _, _ = swiglu_grads(dh, xt, wg.double(), wu.double(), gu[-tail:, 0].double(), gu[-tail:, 1].double())
    hs = half_step(bf)
    ag, au = dg.abs() @ wg.double().abs(), du.abs() @ wu.double().abs()
    u_abs, g_abs = gu[-tail:, 1].double().abs(), gu[-tail:, 0].double().abs()
    # dg, du: 32 fp32 roundings on terms up to |dh u| (1 + |g|), one to bf16; the sums; the result
    tol = (1 + 1e-3) * hs * (ag + au) + 32 * U * (((dh.abs() * u_abs * (1 + g_abs)) @ wg.double().abs())
                                                  + ((dh.abs() * g_abs) @ wu.double().abs())) \
        + 5 * i * U * (ag + au)
    within(dx[-tail:], rx, tol + hs * (rx.abs() + tol), "dx")
    del out, gu, dx, dwg, dwu
    t, c = 300000, 8192
    res = torch.zeros(t, c, dtype=bf, device="cuda")
    res[-tail:] = randn(g, tail, c).to(bf)
    w = torch.ones(c, dtype=bf, device="cuda")
    last = res[-tail:].contiguous()
    want, n_want = lib.block_norm_forward(last, y=last, w_pre=w, w_post=w)
    got, n_got = lib.block_norm_forward(res, y=res, w_pre=w, w_post=w)
    assert torch.equal(got[-tail:], want) and torch.equal(n_got[-tail:], n_want)
    gb = lib.block_norm_backward(got, n_got, res, y=res, w_pre=w, w_post=w)
    ref = lib.block_norm_backward(want, n_want, last, y=last, w_pre=w, w_post=w)
    assert torch.equal(gb["res"][-tail:], ref["res"]) and torch.equal(gb["y"][-tail:], ref["y"])
