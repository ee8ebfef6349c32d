"""Refusals of the token order and the e4m3 products: every bad call is turned down on the host,
before any launch (CPU only)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from int4_group_quantized_g128_amd import _lib
    return _lib


FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)
BIG = 1 << 60


def test_dispatch_validation(L):
    def f(x=FAKE, dt=2, t=5000, h=64, ids=FAKE, k=2, first=0, e=8, out=FAKE, q=None, s=None, offsets=FAKE, perm=FAKE,
          inv=FAKE, work=FAKE, nbytes=BIG):
        return L.raw.moe_dispatch_forward(x, dt, t, h, ids, k, first, e, out, q, s, offsets, perm, inv, work, nbytes,
                                          None)

    assert f(dt=3) == L.Q4_ERR_DTYPE
    for bad in (dict(t=-1), dict(t=1 << 23), dict(h=0), dict(h=(1 << 20) + 1), dict(k=0), dict(k=4097),
                dict(t=1 << 22, k=16), dict(e=0), dict(e=4097), dict(first=-1),
                dict(h=72, out=None, q=FAKE, s=FAKE)):
        assert f(**bad) == L.Q4_ERR_SHAPE, bad
    for bad in ("x", "ids", "out", "offsets", "perm", "inv", "work"):
        assert f(**{bad: None}) == L.Q4_ERR_NULL, bad
    for bad in (dict(q=FAKE), dict(q=FAKE, s=FAKE), dict(out=None, q=FAKE), dict(out=None, s=FAKE)):
        assert f(**bad) == L.Q4_ERR_NULL, bad
    for bad in ("x", "ids", "out", "offsets", "perm", "inv", "work"):
        assert f(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    for bad in ("q", "s"):
        assert f(**{"out": None, "q": FAKE, "s": FAKE, bad: ODD}) == L.Q4_ERR_ALIGN, bad
    need = L.raw.moe_dispatch_workspace_bytes(5000, 2, 8)
    assert need > 0 and f(nbytes=need - 1) == L.Q4_ERR_WORKSPACE
    assert L.raw.moe_dispatch_workspace_bytes(64, 8, 256) == 0   # one launch
    assert L.raw.moe_dispatch_workspace_bytes(-1, 8, 256) == 0
    assert L.raw.moe_dispatch_workspace_bytes(5000, 2, 5000) == 0


def test_combine_validation(L):
    def back(dxp=FAKE, dt=2, t=5, h=64, inv=FAKE, k=2, dx=FAKE):
        return L.raw.moe_dispatch_backward(dxp, dt, t, h, inv, k, dx, None)

    def f(y=FAKE, dt=2, t=5, h=64, inv=FAKE, w=FAKE, add=None, k=2, out=FAKE):
        return L.raw.moe_combine_forward(y, dt, t, h, inv, w, add, k, out, None)

    def b(dout=FAKE, y=FAKE, dt=2, t=5, h=64, inv=FAKE, w=FAKE, k=2, dy=FAKE, dw=FAKE):
        return L.raw.moe_combine_backward(dout, y, dt, t, h, inv, w, k, dy, dw, None)

    for call in (back, f, b):
        assert call(dt=-1) == L.Q4_ERR_DTYPE
        for bad in (dict(t=-1), dict(t=1 << 23), dict(h=0), dict(k=0), dict(k=4097), dict(t=1 << 22, k=16)):
            assert call(**bad) == L.Q4_ERR_SHAPE, bad
        assert call(t=0, inv=None) == L.Q4_OK
    for call, names in ((back, ("dxp", "inv", "dx")), (f, ("y", "inv", "out")), (b, ("dout", "y", "inv", "dy"))):
        for bad in names:
            assert call(**{bad: None}) == L.Q4_ERR_NULL, bad
            assert call(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    assert f(w=ODD) == L.Q4_ERR_ALIGN and f(add=ODD) == L.Q4_ERR_ALIGN
    assert b(dw=None) == L.Q4_ERR_NULL and b(w=None) == L.Q4_ERR_NULL
    assert b(w=ODD) == L.Q4_ERR_ALIGN and b(dw=ODD) == L.Q4_ERR_ALIGN


def test_token_order_limits(L):
    """Calls whose launches would not fit, and experts that no id can name."""
    slots = (1 << 26) - 4
    def d(t, h, k, first=0, e=8):
        return L.raw.moe_dispatch_forward(FAKE, 2, t, h, FAKE, k, first, e, FAKE, None, None, FAKE, FAKE, FAKE, FAKE, 0,
                                          None)
    calls = (d, lambda t, h, k: L.raw.moe_dispatch_backward(None, 2, t, h, None, k, None, None),
             lambda t, h, k: L.raw.moe_combine_forward(None, 0, t, h, None, None, None, k, None, None),
             lambda t, h, k: L.raw.moe_combine_backward(None, None, 1, t, h, None, None, k, None, None, None))
    for call in calls:
        assert call(slots // 12 + 1, 64, 12) == L.Q4_ERR_SHAPE      # t k = 2^26 - 4 + 12 - ..
        assert call(slots // 12, 64, 12) != L.Q4_ERR_SHAPE
        assert call(1 << 22, 4096, 1) == L.Q4_ERR_SHAPE             # t ceil(h / 256) = 2^26
        assert call(1 << 22, 3840, 1) != L.Q4_ERR_SHAPE
    assert d(5, 64, 2, first=2 ** 31 - 8) == L.Q4_ERR_SHAPE         # experts to 2^31
    assert d(5000, 64, 2, first=2 ** 31 - 9) == L.Q4_ERR_WORKSPACE
    assert L.raw.moe_dispatch_workspace_bytes(slots // 12 + 1, 12, 8) == 0


def test_quantize_fp8_validation(L):
    def f(x=FAKE, dt=2, t=5, k=64, gated=0, offsets=None, e=1, q=FAKE, s=FAKE, qc=None, sc=None):
        return L.raw.quantize_fp8_tokens(x, dt, t, k, gated, offsets, e, q, s, qc, sc, None)

    def w(w=FAKE, dt=0, e=1, n=64, k=64, q=FAKE, s=FAKE):
        return L.raw.quantize_fp8_blocks(w, dt, e, n, k, q, s, None)

    assert f(dt=3) == L.Q4_ERR_DTYPE and w(dt=3) == L.Q4_ERR_DTYPE
    for bad in (dict(t=-1), dict(t=1 << 23), dict(k=0), dict(k=24), dict(k=(1 << 20) + 16),
                dict(k=(1 << 19) + 16, gated=1), dict(offsets=FAKE, e=0), dict(offsets=FAKE, e=4097)):
        assert f(**bad) == L.Q4_ERR_SHAPE, bad
    for bad in (dict(x=None), dict(q=None), dict(s=None), dict(q=None, s=None), dict(qc=FAKE), dict(sc=FAKE)):
        assert f(**bad) == L.Q4_ERR_NULL, bad
    for bad in (dict(x=ODD), dict(q=ODD), dict(s=ODD), dict(qc=ODD, sc=FAKE), dict(qc=FAKE, sc=ODD), dict(offsets=ODD)):
        assert f(**bad) == L.Q4_ERR_ALIGN, bad
    assert f(gated=1, qc=FAKE, sc=FAKE) == L.Q4_ERR_UNSUPPORTED
    assert f(t=0, x=None, q=None, s=None) == L.Q4_OK
    for bad in (dict(e=0), dict(e=4097), dict(n=0), dict(n=(1 << 20) + 1), dict(k=8), dict(k=(1 << 20) + 16),
                dict(e=4096, n=1 << 20)):
        assert w(**bad) == L.Q4_ERR_SHAPE, bad
    for bad in ("w", "q", "s"):
        assert w(**{bad: None}) == L.Q4_ERR_NULL and w(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad


def test_fp8_linear_validation(L):
    def f(q=FAKE, s=FAKE, t=70, k=4096, wq=FAKE, ws=FAKE, n=64, offsets=None, e=1, dt=2, y=FAKE, work=FAKE,
          nbytes=BIG):
        return L.raw.fp8_linear_forward(q, s, t, k, wq, ws, n, offsets, e, dt, y, work, nbytes, None)

    def b(dy=FAKE, dt=2, t=70, k=4096, n=64, xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, offsets=None, e=1, dx=FAKE, dw=FAKE,
          work=FAKE, nbytes=BIG):
        return L.raw.fp8_linear_backward(dy, dt, t, k, n, xq, xs, wq, ws, offsets, e, dx, dw, work, nbytes, None)

    for call in (f, b):
        assert call(dt=0) == L.Q4_ERR_DTYPE and call(dt=3) == L.Q4_ERR_DTYPE
        for bad in (dict(t=-1), dict(t=1 << 23), dict(k=0), dict(k=24), dict(k=(1 << 20) + 16), dict(n=0),
                    dict(n=(1 << 20) + 16), dict(e=2), dict(offsets=FAKE, e=0), dict(offsets=FAKE, e=4097)):
            assert call(**bad) == L.Q4_ERR_SHAPE, bad
        for bad in ("wq", "ws", "work"):
            assert call(**{bad: None}) == L.Q4_ERR_NULL, bad
        for bad in ("wq", "ws", "offsets", "work"):
            assert call(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    assert b(n=24) == L.Q4_ERR_SHAPE and b(n=8) == L.Q4_ERR_SHAPE and b(n=1001) == L.Q4_ERR_SHAPE
    for bad in ("q", "s", "y"):
        assert f(**{bad: None}) == L.Q4_ERR_NULL and f(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    for bad in ("dy", "xq", "xs", "dx", "dw"):
        assert b(**{bad: None}) == L.Q4_ERR_NULL and b(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    need = L.raw.fp8_linear_workspace_bytes(70, 4096, 64, 1, 0)
    assert need > 0 and f(nbytes=need - 1) == L.Q4_ERR_WORKSPACE
    need = L.raw.fp8_linear_backward_workspace_bytes(70, 4096, 64, 1, 0)
    assert need > 0 and b(nbytes=need - 1) == L.Q4_ERR_WORKSPACE
    assert L.raw.fp8_linear_workspace_bytes(70, 24, 64, 1, 0) == 0
    assert L.raw.fp8_linear_backward_workspace_bytes(70, 64, 24, 1, 0) == 0
    assert f(t=0, q=None, y=None, work=None, nbytes=0) == L.Q4_OK
    assert b(t=0, dw=None) == L.Q4_ERR_NULL      # zero tokens still write the weights' gradient


def test_binding_refuses(L):
    z, f8 = torch.zeros, torch.float8_e4m3fn
    ids = z(4, 2, dtype=torch.int32)
    for call in (lambda: L.moe_dispatch_forward(z(4, 64), ids, 8),
                 lambda: L.moe_dispatch_backward(z(8, 64), ids),
                 lambda: L.moe_combine_forward(z(8, 64), ids),
                 lambda: L.moe_combine_backward(z(4, 64), z(8, 64), ids),
                 lambda: L.quantize_fp8_tokens(z(4, 64)),
                 lambda: L.quantize_fp8_blocks(z(4, 64)),
                 lambda: L.fp8_linear_forward(z(4, 64).to(f8), z(1, 4), z(8, 64).to(f8), z(1, 1)),
                 lambda: L.fp8_linear_backward(z(4, 8).half(), z(4, 64).to(f8), z(1, 64), z(8, 64).to(f8), z(1, 1))):
        with pytest.raises(ValueError):
            call()
