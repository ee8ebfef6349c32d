"""Refusals of the dense operators (INT8 linear, gated projection, block norms): every bad
call is turned down on the host, before any launch (CPU only)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def L():
    from int4_group_quantized_g128_amd import _lib
    return _lib


FAKE = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4104)


def test_quantize_int8_channel_validation(L):
    f = L.raw.quantize_int8_channel
    assert f(FAKE, 9, 4, 64, FAKE, FAKE, None, None) == L.Q4_ERR_DTYPE
    for n, k in ((0, 64), (4, 0), (4, 24), (4, 131072), ((1 << 20) + 1, 64), (-1, 64), (4, -16)):
        assert f(FAKE, L.Q4_F32, n, k, FAKE, FAKE, None, None) == L.Q4_ERR_SHAPE, (n, k)
    assert f(None, L.Q4_F32, 4, 64, FAKE, FAKE, None, None) == L.Q4_ERR_NULL
    assert f(FAKE, L.Q4_F32, 4, 64, FAKE, None, None, None) == L.Q4_ERR_NULL
    assert f(ODD, L.Q4_F32, 4, 64, FAKE, FAKE, None, None) == L.Q4_ERR_ALIGN


def test_int8_linear_validation(L):
    def f(t=70, k=4096, n=64, q=FAKE, s=FAKE, wq=FAKE, ws=FAKE, bias=None, dt=2, y=FAKE, work=FAKE, nbytes=1 << 40):
        return L.raw.int8_linear_forward(q, s, t, k, wq, ws, n, bias, dt, y, work, nbytes, None)

    assert f(dt=3) == L.Q4_ERR_DTYPE and f(dt=-1) == L.Q4_ERR_DTYPE
    for bad in (dict(t=-1), dict(t=(1 << 24) + 1), dict(k=0), dict(k=40), dict(k=131072), dict(n=0),
                dict(n=(1 << 20) + 1)):
        assert f(**bad) == L.Q4_ERR_SHAPE, bad
    for bad in ("q", "s", "wq", "ws", "y", "work"):
        assert f(**{bad: None}) == L.Q4_ERR_NULL, bad
    for bad in ("q", "s", "wq", "ws", "y", "bias", "work"):
        assert f(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    need = L.raw.int8_linear_workspace_bytes(70, 4096, 64)
    assert need > 0
    assert f(nbytes=need - 1) == L.Q4_ERR_WORKSPACE
    assert L.raw.int8_linear_workspace_bytes(70, 40, 64) == 0
    assert f(t=0, q=None, y=None, work=None, nbytes=0) == L.Q4_OK


def test_swiglu_linear_validation(L):
    def f(t=70, h=4096, i=64, dt=2, x=FAKE, wg=FAKE, wu=FAKE, out=FAKE, gu=None, work=FAKE, nbytes=1 << 40):
        return L.raw.swiglu_linear_forward(x, wg, wu, t, h, i, dt, out, gu, work, nbytes, None)

    def b(t=70, h=4096, i=64, dt=2, dh=FAKE, x=FAKE, wg=FAKE, wu=FAKE, gu=FAKE, dx=FAKE, dwg=FAKE, dwu=FAKE,
          work=FAKE, nbytes=1 << 40):
        return L.raw.swiglu_linear_backward(dh, x, wg, wu, gu, t, h, i, dt, dx, dwg, dwu, work, nbytes, None)

    for call in (f, b):
        assert call(dt=0) == L.Q4_ERR_DTYPE
        for bad in (dict(t=-1), dict(t=(1 << 24) + 1), dict(h=0), dict(h=12), dict(i=0), dict(i=20),
                    dict(h=(1 << 20) + 8), dict(i=(1 << 20) + 8)):
            assert call(**bad) == L.Q4_ERR_SHAPE, bad
        for bad in ("x", "wg", "wu", "work"):
            assert call(**{bad: None}) == L.Q4_ERR_NULL, bad
        for bad in ("x", "wg", "wu", "gu", "work"):
            assert call(**{bad: ODD}) == L.Q4_ERR_ALIGN, bad
    for bad in ("dh", "gu", "dx", "dwg", "dwu"):
        assert b(**{bad: None}) == L.Q4_ERR_NULL, bad
    assert f(out=None) == L.Q4_ERR_NULL
    assert f(nbytes=L.raw.swiglu_linear_workspace_bytes(70, 4096, 64) - 1) == L.Q4_ERR_WORKSPACE
    assert b(nbytes=L.raw.swiglu_linear_backward_workspace_bytes(70, 4096, 64) - 1) == L.Q4_ERR_WORKSPACE
    assert f(t=0, x=None, work=None, nbytes=0) == L.Q4_OK
    assert b(t=0, dwg=None) == L.Q4_ERR_NULL     # zero tokens still write the weight gradients
    assert L.raw.swiglu_linear_workspace_bytes(70, 12, 64) == 0
    assert L.raw.swiglu_linear_backward_workspace_bytes(-1, 64, 64) == 0


def _norm(L, **kw):
    d = dict(rows=4, cols=64, dtype=2, gate_kind=0, alpha=1.0, eps=1e-6, res=4096, y=4096, w_post=4096, gate=None,
             w_pre=4096)
    d.update(kw)
    return L.Q4BlockNorm(**d)


def test_block_norm_validation(L):
    def f(r=FAKE, n=FAKE, q=None, s=None, **kw):
        return L.raw.block_norm_forward(ctypes.byref(_norm(L, **kw)), r, n, q, s, None)

    def b(dr=FAKE, dn=FAKE, dres=FAKE, dy=FAKE, dwpost=FAKE, dgate=None, dwpre=FAKE, work=FAKE, nbytes=1 << 40, **kw):
        return L.raw.block_norm_backward(ctypes.byref(_norm(L, **kw)), dr, dn, dres, dy, dwpost, dgate, dwpre, work,
                                         nbytes, None)

    assert L.raw.block_norm_forward(None, FAKE, FAKE, None, None, None) == L.Q4_ERR_NULL
    for call in (f, b):
        assert call(dtype=3) == L.Q4_ERR_DTYPE
        assert call(gate_kind=4, gate=4096) == L.Q4_ERR_DTYPE
        for bad in (dict(cols=0), dict(cols=16385), dict(rows=-1), dict(eps=0.0), dict(eps=float("nan")),
                    dict(alpha=float("inf"))):
            assert call(**bad) == L.Q4_ERR_SHAPE, bad
        for bad in (dict(y=None), dict(y=None, w_post=None, w_pre=None), dict(gate=4096), dict(gate_kind=1),
                    dict(res=None)):
            assert call(**bad) == L.Q4_ERR_NULL, bad
        for bad in ("res", "y", "w_post", "w_pre"):
            assert call(**{bad: 4104}) == L.Q4_ERR_ALIGN, bad
    assert f(r=None) == L.Q4_ERR_NULL
    assert f(n=None) == L.Q4_ERR_NULL
    assert f(q=FAKE, s=FAKE) == L.Q4_ERR_NULL            # both forms of n
    assert f(n=None, q=FAKE) == L.Q4_ERR_NULL            # codes without scales
    assert f(w_pre=None) == L.Q4_ERR_NULL                # n without its weight
    assert f(r=FAKE, y=None, w_post=None) == L.Q4_ERR_NULL
    assert f(rows=0, res=None, r=None, n=None) == L.Q4_OK
    for bad in ("dn", "dres", "dy", "dwpost", "dwpre", "work"):
        assert b(**{bad: None}) == L.Q4_ERR_NULL, bad
    assert b(dgate=FAKE) == L.Q4_ERR_NULL
    assert b(gate_kind=2, gate=4096) == L.Q4_ERR_NULL
    need = L.raw.block_norm_workspace_bytes(ctypes.byref(_norm(L)))
    assert need > 0 and b(nbytes=need - 1) == L.Q4_ERR_WORKSPACE
    assert L.raw.block_norm_workspace_bytes(ctypes.byref(_norm(L, cols=0))) == 0


def test_binding_refuses_cpu_tensors(L):
    z = torch.zeros
    for call in (lambda: L.quantize_int8_channel(z(4, 64)),
                 lambda: L.int8_linear_forward(z(4, 64, dtype=torch.int8), z(4), z(4, 64, dtype=torch.int8), z(4)),
                 lambda: L.swiglu_linear_forward(z(4, 64).half(), z(8, 64).half(), z(8, 64).half()),
                 lambda: L.block_norm_forward(z(4, 64), w_pre=z(64))):
        with pytest.raises(ValueError):
            call()
