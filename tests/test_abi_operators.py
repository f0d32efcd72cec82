"""Refusals of rms_norm_q8_1, q8_1_dequantize, moe_router and mmvq_q4g that need no
GPU: every call below fails host validation (or is a documented no-op), so the
fake device addresses are never dereferenced."""
import ctypes

import pytest
import torch

qmm = pytest.importorskip("quantized_matmul_q8_amd")
from quantized_matmul_q8_amd import _lib  # noqa: E402

L = _lib.LIB
FAKE, MISAL, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0)
F32, F16, BF16 = _lib.QMM_F32, _lib.QMM_F16, _lib.QMM_BF16


def norm(**kw):
    a = dict(x=FAKE, xt=F32, r=FAKE, ro=FAKE, rt=BF16, w=FAKE, wt=F16, off=0.0, eps=1e-6, xq=FAKE, y=FAKE, yt=F32, T=4,
             K=64) | kw
    return L.rms_norm_q8_1(a["x"], a["xt"], a["r"], a["ro"], a["rt"], a["w"], a["wt"], a["off"], a["eps"], a["xq"],
                           a["y"], a["yt"], a["T"], a["K"], NUL)


def test_norm_errors():
    for t in ("xt", "rt", "wt", "yt"):
        assert norm(**{t: 2}) == _lib.QMM_ERR_UNSUPPORTED
    for K in (0, -32, 48, (1 << 30) + 32):
        assert norm(K=K) == _lib.QMM_ERR_SHAPE
    assert norm(T=-1) == _lib.QMM_ERR_SHAPE and norm(T=1 << 31) == _lib.QMM_ERR_SHAPE
    assert norm(eps=-1e-6) == _lib.QMM_ERR_SHAPE and norm(eps=float("nan")) == _lib.QMM_ERR_SHAPE
    for p in ("x", "w", "xq", "r", "ro"):
        assert norm(**{p: NUL}) == _lib.QMM_ERR_NULL
    for p in ("x", "w", "xq", "r", "ro", "y"):
        assert norm(**{p: MISAL}) == _lib.QMM_ERR_ALIGN
    assert norm(T=0, x=NUL, xq=NUL) == _lib.QMM_OK
    # types of what is not given are not looked at
    assert norm(T=0, r=NUL, ro=NUL, rt=7, y=NUL, yt=7) == _lib.QMM_OK


def test_dequantize_errors():
    f = L.q8_1_dequantize
    assert f(FAKE, FAKE, 5, 1, 32, NUL) == _lib.QMM_ERR_UNSUPPORTED
    assert f(FAKE, FAKE, F32, 1, 33, NUL) == _lib.QMM_ERR_SHAPE
    assert f(FAKE, FAKE, F32, -1, 32, NUL) == _lib.QMM_ERR_SHAPE
    assert f(FAKE, FAKE, F32, 1 << 35, 64, NUL) == _lib.QMM_ERR_SHAPE      # T * K > 2^40
    assert f(NUL, FAKE, F32, 1, 32, NUL) == _lib.QMM_ERR_NULL
    assert f(FAKE, NUL, F32, 1, 32, NUL) == _lib.QMM_ERR_NULL
    assert f(MISAL, FAKE, F32, 1, 32, NUL) == _lib.QMM_ERR_ALIGN
    assert f(NUL, NUL, F32, 0, 32, NUL) == _lib.QMM_OK


def router(**kw):
    a = dict(x=FAKE, t=F32, T=4, E=64, k=8, sc=0, b=NUL, g=1, kg=1, gs=0, rn=0, s=1.0, i=FAKE, w=FAKE) | kw
    return L.moe_router(a["x"], a["t"], a["T"], a["E"], a["k"], a["sc"], a["b"], a["g"], a["kg"], a["gs"], a["rn"],
                        a["s"], a["i"], a["w"], NUL)


def test_router_errors():
    assert router(t=3) == _lib.QMM_ERR_UNSUPPORTED
    assert router(sc=2) == _lib.QMM_ERR_UNSUPPORTED
    assert router(gs=2) == _lib.QMM_ERR_UNSUPPORTED
    for kw in (dict(E=0), dict(E=513), dict(k=0), dict(k=65), dict(E=4, k=5), dict(g=0), dict(g=3), dict(g=65, E=65),
               dict(g=8, kg=0), dict(g=8, kg=9), dict(g=8, kg=1, k=9), dict(T=-1), dict(T=(1 << 25) + 1)):
        assert router(**kw) == _lib.QMM_ERR_SHAPE, kw
    for p in ("x", "i", "w"):
        assert router(**{p: NUL}) == _lib.QMM_ERR_NULL
        assert router(**{p: MISAL}) == _lib.QMM_ERR_ALIGN
    assert router(b=MISAL) == _lib.QMM_ERR_ALIGN
    assert router(T=0, x=NUL) == _lib.QMM_OK


def q4g(**kw):
    a = dict(w=FAKE, s=FAKE, st=F16, z=NUL, x=FAKE, y=FAKE, M=4, K=256, g=64, T=1) | kw
    return L.mmvq_q4g(a["w"], a["s"], a["st"], a["z"], a["x"], a["y"], a["M"], a["K"], a["g"], a["T"], NUL)


def test_q4g_errors():
    assert q4g(st=F32) == _lib.QMM_ERR_UNSUPPORTED
    for kw in (dict(M=0), dict(M=(1 << 26) + 1), dict(K=0, g=32), dict(K=48, g=48), dict(K=256, g=16), dict(K=256, g=96),
               dict(K=256, g=512), dict(K=256, g=0), dict(T=0), dict(T=9), dict(K=(1 << 20) + 32, g=32)):
        assert q4g(**kw) == _lib.QMM_ERR_SHAPE, kw
    for p in ("w", "s", "x", "y"):
        assert q4g(**{p: NUL}) == _lib.QMM_ERR_NULL
    for p in ("w", "s", "x", "y", "z"):
        assert q4g(**{p: MISAL}) == _lib.QMM_ERR_ALIGN


def test_binding_refuses_what_is_not_a_device_tensor():
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="HIP device"):
        qmm.rms_norm_q8_1(x, w)
    with pytest.raises(TypeError):
        qmm.rms_norm_q8_1(x.double(), w)
    with pytest.raises(TypeError):
        qmm.moe_router([1.0], 1)
    with pytest.raises(ValueError, match="HIP device"):
        qmm.moe_router(x, 2)
    with pytest.raises(TypeError):
        qmm.mmvq_q4g(x, w, x)
    with pytest.raises(TypeError):
        qmm.q8_1_dequantize(x)
