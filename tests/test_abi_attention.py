"""Refusals of qk_norm_rope, kv_append_q4, kv_read_q4, attn_q4 and attn_prompt that
need no GPU: every call below fails host validation (or is a documented
no-op), so the fake device addresses are never dereferenced."""
import ctypes

import pytest
import torch

qmm = pytest.importorskip("quantized_matmul_q8_amd")
from quantized_matmul_q8_amd import _lib  # noqa: E402

L = _lib.LIB
FAKE, MISAL, NUL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0)
ODD = ctypes.c_void_p(0x10002)     # lists of whole numbers need the alignment of their type
F32, F16, BF16 = _lib.QMM_F32, _lib.QMM_F16, _lib.QMM_BF16
OK, NULL, SHAPE, ALIGN, WS, UNSUP = (_lib.QMM_OK, _lib.QMM_ERR_NULL, _lib.QMM_ERR_SHAPE, _lib.QMM_ERR_ALIGN,
                                     _lib.QMM_ERR_WORKSPACE, _lib.QMM_ERR_UNSUPPORTED)
HUGE = 1 << 31


def rope(**kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, t=F32, qw=FAKE, kw=FAKE, wt=F16, off=0.0, eps=1e-6, r=FAKE, P=10, rot=64, i=0,
             p=FAKE, qo=FAKE, qos=512, ko=FAKE, kos=256, ot=BF16, T=3, Hq=8, Hk=4, D=64) | kw
    return L.qk_norm_rope(*a.values(), NUL)


def test_rope_errors():
    for t in ("t", "wt", "ot"):
        assert rope(**{t: 2}) == UNSUP
    assert rope(T=0, wt=9, qw=NUL, kw=NUL) == OK                  # the type of weights that are not there
    for kw in (dict(T=-1), dict(T=HUGE), dict(Hq=0), dict(Hq=1025, qs=1 << 17, qos=1 << 17), dict(Hk=0), dict(D=48),
               dict(D=0), dict(D=544, qs=8192, qos=8192, ks=8192, kos=8192), dict(rot=8), dict(rot=-16), dict(rot=80),
               dict(P=0), dict(P=HUGE), dict(eps=-1.0), dict(eps=float("nan")), dict(qs=504), dict(qs=516), dict(ks=248),
               dict(qos=0), dict(kos=260), dict(qs=HUGE), dict(T=1 << 26), dict(T=1 << 26, k=NUL, Hq=1)):
        assert rope(**kw) == SHAPE, kw
    for p in ("q", "qo", "ko", "r", "p"):
        assert rope(**{p: NUL}) == NULL, p
    for p in ("q", "k", "qw", "kw", "r", "qo", "ko"):
        assert rope(**{p: MISAL}) == ALIGN, p
    assert rope(p=ODD) == ALIGN
    assert rope(T=0, q=NUL) == OK
    assert rope(T=0, k=NUL, ko=NUL, Hk=0, ks=0, kos=0) == OK      # no keys: their sizes are not looked at
    assert rope(T=0, rot=0, P=0, r=NUL, p=NUL) == OK


def append(**kw):
    a = dict(k=FAKE, ks=256, kt=F32, v=FAKE, vs=256, vt=F16, r=FAKE, P=10, rot=64, i=0, p=FAKE, s=FAKE, c=FAKE, pages=4, page=16,
             T=3, Hk=4, D=64) | kw
    return L.kv_append_q4(*a.values(), NUL)


def test_append_errors():
    assert append(kt=5) == UNSUP and append(vt=7) == UNSUP
    for kw in (dict(T=-1), dict(T=1 << 30), dict(Hk=0), dict(Hk=1025, ks=1 << 17, vs=1 << 17), dict(D=32), dict(D=160, ks=640, vs=640),
               dict(page=0), dict(page=24), dict(page=(1 << 20) + 16), dict(pages=0), dict(pages=HUGE), dict(ks=255),
               dict(vs=260), dict(rot=24), dict(rot=80), dict(P=0)):
        assert append(**kw) == SHAPE, kw
    assert append(T=1 << 26, Hk=1) == SHAPE and append(T=(1 << 26) - 1, Hk=1, c=NUL) == NULL
    for p in ("k", "v", "r", "p", "s", "c"):
        assert append(**{p: NUL}) == NULL, p
        assert append(**{p: ODD if p in "ps" else MISAL}) == ALIGN, p
    assert append(T=0, k=NUL) == OK


def read(**kw):
    a = dict(c=FAKE, pages=4, page=16, s=FAKE, k=FAKE, v=FAKE, t=F16, T=3, Hk=4, D=64) | kw
    return L.kv_read_q4(*a.values(), NUL)


def test_read_errors():
    assert read(t=7) == UNSUP
    for kw in (dict(T=-1), dict(T=HUGE), dict(Hk=0), dict(D=80), dict(page=8), dict(pages=0), dict(T=1 << 26, Hk=1)):
        assert read(**kw) == SHAPE, kw
    for p in ("c", "s", "k", "v"):
        assert read(**{p: NUL}) == NULL
        assert read(**{p: ODD if p == "s" else MISAL}) == ALIGN
    assert read(T=0, c=NUL) == OK


def cached(**kw):
    a = dict(q=FAKE, qs=512, t=F16, c=FAKE, pages=4, page=16, tab=FAKE, W=2, lens=FAKE, sc=0.125, win=0, y=FAKE, yt=F32,
             B=2, n=1, Hq=8, Hk=4, D=64, ws=FAKE, wsb=1 << 30) | kw
    return L.attn_q4(*a.values(), NUL)


def test_cached_attention_errors():
    assert cached(t=F32) == UNSUP and cached(t=3) == UNSUP and cached(yt=4) == UNSUP
    for kw in (dict(qs=504), dict(qs=513), dict(page=20), dict(pages=0), dict(W=0), dict(W=1 << 27), dict(B=-1), dict(n=0),
               dict(n=9), dict(Hq=6), dict(Hq=2), dict(Hk=0), dict(Hq=1028, qs=1 << 17), dict(D=72), dict(sc=float("inf")),
               dict(sc=float("nan")), dict(win=-1), dict(win=HUGE), dict(B=1 << 20),
               dict(B=1 << 11, W=1 << 21)):
        assert cached(**kw) == SHAPE, kw
    for p in ("q", "c", "tab", "lens", "y"):
        assert cached(**{p: NUL}) == NULL, p
    for p in ("q", "c", "tab", "lens", "y", "ws"):
        assert cached(**{p: ODD if p in ("tab", "lens") else MISAL}) == ALIGN, p
    assert cached(B=0, q=NUL) == OK


def test_cached_attention_workspace():
    f = L.attn_q4_workspace_bytes
    for kw in ((-1, 1, 8, 4, 64, 100), (2, 0, 8, 4, 64, 100), (2, 9, 8, 4, 64, 100), (2, 1, 6, 4, 64, 100),
               (2, 1, 8, 4, 80, 100), (2, 1, 8, 4, 64, 0), (2, 1, 8, 4, 64, (1 << 30) + 16)):
        assert f(*kw) == 0
    need = f(1, 1, 8, 4, 64, 1 << 20)
    if need:
        assert cached(B=1, W=1 << 16, wsb=need - 1) == WS
        assert cached(B=1, W=1 << 16, ws=NUL, wsb=0) == NULL


def prompt(**kw):
    a = dict(q=FAKE, qs=512, k=FAKE, ks=256, v=FAKE, vs=256, t=BF16, cq=FAKE, ck=FAKE, B=2, sc=0.1, ca=1, win=0, y=FAKE,
             yt=F16, Tq=10, Tk=20, Hq=8, Hk=4, D=64, ws=FAKE, wsb=1 << 40) | kw
    return L.attn_prompt(*a.values(), NUL)


def test_prompt_errors():
    assert prompt(t=F32) == UNSUP and prompt(yt=2) == UNSUP and prompt(win=5, ca=0) == UNSUP
    for kw in (dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(Tq=1 << 30), dict(Tk=1 << 30), dict(Hq=6), dict(Hk=0), dict(Hq=0),
               dict(D=32), dict(D=320), dict(qs=500), dict(ks=8), dict(vs=257), dict(win=-1), dict(win=HUGE),
               dict(sc=float("nan")), dict(B=HUGE), dict(B=1 << 20), dict(Hq=1032, qs=1 << 17)):
        assert prompt(**kw) == SHAPE, kw
    for p in ("q", "k", "v", "cq", "ck", "y"):
        assert prompt(**{p: NUL}) == NULL, p
        assert prompt(**{p: ODD if p in ("cq", "ck") else MISAL}) == ALIGN, p
    assert prompt(ws=MISAL) == ALIGN
    assert prompt(B=0, q=NUL) == OK and prompt(Tq=0, y=NUL) == OK


def test_prompt_workspace():
    f = L.attn_prompt_workspace_bytes
    for sizes in ((-1, 1, 1, 8, 4, 64), (1, -1, 1, 8, 4, 64), (1, 1, -1, 8, 4, 64), (1, 1, 1, 6, 4, 64), (1, 1, 1, 8, 4, 80),
                  (1, 1 << 30, 1, 8, 4, 64)):
        assert f(*sizes) == 0
    need = f(1, 16, 1 << 16, 8, 4, 64)
    if need:
        assert prompt(B=1, Tq=16, Tk=1 << 16, wsb=need - 1) == WS
        assert prompt(B=1, Tq=16, Tk=1 << 16, ws=NUL, wsb=0) == NULL


def test_binding_refuses_what_does_not_fit():
    x, i = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="HIP device"):
        qmm.qk_norm_rope(x)
    with pytest.raises(TypeError):
        qmm.qk_norm_rope(x.double())
    with pytest.raises(TypeError):
        qmm.qk_norm_rope([1.0])
    with pytest.raises(ValueError):
        qmm.kv_cache_q4(2, 24, 4, 64, "cpu")
    c = qmm.kv_cache_q4(2, 32, 4, 64, "cpu")
    assert tuple(c.shape) == (2, 4, 2, 1280) and not c.any()
    with pytest.raises(ValueError, match="HIP device"):
        qmm.kv_append_q4(x, x, c, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="HIP device"):
        qmm.kv_read_q4(c, torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="HIP device"):
        qmm.attn_q4(x.half(), c, i.view(1, 2), i)
    with pytest.raises(ValueError, match="HIP device"):
        qmm.attn_prompt(x.half(), x.half(), x.half(), i)
