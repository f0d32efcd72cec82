"""GPU: rms_norm_q8_1 and q8_1_dequantize.

The unquantized rows are compared with the float64 oracle, and the Q8_1 bytes
exactly with the oracle's quantizer applied to the kernel's own fp32 rows.

Tolerance of n (relative, per element): the sum of K squares is one of
positive terms, so its error is at most its longest chain of additions, at
most K/64 + 10 of them for any split over 64 or more lanes, plus one rounding
for each square; the square root halves it.  The division by K, eps's
addition (halved), the square root, its reciprocal, the two products and the
weight's offset add at most 7 roundings, each of 2^-24 relative.
"""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def tolerance(K):
    return ((K / 64 + 11) / 2 + 7) * 2.0**-24


def inputs(T, K, xt, rt, wt, seed):
    g = qmm_synth.rng(seed)
    x = torch.from_numpy(qmm_synth.activations(g, T, K, 0.01)).to(xt)
    r = None if rt is None else torch.from_numpy(2 * qmm_synth.activations(g, T, K, 0.01)).to(rt)
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(K).astype(np.float32)).to(wt)
    return x, r, w


def check(T, K, xt=F32, rt=None, wt=F32, offset=0.0, eps=1e-6, seed=1, x=None):
    x0, r, w = inputs(T, K, xt, rt, wt, seed)
    x = x0 if x is None else x
    say("rms_norm_q8_1", f"T={T} K={K} x={xt} residual={rt} w={wt} offset={offset} eps={eps}")
    rd = None if r is None else r.to(DEV)
    xq, ro, y = qmm.rms_norm_q8_1(x.to(DEV), w.to(DEV), eps, residual=rd, weight_offset=offset, y_dtype=F32)
    h = x
    if r is None:
        assert ro is None
    else:
        h = (x.float() + r.float()).to(rt)          # one fp32 addition, rounded once
        assert torch.equal(ro.cpu(), h)
        assert torch.equal(rd.cpu(), r)
    n = oracle.rms_norm(h.double().numpy(), w.double().numpy(), eps, offset)
    yh = host(y)
    assert np.all(np.abs(yh - n) <= tolerance(K) * np.abs(n) + 2.0**-126)
    assert np.array_equal(host(xq), oracle.quantize_q8_1(yh))
    return xq, ro, y


@pytest.mark.parametrize("K", [32, 64, 96, 256, 992, 1024, 1056, 2048, 2080, 4096, 5120, 8192, 8224, 11008, 16384, 20000,
                               32768, 40960, 65536 + 32])
@pytest.mark.parametrize("T", [1, 5])
def test_sizes(T, K):
    check(T, K, F32, BF16, F32, seed=K + T)
    check(T, K, BF16, None, BF16, seed=K + T + 1)


@pytest.mark.parametrize("xt", [F32, F16, BF16])
@pytest.mark.parametrize("rt", [None, F32, F16, BF16])
@pytest.mark.parametrize("wt", [F32, F16, BF16])
def test_types(xt, rt, wt):
    check(3, 672, xt, rt, wt, offset=1.0 if wt == F32 else 0.0, eps=1e-5, seed=7)
    check(2, 4096, xt, rt, wt, eps=1e-5, seed=8)


@pytest.mark.parametrize("T,K", [(70, 2048), (700, 4096), (4097, 128), (300, 8192), (40, 20480)])
def test_many_rows(T, K):
    check(T, K, BF16, BF16, BF16, seed=T)


def test_copy_is_the_rounded_row_and_changes_nothing():
    x, r, w = (t.to(DEV) for t in inputs(9, 2080, F16, F32, F16, 3))
    xq, ro, y = qmm.rms_norm_q8_1(x, w, 1e-6, residual=r, y_dtype=F32)
    for t in (F16, BF16):
        xq2, ro2, y2 = qmm.rms_norm_q8_1(x, w, 1e-6, residual=r, y_dtype=t)
        assert torch.equal(xq, xq2) and torch.equal(ro, ro2) and torch.equal(y2, y.to(t))
    xq3, ro3, none = qmm.rms_norm_q8_1(x, w, 1e-6, residual=r)
    assert none is None and torch.equal(xq, xq3) and torch.equal(ro, ro3)


def test_a_row_does_not_depend_on_the_others():
    for K in (64, 2048, 4096, 11008):
        x, r, w = (t.to(DEV) for t in inputs(300, K, BF16, BF16, BF16, 4))
        xq, ro, y = qmm.rms_norm_q8_1(x, w, 1e-5, residual=r, y_dtype=F32)
        for i in (0, 17, 299):
            a, b, c = qmm.rms_norm_q8_1(x[i:i + 1], w, 1e-5, residual=r[i:i + 1], y_dtype=F32)
            assert torch.equal(a[0], xq[i]) and torch.equal(b[0], ro[i]) and torch.equal(c[0], y[i])


def test_in_place_and_out_buffers_and_rows_behind():
    x, r, w = (t.to(DEV) for t in inputs(6, 1056, F32, BF16, F32, 5))
    xq, ro, y = qmm.rms_norm_q8_1(x, w, residual=r, y_dtype=F16)
    stream = torch.full((9, 1056), 7.0, dtype=BF16, device=DEV)
    stream[:6] = r
    out = torch.full((9, 33, 40), 0xA5, dtype=torch.uint8, device=DEV)
    copy = torch.full((9, 1056), -3.0, dtype=F16, device=DEV)
    a, b, c = qmm.rms_norm_q8_1(x, w, residual=stream[:6], residual_out=stream[:6], out=out[:6], y=copy[:6])
    assert a.data_ptr() == out.data_ptr() and b.data_ptr() == stream.data_ptr() and c.data_ptr() == copy.data_ptr()
    assert torch.equal(stream[:6], ro) and torch.equal(out[:6], xq) and torch.equal(copy[:6], y)
    assert torch.all(stream[6:] == 7) and torch.all(out[6:] == 0xA5) and torch.all(copy[6:] == -3)
    # the sum written over x, in x's own type
    x2 = x.clone()
    a, b, _ = qmm.rms_norm_q8_1(x2, w, residual=r.float(), residual_out=r.float())
    assert torch.equal(x2, x)


def test_edge_rows():
    K = 256
    x = torch.zeros(6, K)
    x[1, 5] = 1e-20                       # far below eps
    x[2] = 3e4 * torch.sign(torch.randn(K, generator=torch.Generator().manual_seed(1)))
    x[3] = 1e15                           # squares near the top of fp32's range
    x[4, ::2] = -0.0
    x[5, 100] = 65504.0                   # one value in an empty row
    _, _, y = check(6, K, x=x, eps=1e-6)
    assert torch.all(y[0] == 0) and torch.all(y[4] == 0)
    check(6, K, F16, F16, F16, x=torch.randn(6, K, generator=torch.Generator().manual_seed(2)).half(), eps=0.0)


@pytest.mark.parametrize("K", [64, 4096, 40960])
def test_rows_of_zeros_without_eps(K):
    x = torch.zeros(3, K, device=DEV)
    x[1] = torch.linspace(-2, 3, K, device=DEV)
    xq, ro, y = qmm.rms_norm_q8_1(x, torch.ones(K, device=DEV), 0.0, residual=torch.zeros_like(x).half(), y_dtype=F32)
    assert torch.all(y[[0, 2]] == 0) and torch.all(xq[[0, 2]] == 0)
    n = oracle.rms_norm(ro[1:2].double().cpu().numpy(), np.ones(K), 0.0)
    assert np.all(np.abs(host(y)[1] - n[0]) <= tolerance(K) * np.abs(n[0]))


def test_more_rows_than_workgroups():
    # rows of one block, past the launch's workgroups of four and eight rows
    T = (1 << 22) + 5
    x = torch.randn(T, 32, device=DEV, generator=torch.Generator(DEV).manual_seed(3)).bfloat16()
    w = torch.ones(32, device=DEV)
    xq, _, _ = qmm.rms_norm_q8_1(x, w)
    tail, _, _ = qmm.rms_norm_q8_1(x[-1000:], w)
    head, _, _ = qmm.rms_norm_q8_1(x[:1000], w)
    assert torch.equal(xq[-1000:], tail) and torch.equal(xq[:1000], head)
    back = qmm.q8_1_dequantize(xq, BF16)
    assert torch.equal(back[-1000:], qmm.q8_1_dequantize(tail, BF16))


def test_empty_and_refused():
    w = torch.ones(64, device=DEV)
    xq, ro, y = qmm.rms_norm_q8_1(torch.empty(0, 64, device=DEV), w, residual=torch.empty(0, 64, device=DEV), y_dtype=F16)
    assert tuple(xq.shape) == (0, 2, 40) and tuple(ro.shape) == (0, 64) and tuple(y.shape) == (0, 64)
    x = torch.zeros(4, 64, device=DEV)
    for bad in (lambda: qmm.rms_norm_q8_1(torch.zeros(4, 48, device=DEV), w),
                lambda: qmm.rms_norm_q8_1(x, torch.ones(32, device=DEV)),
                lambda: qmm.rms_norm_q8_1(x, w, -1.0),
                lambda: qmm.rms_norm_q8_1(x, w, residual=x[:3]),
                lambda: qmm.rms_norm_q8_1(x, w, residual_out=x),
                lambda: qmm.rms_norm_q8_1(torch.zeros(4, 128, device=DEV)[:, :64], w),
                lambda: qmm.rms_norm_q8_1(torch.zeros(64, 4, device=DEV).t(), w),
                lambda: qmm.rms_norm_q8_1(x, w, out=torch.empty(3, 2, 40, dtype=torch.uint8, device=DEV)),
                lambda: qmm.rms_norm_q8_1(x, w, residual=x.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: qmm.rms_norm_q8_1(x.double(), w), lambda: qmm.rms_norm_q8_1(x, w, y_dtype=torch.int8),
                lambda: qmm.rms_norm_q8_1(x, w, y_dtype=F16, y=torch.empty(4, 64, device=DEV))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(qmm.QmmError):       # 4-byte aligned only
        qmm.rms_norm_q8_1(torch.zeros(65, device=DEV)[1:].view(1, 64), w)


@pytest.mark.parametrize("T,K", [(1, 32), (1, 4096), (3, 96), (7, 2080), (130, 11008), (1000, 992)])
def test_dequantize(T, K):
    g = qmm_synth.rng(T + K)
    x = qmm_synth.activations(g, T, K, 0.01)
    x[0, :32] = 0
    x[T - 1, K - 32:] *= np.float32(1e-6)          # a subnormal f16 scale
    xq = oracle.quantize_q8_1(x)
    say("q8_1_dequantize", f"T={T} K={K}")
    ref = torch.from_numpy(oracle.q8_1_dequant(xq)).float()      # 19 significant bits: exact in fp32
    d = dev(xq)
    assert torch.equal(qmm.q8_1_dequantize(d).cpu(), ref)
    for t in (F16, BF16):
        assert torch.equal(qmm.q8_1_dequantize(d, t).cpu(), ref.to(t))


def test_dequantize_every_int8_and_scale_corner():
    q = np.zeros((8, 8, 40), np.uint8)
    q[:, :, 4:36] = np.arange(256, dtype=np.uint8).reshape(8, 32)
    for i, d in enumerate([0.0, 2.0**-24, -1.5, 1.0, 65504.0, 2.0**-14, 3e-5, 123.4]):
        q[i, :, 0:2] = np.array([d], np.float16).view(np.uint8)
    ref = torch.from_numpy(oracle.q8_1_dequant(q)).float()
    assert torch.equal(qmm.q8_1_dequantize(dev(q)).cpu(), ref)
    assert torch.equal(qmm.q8_1_dequantize(dev(q), F16).cpu(), ref.half())       # infinite above 65504


def test_dequantize_buffers_and_refusals():
    xq = dev(oracle.quantize_q8_1(qmm_synth.activations(qmm_synth.rng(1), 3, 64)))
    big = torch.full((5, 64), 9.0, dtype=BF16, device=DEV)
    out = qmm.q8_1_dequantize(xq, BF16, out=big[:3])
    assert out.data_ptr() == big.data_ptr() and torch.all(big[3:] == 9)
    assert tuple(qmm.q8_1_dequantize(xq[:0]).shape) == (0, 64)
    with pytest.raises(ValueError):
        qmm.q8_1_dequantize(xq, BF16, out=big)
    with pytest.raises(ValueError):
        qmm.q8_1_dequantize(xq[..., :36].contiguous())
    with pytest.raises(TypeError):
        qmm.q8_1_dequantize(xq, torch.float64)


@pytest.mark.parametrize("K", [64, 512, 768, 1024, 2048, 4096, 8192, 11008, 20000, 40960])
@pytest.mark.parametrize("rt", [None, F32, BF16])
def test_rows_whose_squares_leave_fp32(K, rt):
    """Finite rows whose squares, or their sum, are above or below what fp32 holds, between ordinary rows."""
    g = torch.Generator().manual_seed(K)
    x = torch.randn(11, K, generator=g)
    x[1] *= 2.0**60                       # from K = 512: the sum is past fp32, the mean is not
    x[2] *= 2.0**63
    x[4] *= 2.0**120                      # the mean is past fp32
    x[5] = x[5].clamp(-1, 1) * 3e38
    x[5, ::7] *= 2.0**-140                # and values far smaller in the same row
    x[2, ::5] *= 2.0**-100
    x[8, ::5] *= 2.0**-30
    x[7] *= 2.0**-50
    x[8] *= 2.0**-66                      # subnormal squares
    x[9] *= 2.0**-75                      # squares below every fp32 value
    x[10] = x[10].sign() * 2.0**(-133 if rt == BF16 else -149)       # the type's smallest
    assert torch.all(x[10] != 0)
    r = None if rt is None else torch.zeros(11, K, dtype=rt)
    w = 1 + 0.2 * torch.randn(K, generator=g)
    for eps in (0.0, 1e-38, 1e-6):
        say("rms_norm_q8_1", f"K={K} residual={rt} eps={eps}")
        xq, ro, y = qmm.rms_norm_q8_1(x.to(DEV), w.to(DEV), eps, residual=None if r is None else r.to(DEV), y_dtype=F32)
        h = x if rt is None else ro.cpu()
        assert rt is None or torch.equal(h, x.to(rt))
        n = oracle.rms_norm(h.double().numpy(), w.double().numpy(), float(np.float32(eps)))
        yh = host(y)
        assert np.all(np.isfinite(n)) and np.all(np.abs(yh - n) <= tolerance(K) * np.abs(n) + 2.0**-126), eps
        assert np.array_equal(host(xq), oracle.quantize_q8_1(yh))
        for i in (0, 1, 3, 6, 9):         # an ordinary row's neighbours change nothing in it
            a, _, b = qmm.rms_norm_q8_1(h[i:i + 1].to(DEV), w.to(DEV), eps, y_dtype=F32)
            assert torch.equal(a[0], xq[i]) and torch.equal(b[0], y[i])


@pytest.mark.parametrize("K", [64, 768, 2080, 4096, 11008, 20000, 40960])
@pytest.mark.parametrize("rt", [F32, F16, BF16])
def test_stream_updated_in_place(K, rt):
    x, r, w = (t.to(DEV) for t in inputs(7, K, F32, rt, F32, K))
    x[2], r[2] = 2.0**-70 * x[2], 0      # with eps = 0 rows that are read again from the updated stream
    if rt != F16:
        x[5], r[5] = 2.0**100 * x[5], 0
    for eps in (1e-6, 0.0):
        say("rms_norm_q8_1", f"in place K={K} residual={rt} eps={eps}")
        xq, ro, y = qmm.rms_norm_q8_1(x, w, eps, residual=r, y_dtype=F32)
        stream = r.clone()
        a, b, c = qmm.rms_norm_q8_1(x, w, eps, residual=stream, residual_out=stream, y_dtype=F32)
        assert b.data_ptr() == stream.data_ptr()
        assert torch.equal(ro, (x + r.float()).to(rt)) and torch.equal(stream, ro)
        assert torch.equal(a, xq) and torch.equal(c, y)


# streams of 128 MB and more are stored past the caches; rows of such a call are those of smaller ones
@pytest.mark.parametrize("T,K,rt", [(8195, 4096, F32), (16389, 4096, BF16), (8197, 8192, F16), (2051, 16416, F32)])
def test_large_streams(T, K, rt):
    g = torch.Generator(DEV).manual_seed(K)
    x = torch.randn(T, K, device=DEV, generator=g).to(rt)
    r = (2 * torch.randn(T, K, device=DEV, generator=g)).to(rt)
    w = 1 + 0.2 * torch.randn(K, device=DEV, generator=g)
    assert T * K * r.element_size() >= 1 << 27
    say("rms_norm_q8_1", f"large T={T} K={K} {rt}")
    xq, ro, _ = qmm.rms_norm_q8_1(x, w, residual=r)
    assert torch.equal(ro, (x.float() + r.float()).to(rt))
    for i in range(0, T, 1000):
        a, b, _ = qmm.rms_norm_q8_1(x[i:i + 1000], w, residual=r[i:i + 1000])
        assert torch.equal(a, xq[i:i + 1000]) and torch.equal(b, ro[i:i + 1000])
    stream = r.clone()
    a, b, _ = qmm.rms_norm_q8_1(x, w, residual=stream, residual_out=stream)
    assert torch.equal(a, xq) and torch.equal(stream, ro)


def test_scaled_rows_past_the_first_workgroups():
    T = (1 << 22) + 5                     # four rows to a workgroup, and one row more than all of them have at first
    x = torch.randn(T, 32, device=DEV, generator=torch.Generator(DEV).manual_seed(4)).bfloat16()
    for i in (0, 1, 77, (1 << 22) - 1, 1 << 22, T - 1):
        x[i] = x[i] * 2.0**-100
    x[2], x[T - 2] = x[2] * 2.0**100, x[T - 2] * 2.0**100
    w = torch.ones(32, device=DEV)
    xq, _, y = qmm.rms_norm_q8_1(x, w, 0.0, y_dtype=F32)
    assert torch.all(y.abs().amax(1) > 0.5)
    for rows in (slice(0, 100), slice((1 << 22) - 50, T)):
        n = oracle.rms_norm(x[rows].double().cpu().numpy(), np.ones(32), 0.0)
        assert np.all(np.abs(host(y[rows]) - n) <= tolerance(32) * np.abs(n))
        a, _, b = qmm.rms_norm_q8_1(x[rows].contiguous(), w, 0.0, y_dtype=F32)
        assert torch.equal(a, xq[rows]) and torch.equal(b, y[rows])
