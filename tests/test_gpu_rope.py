"""GPU: qk_norm_rope.

Tolerance of a normed value (relative): the sum of D <= 512 squares is one of
positive terms, sixteen in a chain per lane and five exchanges, each square and
addition one rounding: 22, halved by the square root; the division by D, eps's
addition (both halved), the square root, its reciprocal, three products and the
weight's offset add at most 7.  A turned value is the sum of two products of
these by exact table entries: |a c| + |b s| times that and three more
roundings.  Each rounding is 2^-24; the output's is half a step of its type.
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
U = 2.0**-24
HALF_STEP = {F32: 2.0**-24, F16: 2.0**-11, BF16: 2.0**-8}
LEAST = {F32: 2.0**-126, F16: 2.0**-25, BF16: 2.0**-126}      # half a step of the smallest numbers


def expected(x, w, eps, offset, table, pos, interleaved, yt):
    """(value, allowed error) of one side in float64."""
    x = x.double().cpu().numpy()
    n = x if w is None else oracle.head_norm(x, w.double().cpu().numpy(), eps, offset)
    rel = 0.0 if w is None else (22 / 2 + 7) * U
    y, size = n, np.abs(n)
    if table is not None:
        t = table.double().cpu().numpy()
        y = oracle.turn(n, t, pos.cpu().numpy(), interleaved)
        both = oracle.turn(np.abs(n), np.abs(t) * np.where(np.arange(t.shape[1]) < t.shape[1] // 2, 1, -1), pos.cpu().numpy(),
                           interleaved)
        other = oracle.turn(np.abs(n), np.abs(t), pos.cpu().numpy(), interleaved)
        size = np.maximum(np.abs(both), np.abs(other))         # |a c| + |b s| of either of the pair
        rel += 3 * U
    err = rel * size
    return y, err + HALF_STEP[yt] * (np.abs(y) + err) + LEAST[yt]


def check(T, Hq, Hk, D, xt=F32, yt=F32, wt=F32, rot=None, interleaved=False, offset=0.0, eps=1e-6, seed=1, x=None, P=50,
          pos=None):
    say("qk_norm_rope", f"T={T} Hq={Hq} Hk={Hk} D={D} x={xt} y={yt} w={wt} rot={rot} interleaved={interleaved}")
    g = qmm_synth.rng(seed)
    rot = D if rot is None else rot
    if x is None:
        x = dev(qmm_synth.activations(g, T, (Hq + 2 * Hk) * D, 0.01)).to(xt)
    x = x.view(T, Hq + 2 * Hk, D)
    q, k = x[:, :Hq], x[:, Hq:Hq + Hk]
    wq, wk = (None if wt is None else dev(1 + 0.2 * g.standard_normal(D).astype(np.float32)).to(wt) for _ in range(2))
    table = dev(oracle.rope_table(P, rot)) if rot else None
    if pos is None:
        pos = g.integers(0, P, T).astype(np.int32)
    pos = dev(np.asarray(pos, np.int32)) if rot else None
    before = x.clone()
    yq, yk = qmm.qk_norm_rope(q, k, table, pos, q_weight=wq, k_weight=wk, eps=eps, weight_offset=offset,
                              interleaved=interleaved, dtype=yt)
    assert torch.equal(x, before)
    for y, side, w in ((yq, q, wq), (yk, k, wk)):
        assert y.dtype == yt and y.shape == side.shape
        ref, tol = expected(side, w, eps, offset, table, pos, interleaved, yt)
        got = y.double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= tol), float(np.max(np.abs(got - ref) - tol))
    return yq, yk


@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 256, 352, 512])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes(D, interleaved):
    check(3, 5, 2, D, seed=D, interleaved=interleaved)
    check(1, 1, 1, D, F16, F16, None, seed=D + 1, interleaved=interleaved)
    for rot in (16, D // 2 // 16 * 16, D - 16):
        if 0 < rot:
            check(2, 3, 3, D, BF16, F32, BF16, rot, interleaved, seed=D + rot)


@pytest.mark.parametrize("xt", [F32, F16, BF16])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
@pytest.mark.parametrize("wt", [None, F32, F16, BF16])
def test_types(xt, yt, wt):
    check(5, 7, 1, 128, xt, yt, wt, offset=1.0 if wt == F32 else 0.0, eps=1e-5, seed=3)


@pytest.mark.parametrize("T,Hq,Hk,D", [(1, 32, 8, 128), (333, 32, 8, 128), (2500, 28, 4, 128), (5000, 15, 15, 64),
                                       (700, 40, 1, 96), (600, 10, 5, 256), (70, 1024, 1, 32)])
def test_many(T, Hq, Hk, D):
    # enough tokens that a wave goes over several heads of one
    check(T, Hq, Hk, D, BF16, BF16, BF16, seed=T, P=T)
    check(T, Hq, Hk, D, F32, F16, F32, D // 2, True, seed=T + 1, P=7)


def test_norm_without_turn_and_neither():
    check(9, 4, 2, 128, rot=0)
    check(9, 4, 2, 128, F16, F16, None, rot=0)                 # a copy
    check(9, 4, 2, 128, F32, BF16, None, rot=0)


def test_positions_outside_the_table_count_as_the_nearest():
    check(6, 2, 1, 64, pos=[-1, 0, 49, 50, 2**31 - 1, -2**31])


def test_one_side_normed_and_no_keys():
    g = qmm_synth.rng(8)
    x = dev(qmm_synth.activations(g, 6, 8 * 64)).view(6, 8, 64)
    w, table = torch.full((64,), 2.0, device=DEV), dev(oracle.rope_table(9, 64))
    pos = torch.arange(6, dtype=torch.int32, device=DEV)
    a, none = qmm.qk_norm_rope(x, None, table, pos, q_weight=w)
    assert none is None
    b, c = qmm.qk_norm_rope(x, x, table, pos, q_weight=w)
    assert torch.equal(a, b)
    d, _ = qmm.qk_norm_rope(x, None, table, pos)
    assert torch.equal(c, d)
    e, f = qmm.qk_norm_rope(x, x, table, pos, k_weight=w)
    assert torch.equal(e, d) and torch.equal(f, a)


def test_in_place_and_out_buffers_and_rows_behind():
    g = qmm_synth.rng(9)
    T, Hq, Hk, D = 6, 4, 2, 96
    x = dev(qmm_synth.activations(g, T, 10 * D)).to(BF16).view(T, 10, D)
    w, table = torch.ones(D, device=DEV), dev(oracle.rope_table(9, D))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    yq, yk = qmm.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], table, pos, q_weight=w, k_weight=w)
    y = x.clone()
    a, b = qmm.qk_norm_rope(y[:, :Hq], y[:, Hq:Hq + Hk], table, pos, q_weight=w, k_weight=w, q_out=y[:, :Hq],
                            k_out=y[:, Hq:Hq + Hk])
    assert a.data_ptr() == y.data_ptr()
    assert torch.equal(y[:, :Hq], yq) and torch.equal(y[:, Hq:Hq + Hk], yk) and torch.equal(y[:, Hq + Hk:], x[:, Hq + Hk:])
    big = torch.full((T + 3, 16, D), 5.0, dtype=F16, device=DEV)
    qmm.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], table, pos, q_weight=w, k_weight=w, q_out=big[:T, 1:1 + Hq],
                     k_out=big[:T, 8:8 + Hk])
    ref = qmm.qk_norm_rope(x[:, :Hq], x[:, Hq:Hq + Hk], table, pos, q_weight=w, k_weight=w, dtype=F16)
    assert torch.equal(big[:T, 1:1 + Hq], ref[0]) and torch.equal(big[:T, 8:8 + Hk], ref[1])
    big[:T, 1:1 + Hq] = 5
    big[:T, 8:8 + Hk] = 5
    assert torch.all(big == 5)
    empty = qmm.qk_norm_rope(x[:0, :Hq], x[:0, Hq:Hq + Hk], table, pos[:0])
    assert empty[0].shape == (0, Hq, D)


@pytest.mark.parametrize("yt,T", [(BF16, 20000), (F16, 15000), (F32, 9001)])
def test_large_outputs_equal_small_ones(yt, T):
    """Outputs past the caches' size are stored another way; the values are the same."""
    Hq, Hk, D = 32, 8, 128
    g = torch.Generator(device=DEV).manual_seed(6)
    x = torch.randn(T, Hq + Hk, D, device=DEV, generator=g).to(BF16)
    pos = torch.randint(0, 50, (T,), dtype=torch.int32, device=DEV, generator=g)
    table = dev(oracle.rope_table(50, D))
    w = 1 + 0.1 * torch.randn(D, device=DEV, generator=g)
    q, k = qmm.qk_norm_rope(x[:, :Hq], x[:, Hq:], table, pos, q_weight=w, k_weight=w, dtype=yt)
    for i in range(0, T, 5000):
        qs, ks = qmm.qk_norm_rope(x[i:i + 5000, :Hq], x[i:i + 5000, Hq:], table, pos[i:i + 5000].clone(), q_weight=w, k_weight=w,
                                  dtype=yt)
        assert torch.equal(q[i:i + 5000], qs) and torch.equal(k[i:i + 5000], ks), i


def test_rows_far_apart():
    # a stride that takes the offsets past 32 bits
    stride, T, D = (1 << 24) - 8, 140, 64
    g = qmm_synth.rng(7)
    x = dev(qmm_synth.activations(g, T, 6 * D)).to(BF16)
    wide = torch.zeros((T, stride), dtype=BF16, device=DEV)
    wide[:, stride - 6 * D:] = x
    far = wide[:, stride - 6 * D:].view(T, 6, D)
    pos, table = dev(g.integers(0, 50, T).astype(np.int32)), dev(oracle.rope_table(50, D))
    for a, b in zip(qmm.qk_norm_rope(far[:, :4], far[:, 4:], table, pos),
                    qmm.qk_norm_rope(x.view(T, 6, D)[:, :4], x.view(T, 6, D)[:, 4:], table, pos)):
        assert torch.equal(a, b)


def test_edge_heads():
    D = 64
    x = torch.zeros(1, 10, D, device=DEV)
    x[0, 1] = 1e-30 * torch.linspace(-1, 1, D, device=DEV)     # squares below fp32
    x[0, 2] = 1e36 * torch.linspace(-1, 1, D, device=DEV)      # and past it
    x[0, 3, 7] = 3e38
    x[0, 4] = -0.0
    x[0, 5, 0] = 1e-45
    x[0, 6] = torch.linspace(-3, 2, D, device=DEV)
    for eps in (0.0, 1e-6):
        yq, yk = check(1, 8, 1, D, x=x, eps=eps, P=5, pos=[3])
        assert torch.all(yq[0, 0] == 0) and torch.all(yq[0, 4] == 0)
    x[0, 2, 5] = float("nan")
    x[0, 3, 1] = float("inf")
    y, _ = qmm.qk_norm_rope(x[:, :8], None, q_weight=torch.ones(D, device=DEV))
    assert torch.isnan(y[0, 2]).all() and torch.isnan(y[0, 3, 1]) and torch.isfinite(y[0, [0, 1, 4, 5, 6, 7]]).all()


def test_refusals_of_the_binding():
    x = torch.zeros(4, 6, 64, device=DEV)
    table, pos = torch.zeros(8, 64, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    w = torch.ones(64, device=DEV)
    bad = [dict(rope=table), dict(positions=pos), dict(rope=table, positions=pos[:3]), dict(rope=table[:, :24].contiguous(), positions=pos),
           dict(rope=torch.zeros(8, 80, device=DEV), positions=pos), dict(rope=table[:0], positions=pos),
           dict(q_weight=w[:32].contiguous()), dict(k_weight=w), dict(eps=-1.0), dict(k_out=x),
           dict(q_out=torch.zeros(4, 5, 64, device=DEV)), dict(q_out=x, dtype=F16), dict(q_out=x[:, :, :32])]
    for kw in bad:
        with pytest.raises((ValueError, TypeError)):
            qmm.qk_norm_rope(x, **kw)
    for q in (x.transpose(0, 1), x[:, :, ::2], x[:, ::2], x[:1].expand(4, 6, 64), x.view(4, 384), x[..., :40]):
        with pytest.raises(ValueError):
            qmm.qk_norm_rope(q)
    with pytest.raises(TypeError):
        qmm.qk_norm_rope(x, x.half())
    with pytest.raises(TypeError):
        qmm.qk_norm_rope(x, x, q_weight=w, k_weight=w.half())
    with pytest.raises(ValueError):
        qmm.qk_norm_rope(x, x[:2])
    with pytest.raises(qmm.QmmError):
        qmm.qk_norm_rope(torch.zeros(4 * 64 + 2, device=DEV)[2:].view(4, 1, 64))      # 8-byte aligned
