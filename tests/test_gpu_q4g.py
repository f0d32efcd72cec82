"""GPU: mmvq_q4g against the float64 oracle.

Tolerance: the integer part of a block is exact; its product with the two
scales takes two roundings, and a sum over K/32 blocks in chains of at most
K/512 + 16 additions (any split over 16 or more lanes) as many, each of 2^-24
relative to sum |w||x|.
"""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu


def check(M, K, group, T, zeros=False, dtype=torch.float16, seed=0, out=None):
    g = qmm_synth.rng(seed + M + K + T)
    w, s, z = qmm_synth.q4g_weights(g, M, K, group, zeros)
    xq = oracle.quantize_q8_1(qmm_synth.activations(g, T, K, 0.01))
    say("mmvq_q4g", f"M={M} K={K} group={group} T={T} zeros={zeros} {dtype}")
    y = qmm.mmvq_q4g(dev(w), dev(s).to(dtype), dev(xq), zeros=None if z is None else dev(z), out=out)
    W, X = oracle.q4g_dequant(w, s, z), oracle.q8_1_dequant(xq)
    # without its zero points a block's sum can cancel: the terms q * a and z * sum(a) are exact integers first
    ref, bound = oracle.dense(W, X), oracle.abs_bound(W, X)
    err = np.abs(host(y) - ref)
    assert np.all(err <= (K / 512 + 18) * 2.0**-24 * bound), (err / bound).max() * 2.0**24
    return y


@pytest.mark.parametrize("K,group", [(32, 32), (64, 32), (64, 64), (96, 96), (96, 32), (128, 64), (160, 160), (1024, 64),
                                     (1056, 32), (1056, 352), (1984, 64), (2048, 128), (2080, 32), (2272, 2272),
                                     (4096, 128), (4096, 32), (6144, 96), (8192, 256), (11008, 128), (11008, 32),
                                     (11008, 11008), (14336, 64), (16384, 128), (20000, 32), (28672, 128)])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_lengths_and_groups(K, group, T):
    check(37, K, group, T, zeros=(K // 32 + T) % 2 == 0, dtype=torch.bfloat16 if T == 3 else torch.float16)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("zeros", [False, True])
def test_tokens(T, zeros):
    check(130, 2080, 32, T, zeros)
    check(67, 4096, 128, T, zeros, torch.bfloat16)


@pytest.mark.parametrize("M", [1, 2, 3, 5, 7, 8, 15, 16, 17, 31, 33, 64, 255, 1003, 2048, 4096, 5003])
def test_rows(M):
    check(M, 1024, 64, 1)
    check(M, 672, 32, 4, True)


@pytest.mark.parametrize("M,K,group,T", [(4096, 11008, 128, 1), (4096, 4096, 64, 4), (11008, 4096, 128, 8), (1, 65536, 128, 2),
                                         (3, 131072, 64, 8), (20000, 256, 32, 1)])
def test_large(M, K, group, T):
    check(M, K, group, T, True)


def test_integers_come_out_exactly():
    # scales 1 and activation scales 1: every product and partial sum is an integer below 2^24
    g = qmm_synth.rng(3)
    M, K = 50, 4096
    w = g.integers(0, 256, size=(M, K // 2), dtype=np.uint8)
    x = g.integers(-127, 128, size=(8, K)).astype(np.float32)
    x[:, ::32] = 127
    xq = oracle.quantize_q8_1(x)
    for group, z in ((32, None), (128, g.integers(0, 256, size=(M, K // 256), dtype=np.uint8))):
        s = np.ones((M, K // group), np.float32)
        y = qmm.mmvq_q4g(dev(w), dev(s).half(), dev(xq), zeros=None if z is None else dev(z))
        assert np.array_equal(host(y), oracle.dense(oracle.q4g_dequant(w, s, z), x))


def test_one_hot_rows_return_the_weights():
    g = qmm_synth.rng(4)
    M, K, group = 19, 2080, 160
    w, s, z = qmm_synth.q4g_weights(g, M, K, group, True)
    W = oracle.q4g_dequant(w, s, z)
    at = g.permutation(K)[:64]
    for i in range(0, 64, 8):
        x = np.zeros((8, K), np.float32)
        x[np.arange(8), at[i:i + 8]] = 127.0
        y = qmm.mmvq_q4g(dev(w), dev(s).half(), dev(oracle.quantize_q8_1(x)), zeros=dev(z))
        assert np.array_equal(host(y), 127 * W[:, at[i:i + 8]].T)


def test_repeatable_token_alone_and_buffers():
    g = qmm_synth.rng(6)
    M, K = 300, 4096
    w, s, _ = qmm_synth.q4g_weights(g, M, K, 128)
    w, s = dev(w), dev(s).half()
    xq = dev(oracle.quantize_q8_1(qmm_synth.activations(g, 8, K)))
    y = qmm.mmvq_q4g(w, s, xq)
    assert torch.equal(y, qmm.mmvq_q4g(w, s, xq))
    big = torch.full((9, M), -1.0, device=DEV)
    out = qmm.mmvq_q4g(w, s, xq, out=big[:8])
    assert out.data_ptr() == big.data_ptr() and torch.equal(out, y) and torch.all(big[8] == -1)


def test_refusals():
    w = torch.zeros(4, 128, dtype=torch.uint8, device=DEV)
    s = torch.zeros(4, 8, dtype=torch.float16, device=DEV)
    z = torch.zeros(4, 4, dtype=torch.uint8, device=DEV)
    xq = torch.zeros(1, 8, 40, dtype=torch.uint8, device=DEV)
    qmm.mmvq_q4g(w, s, xq, zeros=z)
    for bad in (lambda: qmm.mmvq_q4g(w, s[:3], xq), lambda: qmm.mmvq_q4g(w, s[:, :3].contiguous(), xq),
                lambda: qmm.mmvq_q4g(w, s.new_zeros(4, 16), xq), lambda: qmm.mmvq_q4g(w, s, xq, zeros=z[:, :3].contiguous()),
                lambda: qmm.mmvq_q4g(w, s, xq[:, :4].contiguous()), lambda: qmm.mmvq_q4g(w[:, ::2], s, xq),
                lambda: qmm.mmvq_q4g(w, s, xq, out=torch.empty(1, 5, device=DEV)),
                lambda: qmm.mmvq_q4g(w, s, xq, zeros=z.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: qmm.mmvq_q4g(w, s.float(), xq), lambda: qmm.mmvq_q4g(w.to(torch.int8), s, xq)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(qmm.QmmError):
        qmm.mmvq_q4g(w, s, xq.repeat(9, 1, 1))
    with pytest.raises(qmm.QmmError):
        qmm.mmvq_q4g(w, s, xq[:0])


def check_tall(M, K, group, T, zeros, dtype=torch.float16):
    """Many rows: copies of 67 different ones in a random order, so that the oracle works out 67."""
    g = qmm_synth.rng(M + K + T)
    w, s, z = qmm_synth.q4g_weights(g, 67, K, group, zeros)
    pick = g.integers(0, 67, size=M)
    xq = oracle.quantize_q8_1(qmm_synth.activations(g, T, K, 0.01))
    say("mmvq_q4g", f"M={M} K={K} group={group} T={T} zeros={zeros} {dtype}")
    at = dev(pick)
    out = torch.full((T * M + 64,), 7.0, device=DEV)
    y = qmm.mmvq_q4g(dev(w)[at], dev(s).to(dtype)[at], dev(xq), zeros=None if z is None else dev(z)[at],
                     out=out[:T * M].view(T, M))
    W, X = oracle.q4g_dequant(w, s, z), oracle.q8_1_dequant(xq)
    ref, bound = oracle.dense(W, X)[:, pick], oracle.abs_bound(W, X)[:, pick]
    assert np.all(np.abs(host(y) - ref) <= (K / 512 + 18) * 2.0**-24 * bound)
    assert torch.all(out[T * M:] == 7)


# two rows per lane: 64 lanes a row from 8192 rows on, 16 from 32768 (of 256 CUs); the last tile is not full
@pytest.mark.parametrize("T", [2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("M,K,group", [(8195, 2048, 128), (32771, 256, 64), (32773, 1056, 32)])
def test_two_rows_per_lane(T, M, K, group):
    check_tall(M, K, group, T, zeros=T % 2 == 0, dtype=torch.bfloat16 if T == 3 else torch.float16)


# activations in segments, and as many rows as leave each wave a whole one: the sums live over the segments
@pytest.mark.parametrize("M,K,group,T", [(2100, 28672, 128, 8), (4099, 20000, 32, 8), (8195, 20000, 160, 8), (4097, 24576, 64, 6),
                                         (2049, 114688, 128, 1), (32771, 16416, 32, 8)])
def test_many_rows_over_segments(M, K, group, T):
    check_tall(M, K, group, T, zeros=M % 2 == 1)


@pytest.mark.parametrize("M,K", [(300, 4096), (8195, 2048), (37, 28672)])
def test_a_token_alone(M, K):
    # other variants than with eight, so within both calls' roundings
    g = qmm_synth.rng(M)
    w, s, z = qmm_synth.q4g_weights(g, 67, K, 128, True)
    at = dev(g.integers(0, 67, size=M))
    wd, sd, zd = dev(w)[at], dev(s).half()[at], dev(z)[at]
    xq = oracle.quantize_q8_1(qmm_synth.activations(g, 8, K))
    y = host(qmm.mmvq_q4g(wd, sd, dev(xq), zeros=zd))
    bound = oracle.abs_bound(oracle.q4g_dequant(w, s, z), oracle.q8_1_dequant(xq))[:, host(at)]
    for t in range(8):
        one = host(qmm.mmvq_q4g(wd, sd, dev(xq[t:t + 1]), zeros=zd))
        assert np.all(np.abs(one[0] - y[t]) <= 2 * (K / 512 + 18) * 2.0**-24 * bound[t])
