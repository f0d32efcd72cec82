"""GPU: attn_q4 where finite inputs stand at the ends of their ranges (inputs and tolerances: _ranges.py)."""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, dev, host, say
from _ranges import compare, ints, levels

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def cached(g, lens, Hk, D, page, key):
    """A cache of the keys key(b, n) [n, Hk, D] and random values; (cache, table, what it holds per sequence)."""
    W = max(1, max(-(-x // page) for x in lens))
    cache = qmm.kv_cache_q4(len(lens) * W, page, Hk, D, DEV)
    table = g.permutation(len(lens) * W).reshape(len(lens), W).astype(np.int32)
    kv = []
    for b, x in enumerate(lens):
        if x == 0:
            kv.append((np.zeros((0, Hk, D)), np.zeros((0, Hk, D))))
            continue
        t = np.arange(x)
        slots = dev(table[b, t // page].astype(np.int64) * page + t % page)
        qmm.kv_append_q4(dev(key(b, x).astype(np.float32)), dev(g.standard_normal((x, Hk, D)).astype(np.float32)), cache, slots)
        kv.append(tuple(host(a) for a in qmm.kv_read_q4(cache, slots, F32)))
    return cache, dev(table), kv


# A key's first block holds its level, the rest 2^15, which the cache holds exactly; the query has one value in the
# first block and one size in the rest.
def far_key(g, n, Hk, D):
    k = np.full((n, Hk, D), 2.0**15)
    k[..., :32] = levels(g, D, n, Hk, 1)
    return k


def far_query(rows, Hq, D, amp):
    q = np.zeros((rows, Hq, D))
    sign = np.where(np.arange(rows * Hq).reshape(rows, Hq) % 3 == 2, -1.0, 1.0)
    q[..., 0], q[..., 32:] = amp, amp * sign[..., None]
    return q


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("scale", [4.0, 7.3, -5.0, 2.0**8, 3.0 * 2.0**12])
@pytest.mark.parametrize("lens,n,Hq,Hk,D,page", [
    ([300, 1, 77], 1, 4, 2, 128, 16),          # whole sequences, with few of them and with many
    ([40, 900] * 40, 1, 8, 4, 64, 32),
    ([1500, 33], 1, 4, 2, 128, 16),            # parts, with one, two and four tiles of rows
    ([1200, 5], 8, 4, 1, 256, 16),
    ([1300, 64], 8, 16, 2, 96, 32),
    ([1100, 0, 3, 600] * 33, 1, 4, 2, 64, 16),  # runs
    ([1100, 40] * 33, 4, 8, 4, 192, 16),
])
def test_cache_scores_far_from_zero(lens, n, Hq, Hk, D, page, scale, xt):
    say("attn_q4 far", f"lens={lens[:4]} B={len(lens)} n={n} Hq={Hq} Hk={Hk} D={D} page={page} q={xt} scale={scale}")
    g = qmm_synth.rng(len(lens) + D)
    cache, table, kv = cached(g, lens, Hk, D, page, lambda b, x: far_key(g, x, Hk, D))
    q = far_query(len(lens) * n, Hq, D, 2.0).reshape(len(lens), n, Hq, D)
    y = qmm.attn_q4(dev(q).to(xt), cache, table, ints(lens), scale=scale, out_dtype=F32)
    for b, x in enumerate(lens[:6]):
        compare(y[b], q[b], *kv[b], float(np.float32(scale)), oracle.visible(n, x, True), 6, 2.0**-11, F32)
    assert torch.isfinite(y).all()


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_cache_one_key(D, xt):
    """One key: its value, whatever the score is.  The term is a power of two, so nothing rounds."""
    g = qmm_synth.rng(D)
    B, n, Hq, Hk = 40, 1, 64, 8
    for W in (1, 70):                          # whole sequences, and runs of them
        cache, table, kv = cached(g, [1] * B, Hk, D, 16, lambda b, x: np.exp2(g.uniform(0, 15, (x, Hk, 1))) * g.standard_normal((x, Hk, D)))
        table = torch.cat([table] * W, 1).contiguous()
        q = dev(np.exp2(g.uniform(0, 13, (B, n, Hq, 1))) * np.clip(g.standard_normal((B, n, Hq, D)), -4, 4)).to(xt)
        for scale in (None, 1.0, 1000.0):
            y = qmm.attn_q4(q, cache, table, ints([1] * B), scale=scale, out_dtype=F32)
            want = dev(np.repeat(np.stack([v for _, v in kv]), Hq // Hk, 2))
            assert torch.equal(y, want), (W, scale, int((y != want).sum()))


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, -3.4e38])
@pytest.mark.parametrize("lens,Hq,D", [([100, 1], 4, 128), ([1500, 33], 4, 64), ([1100, 3, 600] * 44, 4, 64), ([1300], 40, 256)])
def test_cache_scales_near_the_end_of_their_range(lens, Hq, D, scale, xt):
    """Products of zero are scores of zero, and the largest of others takes all."""
    g = qmm_synth.rng(len(lens) + D)
    cache, table, kv = cached(g, lens, 2, D, 16, lambda b, x: np.repeat(g.integers(-3, 4, (x, 2, D // 32)), 32, -1))
    q = np.zeros((len(lens), 1, Hq, D))
    q[:, :, 1::2, 0] = 2.0**-20
    y = qmm.attn_q4(dev(q).to(xt), cache, table, ints(lens), scale=scale, out_dtype=F32)
    for b, x in enumerate(lens[:6]):
        compare(y[b], q[b], *kv[b], scale, oracle.visible(1, x, True), 7, 2.0**-11, F32)
    assert torch.isfinite(y).all()


def test_cache_queries_of_bf16_under_large_scales():
    """A scale whose product with a query's power of two leaves fp32, though the scores do not."""
    g = qmm_synth.rng(20)
    for lens in ([90], [1500]):
        cache, table, kv = cached(g, lens, 2, 64, 16, lambda b, x: np.repeat(g.integers(-3, 4, (x, 2, 2)), 32, -1) * 2.0**-16)
        q = np.zeros((1, 1, 4, 64))
        q[..., 0] = 2.0**121
        q[..., 1::2, 1] = 2.0**115
        y = qmm.attn_q4(dev(q).bfloat16(), cache, table, ints(lens), scale=2.0**20, out_dtype=F32)
        compare(y[0], q[0], *kv[0], 2.0**20, oracle.visible(1, lens[0], True), 7, 2.0**-11, F32)


@pytest.mark.parametrize("L", [70, 1500])
def test_cache_infinite_queries_next_to_large_ones(L):
    """Scores of -inf take no part however large the query's other values are: zeros where all are."""
    g = qmm_synth.rng(L)
    D = 64
    cache, table, kv = cached(g, [L], 1, D, 16, lambda b, x: np.full((x, 1, D), -1.0))
    q = np.zeros((1, 1, 4, D))
    q[..., 0] = np.inf
    q[0, 0, 1:, 1] = (-1e5, -1e30, 3e38)
    for xt in (BF16, F16):
        y = qmm.attn_q4(dev(np.clip(q, -6e4, None) if xt == F16 else q).to(xt), cache, table, ints([L]), out_dtype=F32)
        assert not y.any(), (xt, y[0, 0, :, 0])
