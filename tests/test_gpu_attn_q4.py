"""GPU: attn_q4 against the float64 oracle (the tolerance: _attention.py)."""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _attention import allowed
from _gpu import DEV, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def garbage(g, pages, Hk, page, D):
    """A cache as it may stand after use: random bytes, NaN and infinite scales among them."""
    return g.integers(0, 256, (pages, Hk, page // 16, 20 * D)).astype(np.uint8)


def setup(lens, n, Hq, Hk, D, page, xt, seed, spare=3, amp=1.0):
    g = qmm_synth.rng(seed)
    B = len(lens)
    W = max(1, max(-(-max(0, x) // page) for x in lens))
    pages = sum(-(-max(0, x) // page) for x in lens) + spare
    cache = dev(garbage(g, pages, Hk, page, D))
    free = list(g.permutation(pages))
    table = g.integers(-5, pages + 5, (B, W)).astype(np.int32)      # what is behind a sequence's pages is anything
    kv = []
    for b, x in enumerate(lens):
        slots = np.zeros(max(0, x), np.int64)
        for w in range(-(-max(0, x) // page)):
            table[b, w] = free.pop()
            t = np.arange(w * page, min(x, (w + 1) * page))
            slots[t] = int(table[b, w]) * page + t - w * page
        k = amp * qmm_synth.activations(g, max(0, x), Hk * D, 0.01).reshape(-1, Hk, D)
        v = qmm_synth.activations(g, max(0, x), Hk * D, 0.01).reshape(-1, Hk, D) + 0.3
        if x > 0:
            qmm.kv_append_q4(dev(k.astype(np.float32)), dev(v.astype(np.float32)), cache, dev(slots))
            kv.append(tuple(host(t) for t in qmm.kv_read_q4(cache, dev(slots))))
        else:
            kv.append((np.zeros((0, Hk, D)), np.zeros((0, Hk, D))))
    q = dev(qmm_synth.activations(g, B * n, Hq * D)).to(xt).view(B, n, Hq, D)
    return cache, table, kv, q


def compare(y, q, kv, lens, n, window, scale, yt):
    for b, x in enumerate(lens):
        k, v = kv[b]
        seen = oracle.visible(n, k.shape[0], True, window)
        qb = q[b].double().cpu().numpy()
        ref, spread = oracle.attention(qb, k, v, scale, seen)
        tol = allowed(qb, k, scale, seen, ref, spread, 2.0**-11, yt)
        got = y[b].double().cpu().numpy()
        assert np.all(np.isfinite(got)), (b, x)
        bad = np.abs(got - ref) - tol
        assert np.all(bad <= 0), (b, x, float(bad.max()))
        assert not got[~seen.any(1)].any(), (b, x)


def check(lens, n=1, Hq=8, Hk=2, D=128, page=16, xt=F16, yt=None, window=0, scale=None, seed=1, amp=1.0):
    say("attn_q4", f"lens={lens} n={n} Hq={Hq} Hk={Hk} D={D} page={page} q={xt} y={yt} window={window}")
    yt = yt or xt
    cache, table, kv, q = setup(lens, n, Hq, Hk, D, page, xt, seed, amp=amp)
    y = qmm.attn_q4(q, cache, dev(table), dev(np.array(lens, np.int32)), window=window, scale=scale, out_dtype=yt)
    assert y.dtype == yt and y.shape == q.shape
    compare(y, q, kv, lens, n, window, D**-0.5 if scale is None else scale, yt)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("Hq,Hk", [(4, 4), (6, 2), (8, 1), (15, 1), (14, 2), (40, 1)])
def test_heads(D, Hq, Hk):
    check([77, 1, 200], 1, Hq, Hk, D, seed=D + Hq)


@pytest.mark.parametrize("n", [1, 2, 3, 5, 8])
def test_new_tokens(n):
    check([100, n, n + 1, 3, 33], n, 10, 2, 128, seed=n)
    check([64, 65, 300], n, 3, 3, 64, 32, BF16, seed=n + 10)


@pytest.mark.parametrize("n,Hq", [(1, 16), (2, 8), (4, 8), (8, 8)])
def test_whole_tiles_of_rows(n, Hq):
    for D in (64, 128, 256):
        check([90, n, 35], n, Hq, 1, D, seed=n + D)


def test_very_many_rows():
    check([50, 7], 1, 1024, 1, 64, seed=70)
    check([40, 1500], 8, 520, 2, 64, seed=71)
    check([1200] * 3, 8, 130, 1, 256, 16, BF16, window=60, seed=72)


def test_thousands_of_sequences():
    g = qmm_synth.rng(73)
    check([int(x) for x in g.integers(0, 4, 3000)], 1, 2, 1, 64, seed=73)
    check([0] * 700 + [1100] + [1, 0, 2] * 100 + [0] * 30, 2, 2, 1, 64, seed=74)


@pytest.mark.parametrize("n,Hq", [(8, 32), (8, 16), (4, 20), (5, 7)])
def test_many_rows(n, Hq):
    for D in (64, 128, 256):
        check([150, 9], n, Hq, 1, D, seed=Hq + D)


@pytest.mark.parametrize("x", [1, 2, 15, 16, 17, 31, 32, 33, 47, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_lengths(x):
    check([x], seed=x)
    check([x, 2 * x], 2, 4, 4, 64, 48, BF16, seed=x + 1)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 128, 1024])
def test_pages(page):
    check([500, 31, 1], 1, 8, 4, 128, page, seed=page)


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("yt", [F32, F16, BF16])
def test_types(xt, yt):
    check([300, 20], 2, 8, 2, 96, 16, xt, yt, seed=4)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 256, 10**9])
def test_windows(window):
    check([400, 5, 256], 1, 8, 2, 128, 16, window=window, seed=window % 1000)
    check([400, 5, 256], 5, 4, 2, 64, 32, BF16, window=window, seed=window % 1000 + 1)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_short_sequences_of_a_large_batch(D):
    g = qmm_synth.rng(D)
    check([int(x) for x in g.integers(0, 70, 130)], 1, 4, 2, D, seed=D + 7)
    check([int(x) for x in g.integers(0, 40, 140)], 3, 6, 2, D, 32, BF16, F32, window=9, seed=D + 8)


@pytest.mark.parametrize("n", [1, 4])
def test_long_sequences(n):
    check([5000, 17, 2100], n, 8, 2, 128, 64, seed=30 + n)
    check([9000], n, 4, 1, 64, 16, BF16, seed=31 + n)
    check([6000, 1], n, 4, 2, 64, 16, window=4500, seed=32 + n)


def ragged(B, longest, seed):
    """Lengths of a batch: mostly short ones, empty ones, single tokens, and the longest somewhere inside."""
    g = qmm_synth.rng(seed)
    lens = [int(x) for x in g.integers(0, 200, B)]
    lens[1], lens[B // 3], lens[B // 2], lens[-1] = 1, longest, 0, 0
    return lens


# many sequences whose table allows long ones: equal runs of all sequences' steps, a run over several sequences
@pytest.mark.parametrize("n,Hq,Hk,D,B", [(1, 8, 4, 128, 64), (3, 8, 4, 64, 66), (8, 32, 2, 128, 66), (8, 8, 2, 96, 128),
                                         (2, 4, 2, 256, 130), (8, 10, 1, 192, 100), (1, 1, 1, 64, 300)])
def test_runs_over_many_sequences(n, Hq, Hk, D, B):
    check(ragged(B, 1500, n + B), n, Hq, Hk, D, 16, seed=B + D)
    check(ragged(B, 1100, n + B + 1), n, Hq, Hk, D, 32, BF16, window=150, seed=B + D + 1)


def test_runs_of_equal_and_of_single_sequences():
    check([1030] * 64, 1, 4, 4, 64, seed=40)
    check([0] * 40 + [4000] + [0] * 23, 2, 8, 4, 128, 16, seed=41)   # one sequence over many runs
    check([0] * 63 + [1025], 1, 4, 4, 64, 16, window=3, seed=42)
    check([1] * 63 + [1025], 8, 4, 4, 64, 16, BF16, window=1, seed=43)


def test_runs_where_no_sequence_is_left():
    cache, table, kv, q = setup([1100] * 64, 1, 4, 4, 64, 16, F16, 44)
    for x in (0, -5):
        assert not qmm.attn_q4(q, cache, dev(table), torch.full((64,), x, dtype=torch.int32, device=DEV)).any()


# few sequences: equal parts, with every number of tiles of rows
@pytest.mark.parametrize("n,Hq", [(8, 31), (8, 15), (4, 20), (5, 7), (2, 9)])
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_parts_of_many_rows(n, Hq, D):
    check([1700, 9, 0, 600], n, Hq, 1, D, seed=Hq + D)
    check([1500, 40], n, Hq, 1, D, 32, BF16, window=333, seed=Hq + D + 1)


@pytest.mark.parametrize("n", [1, 8])
def test_widest_windows_see_all(n):
    for window in (2**30 - 1, 2**30, 2**31 - 1):
        check([1, 5, 200], n, 4, 2, 64, 16, window=window, seed=50 + n)
        check([2000, 3], n, 4, 2, 64, 16, window=window, seed=51 + n)


@pytest.mark.parametrize("B,longest,n", [(64, 1100, 1), (3, 3000, 4), (5, 900, 2)])
def test_replays_with_other_lengths(B, longest, n):
    """A graph's cut follows the lengths in memory, not those of its capture."""
    g = qmm_synth.rng(60)
    cache, table, kv, q = setup([longest] * B, n, 4, 4, 64, 16, F16, 61)
    lens, t = torch.zeros(B, dtype=torch.int32, device=DEV), dev(table)
    ws = torch.empty(max(16, qmm.attn_q4_workspace_bytes(B, n, 4, 4, 64, table.shape[1] * 16)), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(q)
    qmm.attn_q4(q, cache, t, lens, out=out, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.attn_q4(q, cache, t, lens, out=out, ws=ws)
    for r in range(5):
        now = [longest] * B if r == 2 else [int(x) for x in g.integers(0, longest + 1, B)]
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        out.fill_(7)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, qmm.attn_q4(q, cache, t, lens)), r
        compare(out[:2], q[:2], [(k[:x], v[:x]) for (k, v), x in zip(kv, now[:2])], now[:2], n, 0, 0.125, F16)


def test_rows_far_apart():
    # a stride of queries that takes the offsets past 32 bits
    stride = (1 << 24) - 8
    B, n = 50, 3
    wide = torch.zeros((B * n, stride), dtype=F16, device=DEV)
    cache, table, kv, q = setup([40] * B, n, 4, 2, 64, 16, F16, 62)
    wide[:, 8:8 + 256] = q.view(B * n, 256)
    far = wide[:, 8:8 + 256].view(B, n, 4, 64)
    lens = torch.full((B,), 40, dtype=torch.int32, device=DEV)
    assert torch.equal(qmm.attn_q4(far, cache, dev(table), lens), qmm.attn_q4(q, cache, dev(table), lens))


def test_rows_that_see_nothing():
    check([0], 1)
    check([0, 5, 0, 2, 1], 4, 6, 2, 64)
    check([-3, 5], 1)                                             # a negative length counts as 0


def test_scales_and_large_scores():
    check([200], scale=0.0, seed=5)
    check([200], scale=-0.3, seed=6)
    check([200, 40], 2, scale=4.0, amp=20.0, seed=7)              # scores of thousands: one key takes all
    check([1000], xt=BF16, amp=30.0, seed=8)


def test_scores_that_rise_and_fall():
    """Keys in the order of their scores, both ways, so that the maximum moves in every step or never."""
    D, L = 128, 700
    g = qmm_synth.rng(9)
    q = dev(qmm_synth.activations(g, 1, 4 * D)).half().view(1, 1, 4, D)
    u = host(q)[0, 0, 0].astype(np.float32)
    u /= np.linalg.norm(u)
    for sign in (1, -1):
        k = (np.linspace(-30, 30, L)[::sign, None] * u + 0.1 * g.standard_normal((L, D))).astype(np.float32).reshape(L, 1, D)
        v = g.standard_normal((L, 1, D)).astype(np.float32)
        cache, slots = qmm.kv_cache_q4(44, 16, 1, D, DEV), dev(np.arange(L))
        qmm.kv_append_q4(dev(k), dev(v), cache, slots)
        kv = [tuple(host(t) for t in qmm.kv_read_q4(cache, slots))]
        table = torch.arange(44, dtype=torch.int32, device=DEV).view(1, 44)
        y = qmm.attn_q4(q, cache, table, torch.tensor([L], dtype=torch.int32, device=DEV))
        compare(y, q, kv, [L], 1, 0, D**-0.5, F16)


def test_queries_of_any_size_in_bf16():
    # beyond f16's range at both ends: the scores have to be those of the bf16 numbers
    D, L = 64, 90
    cache, table, kv, q = setup([L, L, L], 1, 4, 2, D, 16, BF16, 12)
    q = q.float()
    q[0] *= 1e30
    q[1] *= 1e-30
    q[2, :, :, ::2] *= 1e-6
    q = q.bfloat16()
    lens = dev(np.array([L] * 3, np.int32))
    for b, scale in enumerate((1e-30, 1e30, 0.125)):
        y = qmm.attn_q4(q, cache, dev(table), lens, scale=scale, out_dtype=F32)
        k, v = kv[b]
        seen = oracle.visible(1, L, True)
        qb = q[b].double().cpu().numpy()
        ref, spread = oracle.attention(qb, k, v, float(np.float32(scale)), seen)
        tol = allowed(qb, k, scale, seen, ref, spread, 2.0**-11, F32)
        assert np.all(np.abs(y[b].double().cpu().numpy() - ref) <= tol)


def test_queries_that_are_not_finite_stay_alone():
    cache, table, kv, q = setup([60, 60], 2, 8, 2, 128, 16, BF16, 13)
    lens = dev(np.array([60, 60], np.int32))
    good = qmm.attn_q4(q, cache, dev(table), lens)
    q2 = q.clone()
    q2[0, 1, 3, 5] = float("nan")
    q2[1, 0, 2, 7] = float("inf")
    y = qmm.attn_q4(q2, cache, dev(table), lens)
    assert torch.isnan(y[0, 1, 3]).all() and torch.isnan(y[1, 0, 2]).all()
    y[0, 1, 3] = good[0, 1, 3]
    y[1, 0, 2] = good[1, 0, 2]
    assert torch.equal(y, good)


def test_pages_outside_the_cache_are_not_seen():
    lens, page, n = [100, 64], 16, 2
    cache, table, kv, q = setup(lens, n, 4, 2, 64, page, F16, 14)
    table[0, 2], table[0, 5], table[1, 0] = -1, cache.shape[0], 2**31 - 1
    y = qmm.attn_q4(q, cache, dev(table), dev(np.array(lens, np.int32)))
    for b, lost in ((0, (2, 5)), (1, (0,))):
        k, v = kv[b]
        seen = oracle.visible(n, lens[b], True)
        for w in lost:
            seen[:, w * page:(w + 1) * page] = False
        qb = q[b].double().cpu().numpy()
        ref, spread = oracle.attention(qb, k, v, 0.125, seen)
        tol = allowed(qb, k, 0.125, seen, ref, spread, 2.0**-11, F16)
        assert np.all(np.abs(y[b].double().cpu().numpy() - ref) <= tol)
    table[:] = -7
    assert not qmm.attn_q4(q, cache, dev(table), dev(np.array(lens, np.int32))).any()


def test_lengths_past_the_table_count_as_its_end():
    cache, table, kv, q = setup([64, 64], 1, 4, 2, 64, 16, F16, 15)
    a = qmm.attn_q4(q, cache, dev(table), dev(np.array([64, 64], np.int32)))
    b = qmm.attn_q4(q, cache, dev(table), dev(np.array([65, 2**31 - 1], np.int32)))
    assert torch.equal(a, b)


def test_strides_out_buffers_workspace_and_equal_bits():
    lens = [3000, 1, 700]
    cache, table, kv, q = setup(lens, 2, 8, 4, 128, 16, BF16, 16)
    t, l = dev(table), dev(np.array(lens, np.int32))
    y = qmm.attn_q4(q, cache, t, l)
    wide = torch.full((6, 20, 128), 3.0, dtype=BF16, device=DEV)
    wide[:, 4:12] = q.flatten(0, 1)
    ws = torch.full((qmm.attn_q4_workspace_bytes(3, 2, 8, 4, 128, table.shape[1] * 16) + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((5, 2, 8, 128), 9.0, dtype=BF16, device=DEV)
    for _ in range(3):
        z = qmm.attn_q4(wide[:, 4:12].view(3, 2, 8, 128), cache, t, l, out=out[1:4], ws=ws[:-64])
        assert z.data_ptr() == out[1].data_ptr() and torch.equal(z, y)
        out[1:4] = 9
    assert torch.all(out == 9) and torch.all(ws[-64:] == 0xFF)
    one = qmm.attn_q4(q[:, 0].contiguous(), cache, t, l)          # [B, Hq, D]: one token each
    assert torch.equal(one, qmm.attn_q4(q[:, :1].contiguous(), cache, t, l)[:, 0])
    assert qmm.attn_q4(q[:0], cache, t[:0], l[:0]).shape == (0, 2, 8, 128)


def test_cache_past_32_bits():
    D, Hk, page = 128, 8, 64
    pages = (5 << 30) // (Hk * page // 16 * 20 * D)
    cache = qmm.kv_cache_q4(pages, page, Hk, D, DEV)
    g = qmm_synth.rng(17)
    slots = dev((pages - 2) * page + np.arange(100))
    k, v = (dev(qmm_synth.activations(g, 100, Hk * D)).view(100, Hk, D) for _ in range(2))
    qmm.kv_append_q4(k, v, cache, slots)
    kv = [tuple(host(t) for t in qmm.kv_read_q4(cache, slots))]
    q = dev(qmm_synth.activations(g, 1, 16 * D)).half().view(1, 1, 16, D)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=DEV)
    y = qmm.attn_q4(q, cache, table, torch.tensor([100], dtype=torch.int32, device=DEV))
    compare(y, q, kv, [100], 1, 0, D**-0.5, F16)


def test_refusals_of_the_binding():
    cache = qmm.kv_cache_q4(3, 16, 2, 64, DEV)
    q = torch.zeros(2, 1, 4, 64, dtype=F16, device=DEV)
    t, l = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    for a, kw in (((q.float(), cache, t, l), {}), ((q[:, :, :3], cache, t, l), {}), ((q, cache, t[:1], l), {}),
                  ((q, cache, t, l[:1]), {}), ((q, cache, t.long(), l), {}), ((q, cache, t[:, :0], l), {}),
                  ((q[..., :32], cache, t, l), {}), ((q, cache, t, l), dict(out=torch.zeros(2, 4, 64, dtype=F16, device=DEV))),
                  ((q, cache, t, l), dict(out_dtype=torch.float64)), ((q[0, 0], cache, t, l), {})):
        with pytest.raises((ValueError, TypeError)):
            qmm.attn_q4(*a, **kw)
    for kw in (dict(window=-1), dict(scale=float("nan"))):
        with pytest.raises(qmm.QmmError):
            qmm.attn_q4(q, cache, t, l, **kw)
    with pytest.raises(qmm.QmmError):
        qmm.attn_q4(torch.zeros(2, 9, 4, 64, dtype=F16, device=DEV), cache, t, l)
