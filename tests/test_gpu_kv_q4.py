"""GPU: kv_append_q4 and kv_read_q4, compared byte for byte with the oracle."""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def rows(g, T, Hk, D, xt):
    """k and v as slices of a stacked product's rows, with loud channels."""
    x = qmm_synth.activations(g, T, (3 * Hk + 1) * D, 0.02) * (1 + 4 * (g.random((3 * Hk + 1) * D) < 0.03)).astype(np.float32)
    x = dev(x).to(xt).view(T, 3 * Hk + 1, D)
    return x[:, Hk:2 * Hk], x[:, 2 * Hk:3 * Hk]


def check(T, Hk, D, page, xt=F32, rot=None, interleaved=False, seed=1, slots=None, pages=None, kv=None):
    say("kv_append_q4", f"T={T} Hk={Hk} D={D} page={page} x={xt} rot={rot} interleaved={interleaved}")
    g = qmm_synth.rng(seed)
    rot = D if rot is None else rot
    k, v = rows(g, T, Hk, D, xt) if kv is None else kv
    pages = -(-T // page) + 2 if pages is None else pages
    if slots is None:
        first = int(g.integers(0, page))
        at = g.permutation(pages)
        t = np.arange(T) + first
        slots = at[t // page] * page + t % page
    slots = np.asarray(slots, np.int64)
    table = oracle.rope_table(60, rot) if rot else None
    pos = g.integers(-2, 63, T).astype(np.int32) if rot else None
    start = g.integers(0, 256, (pages, Hk, page // 16, 20 * D)).astype(np.uint8)
    cache = dev(start)
    back = qmm.kv_append_q4(k, v, cache, dev(slots), rope=dev(table) if rot else None, positions=dev(pos) if rot else None,
                            interleaved=interleaved)
    assert back is cache
    kh, vh = (t.float().cpu().numpy() for t in (k, v))
    if rot:
        kh = oracle.turn(kh, table, pos, interleaved)           # in fp32, every operation rounded
    want = start.copy()
    oracle.cache_store(want, slots, kh, vh)
    assert np.array_equal(host(cache), want)
    # and back: the f16 values, exactly
    rk, rv = oracle.cache_load(want, slots)
    for t in (F16, F32, BF16):
        yk, yv = qmm.kv_read_q4(cache, dev(slots), t)
        for y, r in ((yk, rk), (yv, rv)):
            assert y.dtype == t and torch.equal(y.cpu(), torch.from_numpy(r).to(t))
    return cache


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes(D, interleaved):
    check(19, 3, D, 16, seed=D, interleaved=interleaved)
    for rot in (0, 16, D // 2, D - 16):
        check(5, 2, D, 32, BF16, rot, interleaved, seed=D + rot)


@pytest.mark.parametrize("kt", [F32, F16, BF16])
@pytest.mark.parametrize("vt", [F32, F16, BF16])
def test_types_of_each(kt, vt):
    k, v = rows(qmm_synth.rng(4), 21, 3, 96, F32)
    check(21, 3, 96, 16, kv=(k.to(kt), v.to(vt)))


@pytest.mark.parametrize("xt", [F32, F16, BF16])
def test_types_and_pages(xt):
    for page in (16, 48, 64, 256):
        check(131, 1, 128, page, xt, seed=page)
    check(1, 8, 128, 16, xt, seed=2)
    check(70, 5, 64, 16, xt, seed=3)


@pytest.mark.parametrize("T,Hk,D", [(3000, 8, 128), (5000, 5, 64), (2600, 3, 256), (2000, 16, 96)])
def test_many_tokens(T, Hk, D):
    # enough that a wave goes over several heads of a token
    check(T, Hk, D, 64, BF16, seed=T)


def test_slots_in_any_order_and_left_out():
    g = qmm_synth.rng(5)
    slots = g.permutation(96)[:50]
    slots[[3, 17, 40]] = [-1, 96, 2**62]
    check(50, 2, 128, 32, slots=slots, pages=3)
    check(4, 2, 64, 16, slots=[-1, -(2**62), 48, 49], pages=3)      # nothing is written


def test_edge_blocks():
    D = 64
    x = torch.zeros(1, 2, D, device=DEV)
    x[0, 0, :32] = 3.0
    x[0, 0, 40] = float("nan")
    x[0, 0, 41], x[0, 0, 42], x[0, 0, 43] = float("inf"), -1e30, 1e-30
    x[0, 1, :32] = -0.0
    x[0, 1, 32:] = torch.linspace(-1e-7, 1e-7, 32, device=DEV)      # d below the smallest f16
    check(1, 2, D, 16, rot=0, kv=(x, x.flip(1)))
    y = torch.linspace(-1, 1, 2 * D, device=DEV).view(1, 2, D) * 2.0**-14      # f16 subnormal scales
    check(1, 2, D, 16, rot=0, kv=(y, x))
    z = 32768 * torch.sign(torch.linspace(-1, 1.01, 2 * D, device=DEV)).view(1, 2, D).roll(5, 2)
    check(1, 2, D, 16, rot=0, kv=(z, -z))


def test_every_scale():
    """Each positive f16 as d, with values at and beside every half step: the reciprocal's last bit decides there."""
    d = np.arange(1, np.float16(2180).view(np.uint16) + 1, dtype=np.uint16).view(np.float16).astype(np.float32)
    d = np.resize(d, (len(d) + 3) // 4 * 4).reshape(-1, 4, 1)
    n = np.float32(0.5) + np.arange(15, dtype=np.float32)
    x = np.concatenate((0 * d, 15 * d, n * d, np.nextafter(n * d, np.float32(0))), 2)       # 15 d has at most 15 bits
    k, v = (dev(np.ascontiguousarray(x[:, i:i + 2].reshape(-1, 1, 64))) for i in (0, 2))
    check(len(x), 1, 64, 64, rot=0, kv=(k, v))


def test_spans_between_two_scales():
    """Spans whose fifteenth part lies at, just below and just above the middle of two f16 numbers."""
    f = np.arange(0, np.float16(2180).view(np.uint16), dtype=np.uint16)
    mid = (f.view(np.float16).astype(np.float64) + (f + 1).view(np.float16).astype(np.float64)) / 2 * 15
    mid = np.resize(mid, (len(mid) + 1) // 2 * 2).astype(np.float32)
    spans = np.stack((np.nextafter(mid, np.float32(0)), mid, np.nextafter(mid, np.float32(1e9))), 1).reshape(-1, 6)
    x = np.zeros((len(spans), 6, 32), np.float32)
    x[:, :, 5], x[:, :, 9] = spans, spans / 3
    k, v = (dev(x[:, i:i + 2].reshape(-1, 1, 64)) for i in (0, 2))
    check(len(x), 1, 64, 64, rot=0, kv=(k, v))
    k, v = (dev(x[:, i:i + 2].reshape(-1, 1, 64)) for i in (4, 1))
    check(len(x), 1, 64, 64, rot=0, kv=(k, v))


def test_ties_go_to_even_codes():
    # steps of exactly 1, 0 and 15 in the block: every half is a tie
    x = (torch.arange(32, device=DEV) / 2.0).clamp(max=15.0).repeat(1, 2, 2)
    check(1, 2, 64, 16, rot=0, kv=(x.contiguous(), x.contiguous()))


def test_reads_repeat_and_leave_out():
    g = qmm_synth.rng(6)
    cache = dev(g.integers(0, 256, (4, 3, 2, 20 * 96)).astype(np.uint8))
    half = cache.view(torch.float16)
    half[..., 4 * 96:5 * 96] = torch.rand_like(half[..., 4 * 96:5 * 96])     # scales that are numbers
    half[..., 9 * 96:] = torch.rand_like(half[..., 9 * 96:])
    slots = np.array([5, 5, -1, 127, 128, 64, -(2**63), 2**63 - 1, 0], np.int64)
    k, v = oracle.cache_load(host(cache), slots)
    out = [torch.full((12, 3, 96), 9.0, dtype=F16, device=DEV) for _ in range(2)]
    a, b = qmm.kv_read_q4(cache, dev(slots), k=out[0][:9], v=out[1][:9])
    assert np.array_equal(host(a), k) and np.array_equal(host(b), v)
    assert torch.all(out[0][9:] == 9) and torch.all(out[1][9:] == 9)
    assert qmm.kv_read_q4(cache, dev(slots[:0]))[0].shape == (0, 3, 96)


@pytest.mark.parametrize("xt,T", [(BF16, 70000), (F16, 70001), (F32, 33000)])
def test_large_reads_equal_small_ones(xt, T):
    """Outputs past the caches' size are stored another way; the values are the same."""
    Hk, D, page = 8, 128, 48
    g = torch.Generator(device=DEV).manual_seed(5)
    cache = torch.randint(0, 256, (300, Hk, 3, 20 * D), dtype=torch.uint8, device=DEV, generator=g)
    half = cache.view(F16).view(300, Hk, 3, 2, 5 * D)
    half[..., 4 * D:] = torch.rand(300, Hk, 3, 2, D, device=DEV, generator=g).half()       # scales and offsets
    slots = torch.randint(-3, 300 * page + 3, (T,), dtype=torch.int64, device=DEV, generator=g)
    k, v = qmm.kv_read_q4(cache, slots, xt)
    for i in range(0, T, 10000):
        ks, vs = qmm.kv_read_q4(cache, slots[i:i + 10000].clone(), xt)
        assert torch.equal(k[i:i + 10000], ks) and torch.equal(v[i:i + 10000], vs), i


def test_long_cache_offsets_past_32_bits():
    # 5 GB: the last pages lie behind 4 GiB
    D, Hk, page = 128, 8, 64
    pages = (5 << 30) // (Hk * page // 16 * 20 * D)
    cache = qmm.kv_cache_q4(pages, page, Hk, D, DEV)
    assert cache.numel() > 1 << 32
    g = qmm_synth.rng(7)
    k, v = rows(g, 70, Hk, D, BF16)
    slots = (pages - 2) * page + np.arange(70) + 20
    qmm.kv_append_q4(k, v, cache, dev(slots))
    want = np.zeros((2, Hk, page // 16, 20 * D), np.uint8)
    oracle.cache_store(want, slots - (pages - 2) * page, k.float().cpu().numpy(), v.float().cpu().numpy())
    assert np.array_equal(host(cache[-2:]), want)
    assert not cache[:-2].any()
    rk, rv = qmm.kv_read_q4(cache, dev(slots))
    ok, ov = oracle.cache_load(want, slots - (pages - 2) * page)
    assert np.array_equal(host(rk), ok) and np.array_equal(host(rv), ov)


def test_refusals_of_the_binding():
    k = torch.zeros(4, 2, 64, device=DEV)
    cache, slots = qmm.kv_cache_q4(3, 16, 2, 64, DEV), torch.arange(4, device=DEV)
    table, pos = torch.zeros(8, 64, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)
    for a, kw in (((k, k[:3], cache, slots), {}), ((k, k, cache, slots[:3]), {}),
                  ((k, k, cache, slots.int()), {}), ((k[:, :1], k[:, :1], cache, slots), {}),
                  ((k, k, cache[..., :1270], slots), {}), ((k, k, cache.float(), slots), {}),
                  ((k, k, cache, slots), dict(rope=table)), ((k, k, cache, slots), dict(positions=pos)),
                  ((k, k, cache, slots), dict(rope=table, positions=pos.long()))):
        with pytest.raises((ValueError, TypeError)):
            qmm.kv_append_q4(*a, **kw)
    assert not cache.any()
    for a, kw in (((cache, slots.int()), {}), ((cache, slots, torch.float64), {}), ((cache, slots), dict(k=k)),
                  ((cache.view(-1), slots), {})):
        with pytest.raises((ValueError, TypeError)):
            qmm.kv_read_q4(*a, **kw)
