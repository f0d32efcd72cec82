"""GPU: attn_prompt against the float64 oracle (the tolerance: _attention.py)."""
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
TERM = {F16: 2.0**-11, BF16: 2.0**-8}


def cu(lens, start=0):
    return dev(np.concatenate(([start], start + np.cumsum(lens))).astype(np.int32))


def inputs(nq, nk, Hq, Hk, D, xt, seed, amp=1.0):
    g = qmm_synth.rng(seed)
    q = dev(amp * qmm_synth.activations(g, sum(nq), Hq * D, 0.01)).to(xt).view(-1, Hq, D)
    kv = dev(qmm_synth.activations(g, sum(nk), 3 * Hk * D, 0.01)).to(xt).view(-1, 3 * Hk, D)
    return q, kv[:, :Hk], kv[:, 2 * Hk:]


def compare(y, q, k, v, nq, nk, causal, window, scale, yt, q0=0, k0=0):
    xt = q.dtype
    for n, L in zip(nq, nk):
        qb, kb, vb = (t.double().cpu().numpy() for t in (q[q0:q0 + n], k[k0:k0 + L], v[k0:k0 + L]))
        seen = oracle.visible(n, L, causal, window)
        ref, spread = oracle.attention(qb, kb, vb, scale, seen)
        tol = allowed(qb, kb, scale, seen, ref, spread, TERM[xt], yt)
        got = y[q0:q0 + n].double().cpu().numpy()
        assert np.all(np.isfinite(got)), (n, L)
        bad = np.abs(got - ref) - tol
        assert np.all(bad <= 0), (n, L, float(bad.max()), np.unravel_index(bad.argmax(), bad.shape))
        assert not got[~seen.any(1)].any()
        q0, k0 = q0 + n, k0 + L


def check(nq, nk=None, Hq=4, Hk=2, D=128, xt=BF16, yt=None, causal=True, window=0, scale=None, seed=1, amp=1.0):
    nk = nq if nk is None else nk
    yt = yt or xt
    say("attn_prompt", f"nq={nq} nk={nk} Hq={Hq} Hk={Hk} D={D} x={xt} y={yt} causal={causal} window={window}")
    q, k, v = inputs(nq, nk, Hq, Hk, D, xt, seed, amp)
    y = qmm.attn_prompt(q, k, v, cu(nq), cu(nk), causal=causal, window=window, scale=scale, out_dtype=yt)
    assert y.dtype == yt and y.shape == q.shape
    compare(y, q, k, v, nq, nk, causal, window, float(D**-0.5 if scale is None else scale), yt)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("causal", [True, False])
def test_head_sizes(D, xt, causal):
    check([70, 1, 33], Hq=4, Hk=2, D=D, xt=xt, causal=causal, seed=D)
    check([150], [300], Hq=3, Hk=3, D=D, xt=xt, causal=causal, seed=D + 1)


@pytest.mark.parametrize("x", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 95, 127, 128, 129, 191, 193, 255, 256, 257])
def test_lengths(x):
    check([x], Hq=2, Hk=1, seed=x)
    check([x], Hq=2, Hk=1, causal=False, xt=F16, D=64, seed=x + 1)
    check([min(x, 40)], [x + 7], Hq=2, Hk=1, seed=x + 2)


@pytest.mark.parametrize("Hq,Hk", [(1, 1), (5, 5), (6, 2), (8, 1), (7, 1), (16, 4)])
def test_grouped_heads(Hq, Hk):
    check([40, 90], Hq=Hq, Hk=Hk, D=64, seed=Hq)
    check([3], [500], Hq=Hq, Hk=Hk, D=128, xt=F16, seed=Hq + 1)


def test_packed_sequences_of_many_lengths():
    check([1, 17, 130, 0, 64, 5, 0, 200, 1], Hq=4, Hk=1, D=64, seed=2)
    check([1] * 70 + [3] * 30 + [0] * 40 + [9], Hq=2, Hk=2, D=64, xt=F16, seed=3)
    check([10, 1, 100], [300, 64, 100], Hq=4, Hk=2, seed=4)


def test_groups_wider_than_a_tile():
    check([3, 2, 1], Hq=200, Hk=1, D=64, seed=40)
    check([2], [700], Hq=300, Hk=2, D=64, xt=F16, seed=41)
    check([2], [600], Hq=1024, Hk=1, D=64, window=70, seed=42)


def test_thousands_of_sequences():
    g = qmm_synth.rng(43)
    check([int(x) for x in g.integers(0, 3, 3000)], Hq=2, Hk=1, D=64, seed=43)
    check([0] * 2500 + [70] + [0] * 300 + [1], Hq=2, Hk=1, D=64, xt=F16, seed=44)


@pytest.mark.parametrize("yt", [F32, F16, BF16])
@pytest.mark.parametrize("xt", [F16, BF16])
def test_types(xt, yt):
    check([100], Hq=2, Hk=1, D=96, xt=xt, yt=yt, seed=5)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 10**9])
def test_windows(window):
    check([300], Hq=2, Hk=1, D=64, window=window, seed=window % 999)
    check([130, 20], [400, 20], Hq=2, Hk=2, D=128, xt=F16, window=window, seed=window % 999 + 1)


def test_rows_that_see_nothing():
    check([40], [10], Hq=2, Hk=1, seed=6)               # the first 30 queries stand before the first key
    check([200, 100], [70, 0], Hq=2, Hk=1, D=64, seed=7)
    check([5, 7], [0, 0], Hq=2, Hk=1, D=64, seed=8)
    check([50, 3], [0, 9], Hq=2, Hk=1, D=64, causal=False, seed=9)
    q = torch.ones(4, 2, 64, dtype=F16, device=DEV)
    none = torch.empty(0, 1, 64, dtype=F16, device=DEV)
    assert not qmm.attn_prompt(q, none, none, cu([4]), cu([0])).any()


# few rows and many keys: the keys of a tile are split and joined
@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
@pytest.mark.parametrize("xt", [F16, BF16])
def test_split_keys(D, xt):
    check([40], [1700], Hq=4, Hk=2, D=D, xt=xt, seed=D)
    check([40], [1700], Hq=4, Hk=1, D=D, xt=xt, causal=False, seed=D + 1)
    check([1], [2100], Hq=6, Hk=2, D=D, xt=xt, seed=D + 2)
    check([150], [1030], Hq=2, Hk=2, D=D, xt=xt, yt=F32, window=200, seed=D + 3)      # most splits see nothing


def test_split_keys_of_packed_sequences():
    check([30, 1, 0, 50, 7], [1500, 700, 900, 2000, 0], Hq=4, Hk=2, D=128, seed=22)
    check([30, 1, 0, 50, 7], [0, 700, 900, 20, 3000], Hq=2, Hk=1, D=64, xt=F16, causal=False, seed=23)
    check([200, 3, 90], [100, 1500, 900], Hq=2, Hk=1, D=64, window=77, seed=24)       # some rows see nothing
    check([300, 300], [1100, 1], Hq=1, Hk=1, D=192, xt=F16, seed=25)


def test_split_rows_that_see_nothing():
    q, k, v = inputs([700], [2000], 1, 1, 64, F16, 26)
    for ends in ((600, 600, 1500), (700, 0, 2000)):
        y = qmm.attn_prompt(q, k, v, cu([ends[0], 700 - ends[0]]), cu([ends[1], ends[2] - ends[1]]))
        compare(y, q, k, v, [ends[0], 700 - ends[0]], [ends[1], ends[2] - ends[1]], True, 0, 0.125, F16)
    assert not qmm.attn_prompt(q, k, v, cu([700]), cu([0])).any()


@pytest.mark.parametrize("D,xt", [(64, BF16), (128, F16), (256, BF16)])
def test_split_keys_that_are_not_seen_have_no_influence(D, xt):
    n, L = 20, 1300
    q, k, v = inputs([n], [L], 4, 2, D, xt, 27)
    nan, inf = float("nan"), float("inf")
    for window in (0, 300):
        clean = qmm.attn_prompt(q, k, v, cu([n]), cu([L]), window=window)
        for cut in (L - n, L - 7, L - 1):
            k2, v2 = k.clone(), v.clone()
            k2[cut + 1:, :, ::3], v2[cut + 1:, :, 1::2] = nan, inf
            y = qmm.attn_prompt(q, k2, v2, cu([n]), cu([L]), window=window)
            assert torch.equal(y[:cut + 1 - (L - n)], clean[:cut + 1 - (L - n)]), (window, cut)
            if window:
                k2[:L - n - window + 1], v2[:L - n - window + 1] = inf, nan
                y = qmm.attn_prompt(q, k2, v2, cu([n]), cu([L]), window=window)
                assert torch.equal(y[:cut + 1 - (L - n)], clean[:cut + 1 - (L - n)]), (window, cut)
    # what is seen shows, from any split; the scale makes terms of about one size
    for at in (5, L // 2, L - n):
        v2 = v.clone()
        v2[at, 0, 3], v2[at, 1, 7] = inf, -inf
        y = qmm.attn_prompt(q, k, v2, cu([n]), cu([L]), scale=1e-3)
        assert torch.all(y[:, :2, 3] == inf) and torch.all(y[:, 2:, 7] == -inf), at
    v2 = v.clone()
    v2[5, 0, 3], v2[900, 1, 7] = inf, nan
    clean, y = qmm.attn_prompt(q, k, v, cu([n]), cu([L])), qmm.attn_prompt(q, k, v2, cu([n]), cu([L]))
    assert torch.isnan(y[:, 2:, 7]).all() and not torch.isfinite(y[:, :2, 3]).any()
    y[:, :2, 3], y[:, 2:, 7] = clean[:, :2, 3], clean[:, 2:, 7]
    assert torch.equal(y, clean)


def test_split_rows_outside_workspace_and_replays():
    nq, nk, Hq, Hk, D = [40, 25], [1400, 700], 4, 2, 128
    q, k, v = inputs([100], [2200], Hq, Hk, D, BF16, 28)
    cq, ck = cu(nq, 10), cu(nk, 30)
    need = qmm.attn_prompt_workspace_bytes(2, 100, 2200, Hq, Hk, D)
    assert need > 0
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full((101, Hq, D), 7.0, dtype=BF16, device=DEV)
    qmm.attn_prompt(q, k, v, cq, ck, out=out[:100], ws=ws[:-64])
    compare(out, q, k, v, nq, nk, True, 0, D**-0.5, BF16, 10, 30)
    assert torch.all(out[:10] == 7) and torch.all(out[75:] == 7) and torch.all(ws[-64:] == 0xFF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qmm.attn_prompt(q, k, v, cq, ck, out=out[:100], ws=ws[:-64])
    for r in range(4):
        # other bounds of the sequences between replays
        nq, nk = [[40, 25], [0, 90], [60, 1], [33, 33]][r], [[1400, 700], [10, 2100], [2000, 0], [60, 1800]][r]
        cq.copy_(cu(nq, 10))
        ck.copy_(cu(nk, 30))
        out.fill_(7)
        ws[:-64] = 0xFF
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        compare(out, q, k, v, nq, nk, True, 0, D**-0.5, BF16, 10, 30)
        assert torch.all(out[:10] == 7) and torch.all(out[10 + sum(nq):] == 7) and torch.all(ws[-64:] == 0xFF)


def test_scales_next_to_zero():
    # terms of all keys alike, whether the keys are split or not: the scale's products vanish
    for nq, nk in (([70], [70]), ([20], [1500])):
        for scale in (1e-38, -1e-42, 2.0**-149):
            check(nq, nk, Hq=2, Hk=1, D=64, scale=scale, seed=29)
            check(nq, nk, Hq=2, Hk=1, D=64, xt=F16, scale=scale, seed=30)


def test_widest_windows_see_all():
    for window in (2**30 - 1, 2**30, 2**31 - 1):
        check([150], [40], Hq=2, Hk=1, D=64, window=window, seed=31)
        check([3, 40], [700, 1500], Hq=2, Hk=1, D=64, window=window, seed=32)


def test_rows_far_apart():
    # strides that take the offsets past 32 bits
    stride, n = (1 << 24) - 8, 140
    q, k, v = inputs([n], [n], 4, 2, 64, BF16, 33)
    wide = torch.zeros((n, stride), dtype=BF16, device=DEV)
    wide[:, 8:264], wide[:, 4096:4224], wide[:, stride - 128:] = q.reshape(n, 256), k.reshape(n, 128), v.reshape(n, 128)
    far = (wide[:, 8:264].view(n, 4, 64), wide[:, 4096:4224].view(n, 2, 64), wide[:, stride - 128:].view(n, 2, 64))
    assert torch.equal(qmm.attn_prompt(*far, cu([60, 80])), qmm.attn_prompt(q, k, v, cu([60, 80])))


def test_long_prompts():
    check([1100], Hq=2, Hk=1, D=128, seed=10)
    check([700, 333], Hq=2, Hk=2, D=64, xt=F16, seed=11)
    check([600], Hq=1, Hk=1, D=256, seed=12)


def test_scales_and_large_scores():
    check([100], Hq=2, Hk=1, scale=0.0, seed=13)
    check([100], Hq=2, Hk=1, scale=-0.2, seed=14)
    check([200], Hq=2, Hk=1, scale=3.0, amp=10.0, seed=15)
    check([200], Hq=2, Hk=1, xt=F16, scale=3.0, amp=10.0, seed=16)


@pytest.mark.parametrize("sign", [1, -1])
def test_scores_that_rise_and_fall(sign):
    D, L = 128, 500
    g = qmm_synth.rng(17)
    u = g.standard_normal(D).astype(np.float32)
    u /= np.linalg.norm(u)
    q = dev((20 * u + 0.1 * g.standard_normal((L, 1, D))).astype(np.float32)).bfloat16()
    k = dev((np.linspace(-25, 25, L)[::sign, None, None] * u + 0.1 * g.standard_normal((L, 1, D))).astype(np.float32)).bfloat16()
    v = dev(g.standard_normal((L, 1, D)).astype(np.float32)).bfloat16()
    y = qmm.attn_prompt(q, k, v, cu([L]))
    compare(y, q, k, v, [L], [L], True, 0, D**-0.5, BF16)


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 192])
def test_what_is_not_seen_has_no_influence(xt, D):
    # rows behind the sequences, later keys and keys before the window hold NaN and infinities
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=xt, device=DEV)
    n = 90
    q, k, v = inputs([n], [n], 4, 2, D, xt, 18)
    for window in (0, 20):
        for cut in (0, 30, 31, 32, 63, 64, 65, 89):
            clean = qmm.attn_prompt(q, k, v, cu([n]), window=window)
            k2, v2 = k.clone(), v.clone()
            k2[cut + 1:, :, ::3] = bad[torch.arange(n - cut - 1, device=DEV) % 3][:, None, None]
            v2[cut + 1:, :, 1::2] = bad[torch.arange(n - cut - 1, device=DEV) % 3][:, None, None]
            y = qmm.attn_prompt(q, k2, v2, cu([n]), window=window)
            assert torch.equal(y[:cut + 1], clean[:cut + 1]), (window, cut)
            if window:
                k3, v3 = k.clone(), v.clone()
                k3[:cut], v3[:cut] = bad[0], bad[1]
                y = qmm.attn_prompt(q, k3, v3, cu([n]), window=window)
                if cut + window - 1 < n:
                    assert torch.equal(y[cut + window - 1:], clean[cut + window - 1:]), (window, cut)
    # other sequences' rows
    y = qmm.attn_prompt(q, k, v, cu([20, 30, 40]))
    k2, v2, q2 = k.clone(), v.clone(), q.clone()
    k2[:20], v2[50:], q2[50:] = bad[0], bad[0], bad[1]
    z = qmm.attn_prompt(q2, k2, v2, cu([20, 30, 40]))
    assert torch.equal(z[20:50], y[20:50])


def test_what_is_seen_and_not_finite():
    n, D = 70, 64
    q, k, v = inputs([n], [n], 2, 1, D, BF16, 19)
    v2 = v.clone()
    v2[40, 0, 3], v2[50, 0, 7] = float("inf"), float("nan")
    y, clean = qmm.attn_prompt(q, k, v2, cu([n])), qmm.attn_prompt(q, k, v, cu([n]))
    assert torch.equal(y[:40], clean[:40])
    assert torch.all(y[40:, :, 3] == float("inf")) and torch.isnan(y[50:, :, 7]).all()
    keep = torch.ones(D, dtype=torch.bool, device=DEV)
    keep[[3, 7]] = False
    assert torch.equal(y[..., keep], clean[..., keep])
    k2 = k.clone()
    k2[40] = float("nan")
    y = qmm.attn_prompt(q, k2, v, cu([n]))
    assert torch.equal(y[:40], clean[:40]) and torch.isnan(y[40:]).all()
    # scores of -inf take no part; where all are, the row gives zeros
    q3, k3 = torch.ones_like(q), torch.ones_like(k)
    k3[::2, 0, 0] = -float("inf")
    y = qmm.attn_prompt(q3, k3, v, cu([n]), out_dtype=F32)
    assert not y[0].any()
    odd = v[1::2, 0].float()
    mean = odd.cumsum(0) / torch.arange(1, odd.shape[0] + 1, device=DEV)[:, None]
    # equal terms: each is exact in 16 bits, so only the sums and the quotient round
    assert torch.all((y[1::2] - mean[:, None]).abs() <= 80 * 2.0**-24 * odd.abs().max())


def test_strides_out_buffers_rows_outside_and_equal_bits():
    nq, Hq, Hk, D = [30, 70], 4, 2, 128
    q, k, v = inputs(nq, nq, Hq, Hk, D, F16, 20)
    y = qmm.attn_prompt(q, k, v, cu(nq))
    assert torch.equal(y, qmm.attn_prompt(q.contiguous(), k.contiguous(), v.contiguous(), cu(nq), cu(nq)))
    wide = torch.full((120, Hq + 2 * Hk + 1, D), float("nan"), dtype=F16, device=DEV)
    wide[10:110, :Hq], wide[10:110, Hq:Hq + Hk], wide[10:110, Hq + Hk:Hq + 2 * Hk] = q, k, v
    out = torch.full((122, Hq, D), 7.0, dtype=F16, device=DEV)
    for _ in range(3):
        z = qmm.attn_prompt(wide[:, :Hq], wide[:, Hq:Hq + Hk], wide[:, Hq + Hk:Hq + 2 * Hk], cu(nq, 10), out=out[:120])
        assert torch.equal(z[10:110], y)
        out[10:110] = 7
        assert torch.all(out == 7)
    assert qmm.attn_prompt(q[:0], k, v, cu([0]), cu([100])).shape == (0, Hq, D)


def test_sequence_bounds_outside_the_rows_touch_nothing():
    q, k, v = inputs([50], [50], 2, 1, 64, BF16, 21)
    out = torch.full((50, 2, 64), 7.0, dtype=BF16, device=DEV)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    y = qmm.attn_prompt(q, k, v, i(0, 20), i(0, 20))
    z = qmm.attn_prompt(q, k, v, i(0, 20, 2**31 - 1), i(0, 20, 2**31 - 1), out=out)
    assert torch.equal(z[:20], y[:20])
    qmm.attn_prompt(q, k, v, i(60, 90, 100), i(-40, 2**31 - 1, 5), out=out)
    qmm.attn_prompt(q, k, v, i(-2**31, 2**31 - 1, 10), i(2**31 - 1, -2**31, 7), out=out)
    torch.cuda.synchronize()


def test_refusals_of_the_binding():
    q, k = torch.zeros(6, 4, 64, dtype=F16, device=DEV), torch.zeros(6, 2, 64, dtype=F16, device=DEV)
    c = cu([6])
    for a, kw in (((q.float(), k.float(), k.float(), c), {}), ((q, k.bfloat16(), k, c), {}), ((q, k, k[:5], c), {}),
                  ((q, k[:, :, :32], k, c), {}), ((q[:, :3], k, k, c), {}), ((q, k, k, c.long()), {}), ((q, k, k, c[:0]), {}),
                  ((q, k, k, c, c[:1]), {}), ((q, k, k, c), dict(out=q[:5])), ((q, k, k, c), dict(out_dtype=torch.int8)),
                  ((q.transpose(0, 1), k, k, c), {})):
        with pytest.raises((ValueError, TypeError)):
            qmm.attn_prompt(*a, **kw)
    for kw in (dict(window=-1), dict(window=3, causal=False), dict(scale=float("inf"))):
        with pytest.raises(qmm.QmmError):
            qmm.attn_prompt(q, k, k, c, **kw)
