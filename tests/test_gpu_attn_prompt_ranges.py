"""GPU: attn_prompt where finite inputs stand at the ends of their ranges (inputs and tolerances: _ranges.py)."""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _attention import U, allowed
from _gpu import DEV, dev, say
from _ranges import compare, ints, levels

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
TERM = {F16: 2.0**-11, BF16: 2.0**-8}


def far_rows(g, n, H, D, xt):
    """Keys of levels in the first dim, 2^15 in the others."""
    k = np.full((n, H, D), 2.0**15)
    k[..., 0] = levels(g, D, n, H)
    return dev(k).to(xt)


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("scale", [4.0, 7.3, -5.0, 2.0**8, 3.0 * 2.0**12])
@pytest.mark.parametrize("nq,nk,Hq,Hk,D,causal", [
    ([100, 1, 33], [100, 1, 33], 4, 2, 128, True),
    ([700], [700], 2, 1, 64, True),            # many whole tiles
    ([130], [640], 2, 2, 192, False),
    ([90], [500], 1, 1, 256, True),
    ([40], [1700], 4, 2, 128, True),           # split keys
    ([9, 1], [1500, 1], 2, 1, 64, False),
    ([20], [1300], 4, 1, 256, True),
])
def test_prompt_scores_far_from_zero(nq, nk, Hq, Hk, D, causal, scale, xt):
    say("attn_prompt far", f"nq={nq} nk={nk} Hq={Hq} Hk={Hk} D={D} x={xt} scale={scale}")
    g = qmm_synth.rng(sum(nk) + D)
    q = np.zeros((sum(nq), Hq, D))
    q[..., 0] = 2.0
    q[..., 1:] = np.where(np.arange(sum(nq) * Hq).reshape(sum(nq), Hq) % 3 == 2, -2.0, 2.0)[..., None]
    k, v = far_rows(g, sum(nk), Hk, D, xt), dev(g.standard_normal((sum(nk), Hk, D))).to(xt)
    y = qmm.attn_prompt(dev(q).to(xt), k, v, ints(np.r_[0, np.cumsum(nq)]), ints(np.r_[0, np.cumsum(nk)]), causal=causal,
                        scale=scale, out_dtype=F32)
    q0 = k0 = 0
    for n, L in zip(nq, nk):
        compare(y[q0:q0 + n], q[q0:q0 + n], k[k0:k0 + L].double().cpu().numpy(), v[k0:k0 + L].double().cpu().numpy(),
                float(np.float32(scale)), oracle.visible(n, L, causal), 6, TERM[xt], F32)
        q0, k0 = q0 + n, k0 + L


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("first", [60, 64, 100, 128, 160, 200, 256, 330])
def test_prompt_scores_that_leave_and_come_back(first, D, xt):
    """Scores next to zero for the first keys, then far above or below, then next to zero again."""
    g = qmm_synth.rng(first + D)
    L = 700
    k = np.zeros((L, 2, D))
    k[:, 0] = np.where((np.arange(L) >= first) & (np.arange(L) < first + 150), 2.0**15, 0.0)[:, None]
    k[:, 1] = np.where((np.arange(L) >= first) & (np.arange(L) < first + 150), 0.0, 2.0**15)[:, None]
    k[..., 0] = levels(g, D, L, 2)
    q = np.full((L, 4, D), 2.0)
    q[:, 1::2, 1:] = -2.0
    v = dev(g.standard_normal((L, 2, D))).to(xt)
    y = qmm.attn_prompt(dev(q).to(xt), dev(k).to(xt), v, ints([0, L]), scale=9.0, out_dtype=F32)
    compare(y, q, k, v.double().cpu().numpy(), 9.0, oracle.visible(L, L, True), 12, TERM[xt], F32)


@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("D", [64, 96, 128, 256])
def test_prompt_one_key(D, xt):
    """One key: its value, whatever the score is.  The term is a power of two, so nothing rounds."""
    g = qmm_synth.rng(D)
    B, Hq, Hk = 150, 16, 4
    top = 15 if xt == F16 else 50
    size = lambda *s: np.exp2(g.uniform(0, top, (*s, 1))) * np.clip(g.standard_normal((*s, D)), -1.9, 1.9)  # noqa: E731
    q, k, v = (dev(x).to(xt) for x in (size(B, Hq), size(B, Hk), g.standard_normal((B, Hk, D))))
    want = v.repeat_interleave(Hq // Hk, 1).float()
    one = ints(np.arange(B + 1))
    for scale in (None, 1.0, 1000.0):
        y = qmm.attn_prompt(q, k, v, one, scale=scale, out_dtype=F32)
        assert torch.equal(y, want), (scale, int((y != want).sum()))
    # equal keys in every split: the values' mean
    k2 = k[:1].expand(1600, Hk, D).contiguous()
    v2 = dev(g.integers(-8, 9, (1600, Hk, D)).astype(np.float32)).to(xt)
    y = qmm.attn_prompt(q[:7], k2, v2, ints([0, 7]), ints([0, 1600]), causal=False, out_dtype=F32)
    mean = v2.double().mean(0).repeat_interleave(Hq // Hk, 0).expand(7, Hq, D)
    assert torch.all((y.double() - mean).abs() <= 4 * U * mean.abs())      # whole numbers: the quotient alone rounds


# ---------------------------------------------------------------- values near the end of their range

@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("nq,nk,D,causal", [(300, 300, 64, True), (90, 400, 128, False), (70, 200, 256, True),
                                            (40, 1700, 128, True), (3, 3000, 64, False)])
def test_prompt_values_near_the_end_of_their_range(nq, nk, D, causal, xt):
    """An average of finite values is finite, whatever their sum would be."""
    say("attn_prompt large values", f"nq={nq} nk={nk} D={D} x={xt}")
    g = qmm_synth.rng(nk + D)
    top = torch.finfo(xt).max
    q, k = dev(g.standard_normal((nq, 2, D))).to(xt), dev(g.standard_normal((nk, 1, D))).to(xt)
    v = dev(g.standard_normal((nk, 1, D))).to(xt)
    v[..., 0::4], v[..., 1::4] = top, -top
    v[..., 2::4] = dev(np.where(g.random((nk, 1, D // 4)) < 0.5, 1.0, -1.0) * float(top)).to(xt)
    seen = oracle.visible(nq, nk, causal)
    qb, kb, vb = (t.double().cpu().numpy() for t in (q, k, v))
    ref, spread = oracle.attention(qb, kb, vb, D**-0.5, seen)
    tol = allowed(qb, kb, D**-0.5, seen, ref, spread, TERM[xt], F32)
    y = qmm.attn_prompt(q, k, v, ints([0, nq]), ints([0, nk]), causal=causal, out_dtype=F32)
    got = y.double().cpu().numpy()
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - ref) <= tol)
    # in the values' own type too: an average that rounds to the largest number stays that
    z = qmm.attn_prompt(q, k, v, ints([0, nq]), ints([0, nk]), causal=causal)
    whole = torch.as_tensor(seen.any(1), device=DEV)
    assert torch.isfinite(z).all() and torch.all(z[whole][..., 0::4] >= top * (1 - 2.0**-7))


@pytest.mark.parametrize("D", [64, 256])
def test_prompt_values_near_the_end_under_terms_above_one(D):
    """All keys but the first few lie just below the distance at which a maximum is followed."""
    L = 5000
    k = torch.zeros(L, 1, D, dtype=BF16, device=DEV)
    k[70:, 0, 0] = 1.0
    q = torch.zeros(9, 1, D, dtype=BF16, device=DEV)
    q[:, 0, 0] = 5.5                                                    # e^5.5 = 2^7.93
    v = torch.full((L, 1, D), torch.finfo(BF16).max, dtype=BF16, device=DEV)
    y = qmm.attn_prompt(q, k, v, ints([0, 9]), ints([0, L]), scale=1.0, causal=False, out_dtype=F32)
    # the average of equal numbers, by terms rounded alike on both sides: the sums' roundings and the quotient's
    assert torch.all((y.double() - v[0, 0, 0].double()).abs() <= 2 * (L + 64) * U * v[0, 0, 0].double())


# ---------------------------------------------------------------- scales near the end of their range

@pytest.mark.parametrize("xt", [F16, BF16])
@pytest.mark.parametrize("scale", [2.4e38, 3.4e38, -3.4e38])
@pytest.mark.parametrize("nq,nk,D", [(100, 100, 64), (300, 300, 128), (20, 1500, 128), (40, 100, 256)])
def test_prompt_scales_near_the_end_of_their_range(nq, nk, D, scale, xt):
    """Products of zero are scores of zero, and the largest of others takes all."""
    g = qmm_synth.rng(nk + D)
    q = torch.zeros(nq, 2, D, dtype=xt, device=DEV)
    k, v = (dev(g.standard_normal((nk, 1, D))).to(xt) for _ in range(2))
    q[:, 1, 0], k[:, 0, 0] = 2.0**-20, dev(g.integers(-3, 4, nk)).to(xt)
    seen = oracle.visible(nq, nk, True)
    y = qmm.attn_prompt(q, k, v, ints([0, nq]), ints([0, nk]), scale=scale, out_dtype=F32)
    compare(y, q.double().cpu().numpy(), k.double().cpu().numpy(), v.double().cpu().numpy(), scale, seen, 7, TERM[xt], F32)
