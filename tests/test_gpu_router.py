"""GPU: moe_router against the float64 oracle.

The ids have to be equal, near ties included.  Tolerance of the weights
(relative): a softmax weight is exp(x - m) of an fp32 difference, whose
rounding is at most |x - m| * 2^-24, two more for exp; the sum over E experts
has positive terms in chains of at most E/4 + 8 additions (any split over four
or more lanes) and inherits the terms' errors, on average at most ln(E) <= 7
for the differences (sum p_i |x_i - m| <= ln E where m is the largest), and
two for exp; division and scale add two.  Sigmoid: exp, addition, division,
then the sum of top_k terms, division and scale.
"""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu


def check(x, top_k, scoring="softmax", bias=None, n_groups=1, topk_groups=None, group_score="max", renormalize=False,
          scale=1.0, dtype=torch.float32):
    x = torch.from_numpy(np.ascontiguousarray(x)).to(dtype)
    T, E = x.shape
    say("moe_router", f"T={T} E={E} top_k={top_k} {scoring} bias={bias is not None} groups={n_groups}/{topk_groups} "
        f"{group_score} renormalize={renormalize} {dtype}")
    ids, w = qmm.moe_router(x.to(DEV), top_k, scoring=scoring, bias=None if bias is None else dev(bias),
                            n_groups=n_groups, topk_groups=topk_groups, group_score=group_score,
                            renormalize=renormalize, scale=scale)
    xf = x.float().numpy()
    i2, w2 = oracle.route(xf, top_k, scoring, bias, n_groups, topk_groups or n_groups, group_score, renormalize, scale)
    ids, w = host(ids), host(w)
    bad = np.argwhere((ids != i2).any(axis=1)).ravel()
    assert not len(bad), f"{len(bad)} rows differ; row {bad[0]}: {ids[bad[0]]} for {i2[bad[0]]}"
    if scoring == "softmax":
        lx = np.take_along_axis(np.nan_to_num(xf, nan=-np.inf), i2.astype(np.int64), 1)
        lx = np.minimum(lx.astype(np.float64), np.finfo(np.float32).max)
        m = lx.max(1, keepdims=True) if renormalize else np.minimum(
            np.where(np.isnan(xf), -np.inf, xf).max(1, keepdims=True), np.finfo(np.float32).max)
        with np.errstate(invalid="ignore"):
            far = np.where(w2 > 0, np.abs(lx - m), 0.0)
        tol = (far + 2 + E / 4 + 8 + 7 + 2 + 2) * 2.0**-24
    else:
        tol = (4 + top_k + 4 + 2) * 2.0**-24
    assert np.all(np.abs(w - w2) <= tol * w2 + 2.0**-126 * abs(scale) * (1 + top_k)), np.abs(w / w2 - 1).max()
    return ids, w


@pytest.mark.parametrize("E,top_k", [(1, 1), (2, 1), (2, 2), (3, 2), (5, 5), (8, 2), (16, 4), (33, 6), (63, 8), (64, 8),
                                     (64, 64), (65, 3), (96, 6), (127, 10), (128, 8), (130, 8), (160, 6), (192, 16),
                                     (255, 9), (256, 8), (257, 64), (320, 12), (384, 6), (511, 32), (512, 10), (512, 64)])
@pytest.mark.parametrize("T", [1, 37])
def test_sizes(T, E, top_k):
    x = qmm_synth.activations(qmm_synth.rng(T + E), T, E) * 1.5
    b = 0.05 * qmm_synth.activations(qmm_synth.rng(E), 1, E)[0]
    check(x, top_k)
    check(x, top_k, "sigmoid", b, renormalize=True, scale=2.5, dtype=torch.bfloat16)
    check(x, top_k, "softmax", b, renormalize=True, dtype=torch.float16)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("E,groups,keep,top_k", [(256, 8, 4, 8), (128, 4, 1, 6), (60, 4, 3, 9), (512, 64, 8, 10),
                                                 (64, 64, 20, 20), (510, 5, 5, 4), (96, 2, 1, 48), (512, 2, 1, 3)])
def test_groups(scoring, with_bias, renormalize, E, groups, keep, top_k):
    x = qmm_synth.activations(qmm_synth.rng(E + keep), 29, E) * 2
    b = 0.1 * qmm_synth.activations(qmm_synth.rng(E), 1, E)[0] if with_bias else None
    for score in ("max", "top2"):
        check(x, top_k, scoring, b, groups, keep, score, renormalize, 1.5, torch.bfloat16)


@pytest.mark.parametrize("T,E", [(1000, 128), (4099, 96), (70000, 8)])
def test_many_tokens(T, E):
    x = qmm_synth.activations(qmm_synth.rng(T), T, E)
    check(x[:1500], min(8, E))
    ids, w = qmm.moe_router(dev(x), min(8, E))
    i2, w2 = qmm.moe_router(dev(x[-1500:]), min(8, E))      # a token's routing does not depend on the others
    assert torch.equal(ids[-1500:], i2) and torch.equal(w[-1500:], w2)
    assert np.array_equal(host(ids)[-1500:], oracle.route(x[-1500:], min(8, E))[0])


@pytest.mark.parametrize("E,groups", [(64, 1), (256, 8), (100, 4), (512, 1)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_equal_values_go_to_the_lower_index(E, groups, scoring):
    g = qmm_synth.rng(E)
    x = g.integers(-2, 3, size=(60, E)).astype(np.float32)       # five different logits
    x[0] = 1.0
    x[1, ::2], x[1, 1::2] = 0.0, -0.0
    b = np.zeros(E, np.float32)
    for score in ("max", "top2"):
        check(x, min(16, E // groups), scoring, None, groups, max(1, groups // 2), score, dtype=torch.bfloat16)
        check(x, min(16, E // groups), scoring, b, groups, max(1, groups // 2), score)
    check(x, 5, scoring, g.integers(-1, 2, size=E).astype(np.float32))


@pytest.mark.parametrize("E,groups", [(128, 1), (256, 8), (384, 1), (512, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_values_closer_than_fp32_resolves(E, groups, scoring):
    # every second expert's bias brings it within an fp32 rounding of its neighbour
    g = qmm_synth.rng(E + 1)
    x = (g.standard_normal((1, E)) * 1.5).astype(np.float32).repeat(8, 0)
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    if scoring == "softmax":
        s = np.exp(x[0].astype(np.float64))
        s /= s.sum()
    b = (0.3 * g.standard_normal(E)).astype(np.float32)
    b[1::2] = (s[0::2] + b[0::2].astype(np.float64) - s[1::2]).astype(np.float32)
    x[1:] = g.permuted(x[1:], axis=1)
    for score in ("max", "top2"):
        check(x, min(32, E // groups), scoring, b, groups, max(1, groups // 2), score, True)
    # the sums of two groups' best within a rounding of each other
    if groups > 1:
        per = E // groups
        y = np.full((4, E), -4.0, np.float32)
        y[:, 0:2], y[:, per:per + 2] = [[0.5, 0.25]], [[0.75, 0.0]]
        y[1, per + 1] = np.log(1 / (1 / (1 + np.exp(-.5)) + 1 / (1 + np.exp(-.25)) - 1 / (1 + np.exp(-.75))) - 1) * -1
        y[2, per + 1] = np.nextafter(y[1, per + 1], np.float32(9))
        y[3, per + 1] = np.nextafter(y[1, per + 1], np.float32(-9))
        check(y, 2, scoring, None, groups, 1, "top2")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_clusters_of_near_ties(scoring):
    # a third of the experts within a few fp32 roundings of one value, from scores of all sizes
    g = qmm_synth.rng(12)
    E = 192
    x = (g.standard_normal((24, E)) * 3).astype(np.float32)
    x[1:] = x[0]
    s = 1 / (1 + np.exp(-x[0].astype(np.float64)))
    if scoring == "softmax":
        s = np.exp(x[0].astype(np.float64))
        s /= s.sum()
    b = (g.standard_normal(E) * 0.1).astype(np.float32)
    b[::3] = (1.25 - s[::3]).astype(np.float32)
    for t in range(1, 24):                       # and the logits a few steps off
        x[t, ::3] = (x[0, ::3].view(np.int32) + g.integers(-3, 4, size=E // 3).astype(np.int32)).view(np.float32)
    for k in (1, 6, 14, 30):
        check(x, k, scoring, b)
        check(x, k, scoring, b, 8, 4, "top2", True)


def test_masks():
    g = qmm_synth.rng(77)
    for E, groups, keep, k in [(128, 1, 1, 8), (64, 8, 3, 20), (10, 2, 1, 5), (512, 1, 1, 64), (300, 4, 2, 12)]:
        x = (g.standard_normal((40, E)) * 2).astype(np.float32)
        x[g.random((40, E)) < 0.6] = -np.inf
        x[0] = -np.inf                                   # nothing left
        x[1, 1:] = -np.inf                               # one left
        x[2] = np.nan
        x[3, :-1] = -np.inf                              # the last one left
        x[4, E // groups:] = -np.inf                     # the first group only
        x[5] = np.finfo(np.float32).min                  # the type's lowest value masks nothing
        x[6, ::3] = np.nan
        b = (g.standard_normal(E)).astype(np.float32)
        for scoring in ("softmax", "sigmoid"):
            for bias in (None, b):
                for renorm in (False, True):
                    for score in ("max", "top2"):
                        ids, w = check(x, k, scoring, bias, groups, keep, score, renorm)
                        assert np.all(w[0] == 0) and np.all(w[2] == 0)
                        assert all(len(set(r)) == k for r in ids.tolist())


def test_extreme_logits():
    g = qmm_synth.rng(5)
    x = (g.standard_normal((12, 96)) * 50).astype(np.float32)
    x[0, 7] = np.inf
    x[1, [3, 90]] = np.inf
    x[2] *= 1e30
    x[3] -= 1e4                                          # sigmoid underflows for all
    x[4, :] = -100.0
    x[5] = -200.0
    x[5, 4] = 88.0
    for renorm in (False, True):
        check(x, 6, "softmax", None, renormalize=renorm)
    check(x[2:], 6, "sigmoid")
    check(x[5:], 6, "softmax", (0.2 * g.standard_normal(96)).astype(np.float32), renormalize=True)
    half = np.clip(x, -65504, 65504)
    check(half, 6, "softmax", dtype=torch.float16)


def test_buffers_and_refusals():
    x = dev(qmm_synth.activations(qmm_synth.rng(2), 6, 64))
    ids, w = qmm.moe_router(x, 4)
    bi = torch.full((9, 4), -5, dtype=torch.int32, device=DEV)
    bw = torch.full((9, 4), -5.0, device=DEV)
    a, b = qmm.moe_router(x, 4, ids=bi[:6], weights=bw[:6])
    assert a.data_ptr() == bi.data_ptr() and b.data_ptr() == bw.data_ptr()
    assert torch.equal(bi[:6], ids) and torch.equal(bw[:6], w) and torch.all(bi[6:] == -5) and torch.all(bw[6:] == -5)
    e = qmm.moe_router(x[:0], 4)
    assert tuple(e[0].shape) == (0, 4) and tuple(e[1].shape) == (0, 4)
    for bad in (lambda: qmm.moe_router(x, 4, scoring="relu"), lambda: qmm.moe_router(x, 4, group_score="sum"),
                lambda: qmm.moe_router(x, 4, bias=torch.zeros(63, device=DEV)),
                lambda: qmm.moe_router(x.t(), 4), lambda: qmm.moe_router(x[:, :32], 4),
                lambda: qmm.moe_router(x, 4, ids=bi), lambda: qmm.moe_router(x, 4, bias=torch.zeros(64))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        qmm.moe_router(x.double(), 4)
    with pytest.raises(TypeError):
        qmm.moe_router(x, 4, bias=torch.zeros(64, dtype=torch.bfloat16, device=DEV))
    for bad in (lambda: qmm.moe_router(x, 0), lambda: qmm.moe_router(x, 65), lambda: qmm.moe_router(x, 4, n_groups=7),
                lambda: qmm.moe_router(x, 9, n_groups=8, topk_groups=1),
                lambda: qmm.moe_router(torch.zeros(1, 513, device=DEV), 4)):
        with pytest.raises(qmm.QmmError):
            bad()


def _near_equal_groups(g, T, groups, scoring):
    """Probabilities or sigmoid scores [T, groups, 2] whose group sums are far apart but for groups 0 and 1 in the
    middle, which are equal but for the logits' rounding; returned as float32 logits [T, 2 * groups]."""
    want = np.empty((T, groups))
    want[:, :2] = g.uniform(0.8, 1.2, size=(T, 1))
    above = (groups - 2) // 2
    want[:, 2:2 + above] = g.uniform(1.5, 1.8, size=(T, above))
    want[:, 2 + above:] = g.uniform(0.1, 0.5, size=(T, groups - 2 - above))
    first = want * g.uniform(0.45, 0.55, size=(T, groups))       # every score below 1
    s = np.stack([first, want - first], -1)
    if scoring == "softmax":
        return np.log(s).reshape(T, -1).astype(np.float32)
    return np.log(s / (1 - s)).reshape(T, -1).astype(np.float32)


@pytest.mark.parametrize("B", [10.0, 30.0, 100.0, 1e3, 1e4])
@pytest.mark.parametrize("groups", [2, 8])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_group_sums_of_biases_that_cancel(B, groups, scoring):
    # a group's two terms c = s + B and s - B are rounded at the size of B, their sum is of the size of s
    x = _near_equal_groups(qmm_synth.rng(int(B) + groups), 1500, groups, scoring)
    b = np.zeros(2 * groups, np.float32)
    b[0::4], b[1::4] = B, -B                             # every second group
    check(x, 2, scoring, b, groups, groups // 2, "top2", True)
    check(x, 1, scoring, -b, groups, groups // 2, "top2", dtype=torch.float32)


def test_group_sums_past_fp32():
    # two biases of the type's lowest value: their sum is below every fp32 value, but above a group that is masked
    low = np.finfo(np.float32).min
    x = np.array([[-np.inf, np.nan, 0.5, 0.25, -np.inf, -np.inf], [0.5, 0.25, 1.0, -1.0, 0.5, 0.5]], np.float32)
    b = np.array([0, 0, low, low, 0, 0], np.float32)
    for scoring in ("softmax", "sigmoid"):
        for keep in (1, 2):
            check(x, 2, scoring, b, 3, keep, "top2")
            check(x, 2, scoring, -b, 3, keep, "top2", True)
        check(x, 2, scoring, np.array([low, 0, low, low, 0, low], np.float32), 3, 1, "max")


@pytest.mark.parametrize("top_k", [4, 20])
@pytest.mark.parametrize("with_bias", [False, True])
def test_sigmoid_shares_of_small_scores(top_k, with_bias):
    # scores below fp32's range, or among its subnormals, still have shares of their sum
    g = qmm_synth.rng(9)
    E = 64
    x = np.empty((14, E), np.float32)
    for i, v in enumerate([-50.0, -79.9, -80.1, -86.0, -88.0, -89.0, -95.0, -100.0, -104.0, -200.0, -700.0]):
        x[i] = v + 0.5 * g.standard_normal(E)
    x[7] = -100.0                                        # all equal
    x[11] = -200.0
    x[11, 4] = 88.0
    x[12] = np.where(np.arange(E) % 2 == 0, -60.0, -101.0)
    x[13] = -100.0
    x[13, 9:] = -np.inf                                  # fewer than top_k = 20 left
    b = (0.1 * g.standard_normal(E)).astype(np.float32) if with_bias else None
    _, w = check(x, top_k, "sigmoid", b, renormalize=True, scale=2.0)
    assert np.allclose(w.sum(1), 2.0, rtol=1e-5)
    check(x, top_k, "sigmoid", b, 4, 3, "top2", True)
    # a token's weights do not depend on its neighbours in the batch
    ids, w = qmm.moe_router(dev(x), top_k, scoring="sigmoid", renormalize=True)
    for t in range(14):
        i1, w1 = qmm.moe_router(dev(x[t:t + 1]), top_k, scoring="sigmoid", renormalize=True)
        assert torch.equal(i1[0], ids[t]) and torch.equal(w1[0], w[t])


@pytest.mark.parametrize("E,groups,keep,top_k", [(8, 1, 1, 8), (8, 1, 1, 6), (6, 2, 1, 3), (64, 1, 1, 6), (96, 8, 2, 14), (512, 4, 3, 9), (100, 1, 1, 40)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_ids_stay_in_range_whatever_the_bias(E, groups, keep, top_k, scoring):
    # ids go on to calls that cannot check them
    g = qmm_synth.rng(E)
    x = dev((g.standard_normal((21, E)) * 2).astype(np.float32))
    x[3, ::2] = -np.inf
    bits = np.array([0x7FC00000, 0xFFC00000, 0xFFFFFFFF, 0xFFFFFE00, 0x7F800001, 0x7F800000, 0xFF800000], np.uint32).view(np.float32)
    for share in (0.1, 0.5, 1.0):
        for one in (None, *range(len(bits))):
            b = (0.1 * g.standard_normal(E)).astype(np.float32)
            odd = g.random(E) < share
            b[odd] = bits[g.integers(0, len(bits), size=odd.sum()) if one is None else one]
            say("moe_router", f"E={E} groups={groups}/{keep} top_k={top_k} {scoring} odd biases {odd.sum()} kind {one}")
            for score in ("max", "top2"):
                ids = torch.full((21, top_k), 1 << 30, dtype=torch.int32, device=DEV)
                qmm.moe_router(x, top_k, scoring=scoring, bias=dev(b), n_groups=groups, topk_groups=keep, group_score=score,
                               renormalize=True, ids=ids)
                ids = host(ids)
                assert ids.min() >= 0 and ids.max() < E and all(len(set(r)) == top_k for r in ids.tolist())
