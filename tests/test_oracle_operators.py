"""Pins for the oracle's norm, routing and group-scaled weights (CPU only), and the
plain forms of perf/operators.py against them on small inputs."""
import importlib.util
import math
import os

import numpy as np
import pytest
import torch

import oracle
import qmm_synth

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_rms_norm_closed_forms():
    h = np.array([[3.0, -4.0], [0.0, 0.0]])
    # mean square of (3, -4) is 12.5
    got = oracle.rms_norm(h, np.array([1.0, 2.0]), 0.0)
    assert np.allclose(got[0], [3 / math.sqrt(12.5), -8 / math.sqrt(12.5)], rtol=1e-15)
    assert np.all(oracle.rms_norm(h, np.ones(2), 1e-6)[1] == 0)
    # an offset is added to the weights; a scaled row has the same norm without eps
    assert np.allclose(oracle.rms_norm(h[:1], np.array([0.0, 1.0]), 0.0, 1.0), got[:1])
    assert np.allclose(oracle.rms_norm(h[:1] * 1e3, np.array([1.0, 2.0]), 0.0), got[:1])


def test_route_by_hand():
    x = np.log(np.array([[1.0, 4.0, 2.0, 3.0]]))        # softmax: .1 .4 .2 .3
    ids, w = oracle.route(x, 2)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[0.4, 0.3]])
    ids, w = oracle.route(x, 2, renormalize=True, scale=7.0)
    assert np.allclose(w, [[4.0, 3.0]])
    ids, w = oracle.route(x, 2, bias=np.array([0.5, 0, 0, 0]))
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.1, 0.4]])   # the bias selects, the weights have none
    ids, w = oracle.route(x, 2, n_groups=2, topk_groups=1, group_score="top2")
    assert ids.tolist() == [[1, 0]]                                    # .1 + .4 = .2 + .3: the first group
    ids, w = oracle.route(np.zeros((1, 4)), 3, scoring="sigmoid")
    assert ids.tolist() == [[0, 1, 2]] and np.all(w == 0.5)
    ids, w = oracle.route(np.array([[-np.inf, 1.0, np.nan, -np.inf]]), 3)
    assert ids.tolist() == [[1, 0, 2]] and w.tolist() == [[1.0, 0.0, 0.0]]
    ids, w = oracle.route(np.full((1, 4), -np.inf), 2, scoring="sigmoid", renormalize=True)
    assert ids.tolist() == [[0, 1]] and not w.any()
    # a masked expert stays masked whatever its bias, and its group counts the others only
    ids, w = oracle.route(np.array([[-np.inf, 1.0, 0.5, 0.0]]), 1, bias=np.array([9.0, 0, 0, 0]), n_groups=2, topk_groups=1)
    assert ids.tolist() == [[1]]


def test_route_agrees_with_the_router_generator():
    g1, g2 = qmm_synth.rng(4), qmm_synth.rng(4)
    ids, probs = qmm_synth.router(g1, 64, 128, 8)
    logits = g2.standard_normal(size=(64, 128))
    i2, w2 = oracle.route(logits, 8)
    assert np.array_equal(ids, i2) and np.allclose(probs, w2, rtol=1e-6)


def test_q4g_dequant_by_hand():
    w = np.zeros((1, 48), np.uint8)
    w[0, 0], w[0, 16], w[0, 47] = 0xA3, 0x0F, 0xF0      # values 0, 1 of group 0; 0 of group 1; 31 of group 2
    s = np.array([[2.0, -1.0, 0.5]])
    got = oracle.q4g_dequant(w, s)
    assert got[0, 0] == (3 - 8) * 2 and got[0, 1] == (10 - 8) * 2 and got[0, 2] == -16
    assert got[0, 32] == -(15 - 8) and got[0, 33] == 8 and got[0, 95] == 3.5 and got[0, 94] == -4
    got = oracle.q4g_dequant(w, s, np.array([[0x21, 0xF7]], np.uint8))    # zero points 1, 2, 7 (and one unused)
    assert got[0, 0] == 4 and got[0, 32] == -13 and got[0, 95] == 4 and got[0, 94] == -3.5


@pytest.fixture(scope="module")
def cases():
    spec = importlib.util.spec_from_file_location("perf_operators", os.path.join(ROOT, "perf", "operators.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.DEVICE = "cpu"
    return m


def test_plain_norm_is_the_oracles(cases):
    s = cases.prepare({"op": "norm", "T": 5, "K": 96, "x": "f32", "res": "f32", "w": "f32", "y": "f32", "offset": 1.0,
                       "eps": 1e-6}, 3)
    values, res, n = cases.run(s)
    assert torch.equal(res, s["x"] + s["res"])
    ref = oracle.rms_norm(res.numpy(), s["w"].numpy(), 1e-6, 1.0)
    assert np.all(np.abs(n.numpy() - ref) <= 24 * 2.0**-24 * np.abs(ref))
    back = oracle.q8_1_dequant(oracle.quantize_q8_1(n.numpy()))
    assert np.array_equal(values.numpy(), back.astype(np.float16))


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias,groups,keep,score", [(False, 1, 1, "max"), (True, 1, 1, "max"), (False, 4, 2, "top2"),
                                                    (True, 4, 3, "top2"), (True, 4, 1, "max")])
def test_plain_route_is_the_oracles(cases, scoring, bias, groups, keep, score):
    c = {"op": "route", "T": 40, "E": 24, "top_k": 5, "x": "bf16", "scoring": scoring, "bias": bias, "groups": groups,
         "keep": keep, "group_score": score, "renorm": bias, "scale": 1.5, "masked": True}
    s = cases.prepare(c, 8)
    ids, w = cases.run(s)
    i2, w2 = oracle.route(s["logits"].float().numpy(), 5, scoring, s["bias"].numpy() if bias else None, groups, keep,
                          score, bias, 1.5)
    assert np.array_equal(ids.numpy(), i2)
    assert np.all(np.abs(w.numpy() - w2) <= 40 * 2.0**-24 * w2)


@pytest.mark.parametrize("zeros", [False, True])
def test_plain_matvec_is_the_oracles(cases, zeros):
    s = cases.prepare({"op": "matvec", "T": 3, "M": 7, "K": 192, "group": 64, "scale": "bf16", "zeros": zeros}, 2)
    W = oracle.q4g_dequant(s["w"].numpy(), s["scales"].float().numpy(), s["zeros"].numpy() if zeros else None)
    X = oracle.q8_1_dequant(s["xq"].numpy())
    assert np.all(np.abs(cases.run(s).numpy() - oracle.dense(W, X)) <= 200 * 2.0**-24 * oracle.abs_bound(W, X))
