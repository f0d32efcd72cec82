"""Pins of the oracle's rotation, 4-bit cache and attention (no GPU)."""
import numpy as np
import pytest

import oracle


def test_turn_by_known_angles():
    table = np.array([[1, 0, 0, 1], [0, 1, 1, 0], [-1, 1, 0, 0]], np.float32)   # cos, cos, sin, sin of two angles
    x = np.arange(1.0, 6.0).reshape(1, 1, 5)
    # position 0: angles 0 and 90 degrees
    assert np.array_equal(oracle.turn(x, table, np.array([0]), False).ravel(), [1, -4, 3, 2, 5])
    assert np.array_equal(oracle.turn(x, table, np.array([0]), True).ravel(), [1, 2, -4, 3, 5])
    # position 1: 90 and 0; position 2: 180 and 0; others count as the nearest
    assert np.array_equal(oracle.turn(x, table, np.array([1]), False).ravel(), [-3, 2, 1, 4, 5])
    assert np.array_equal(oracle.turn(x, table, np.array([9]), False).ravel(), [-1, 2, -3, 4, 5])
    assert np.array_equal(oracle.turn(x, table, np.array([-4]), False).ravel(), [1, -4, 3, 2, 5])


@pytest.mark.parametrize("interleaved", [False, True])
def test_turn_keeps_scores_of_equal_distances(interleaved):
    g = np.random.default_rng(1)
    table = oracle.rope_table(300, 64).astype(np.float64)
    q, k = g.standard_normal((2, 1, 1, 64))
    def dot(i, j):
        return (oracle.turn(q, table, np.array([i]), interleaved) * oracle.turn(k, table, np.array([j]), interleaved)).sum()
    assert abs(dot(7, 3) - dot(204, 200)) < 1e-4
    assert abs(dot(7, 3) - dot(7, 4)) > 1e-3


def test_q4_blocks_within_half_a_step():
    g = np.random.default_rng(2)
    x = (g.standard_normal((50, 2, 128)) * np.exp(g.standard_normal((50, 2, 128)))).astype(np.float32)
    n, d, m = oracle.q4_blocks(x)
    v = oracle.q4_values(n, d, m).astype(np.float64)
    step = np.repeat(d.astype(np.float64), 32, -1)
    size = np.abs(x).reshape(50, 2, 4, 32).max(-1).repeat(32, -1)
    # half a step; m is off by half a unit of f16, d too (fifteen times at the top), and the value itself
    assert np.all(np.abs(v - x) <= step * 0.5 + 2.0**-11 * size * 2 + 15 * 2.0**-11 * step)
    assert n.max() == 15 and n.min() == 0


def test_q4_blocks_edges():
    x = np.zeros((1, 1, 64), np.float32)
    x[0, 0, :32] = 3.0                                # a constant block
    x[0, 0, 32], x[0, 0, 33], x[0, 0, 34], x[0, 0, 35] = np.nan, np.inf, -np.inf, 1e30
    n, d, m = oracle.q4_blocks(x)
    v = oracle.q4_values(n, d, m)[0, 0].astype(np.float64)
    assert np.all(v[:32] == 3.0) and d[0, 0, 0] == 0
    # the largest: 65536 / 15 = 4369.07, as f16 4368, fifteen times above -32768
    assert np.all(np.isfinite(v)) and v[33] == 15 * 4368 - 32768 and v[34] == -32768 and v[35] == v[33]
    n, d, m = oracle.q4_blocks(np.full((1, 1, 32), -0.0, np.float32))
    assert m.view(np.uint16)[0, 0, 0] == 0


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_cache_places_are_a_bijection(D):
    g = np.random.default_rng(3)
    cache = np.zeros((3, 2, 2, 20 * D), np.uint8)
    slots = g.permutation(96)
    x = g.standard_normal((2, 96, 2, D)).astype(np.float32)
    oracle.cache_store(cache, slots, x[0], x[1])
    k, v = oracle.cache_load(cache, slots)
    assert np.array_equal(k, oracle.q4_values(*oracle.q4_blocks(x[0])))
    assert np.array_equal(v, oracle.q4_values(*oracle.q4_blocks(x[1])))
    before = cache.copy()
    oracle.cache_store(cache, [-1, 96], x[0], x[1])
    assert np.array_equal(cache, before)
    assert not oracle.cache_load(cache, [-1, 96])[0].any()
    # writing one token again changes only its own bytes
    oracle.cache_store(cache, [37], x[1][:1], x[0][:1])
    k2, v2 = oracle.cache_load(cache, slots)
    other = slots != 37
    assert np.array_equal(k2[other], k[other]) and np.array_equal(v2[other], v[other])


def test_cache_bytes_of_one_token():
    D = 64
    cache = np.zeros((1, 1, 1, 20 * D), np.uint8)
    k = np.tile(np.arange(32.0) % 16, 2).astype(np.float32).reshape(1, 1, D)     # codes 0..15 twice, d = 1, m = 0
    oracle.cache_store(cache, [6], k, 15 - k)
    c = cache.ravel()
    # block 1 of token 6, second group of eight codes 8..15: bytes of codes {0, 4, 1, 5} and those two further
    assert list(c[(16 + 6) * 16 + 4:(16 + 6) * 16 + 8]) == [0xA8, 0xEC, 0xB9, 0xFD]
    assert np.array_equal(c[8 * D + (16 + 6) * 4:][:4].view(np.float16), np.array([1, 0], np.float16))
    # token 6 is number 2 of quad 1: second byte; codes 15 - c below and 15 - c above (values 16 apart are equal)
    for col in range(16):
        assert c[10 * D + ((16 + col) * 2 + 1) * 4 + 1] == (15 - col) * 17
    assert np.array_equal(c[18 * D + (2 + 1) * 16:][:16].view(np.float16), np.array([0, 0, 1, 0, 0, 0, 0, 0], np.float16))


def test_attention_closed_forms():
    g = np.random.default_rng(4)
    q, k, v = g.standard_normal((3, 4, 64)), g.standard_normal((5, 1, 64)), g.standard_normal((5, 1, 64))
    seen = np.zeros((3, 5), bool)
    seen[0, 2] = True
    seen[1] = True
    y, _ = oracle.attention(q, k, v, 0.0, seen)
    assert np.allclose(y[0], v[2]) and np.allclose(y[1], v.mean(0)) and not y[2].any()
    v[3] = np.nan
    y, _ = oracle.attention(q, k, v, 0.3, np.arange(5)[None] < np.array([3, 4, 0])[:, None])
    assert np.all(np.isfinite(y[0])) and np.all(np.isnan(y[1]))


def test_visible():
    assert np.array_equal(oracle.visible(2, 4, True), [[1, 1, 1, 0], [1, 1, 1, 1]])
    assert np.array_equal(oracle.visible(2, 4, True, 2), [[0, 1, 1, 0], [0, 0, 1, 1]])
    assert np.array_equal(oracle.visible(3, 1, True), [[0], [0], [1]])
    assert oracle.visible(2, 3, False).all()
