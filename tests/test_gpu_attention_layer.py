"""The attention half of a decoder layer as it is called: norm -> stacked q, k, v
product -> norm and rotation of the heads -> append to the cache -> attention
over a prompt, then over the cache for new tokens -> output product.

Every stage is compared with the oracle on the inputs that the GPU's own
earlier stages gave it, and runs are captured and replayed, on two streams at
once, and over a batch padded with sequences that have ended.
"""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _attention import allowed
from _gpu import DEV, assert_parity, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
H, HQ, HK, D, PAGE, PAGES, P = 512, 6, 2, 64, 16, 40, 400
N = (HQ + 2 * HK) * D


class Layer:
    def __init__(self, seed):
        g = qmm_synth.rng(seed)
        self.w = qmm_synth.q4k_weights(g, N, H)
        self.wo = qmm_synth.q4g_weights(g, H, HQ * D, 64)
        self.wd, self.norm = dev(self.w), torch.ones(H, device=DEV)
        self.od = [dev(self.wo[0]), dev(self.wo[1]).half()]
        self.wq, self.wk = (dev(1 + 0.1 * g.standard_normal(D).astype(np.float32)) for _ in range(2))
        self.rope = dev(oracle.rope_table(P, D))
        self.cache = qmm.kv_cache_q4(PAGES, PAGE, HK, D, DEV)

    def heads(self, x, positions, slots, o, dense):
        """Rows x -> q, k, v of their heads, appended."""
        T = x.shape[0]
        qmm.rms_norm_q8_1(x, self.norm, 1e-5, out=o["xq"])
        dense(self.wd, o["xq"], out=o["qkv"])
        qkv = o["qkv"].view(T, HQ + 2 * HK, D)
        qmm.qk_norm_rope(qkv[:, :HQ], qkv[:, HQ:HQ + HK], self.rope, positions, q_weight=self.wq, k_weight=self.wk,
                         q_out=o["q"], k_out=o["k"])
        qmm.kv_append_q4(o["k"], qkv[:, HQ + HK:], self.cache, slots)
        return qkv[:, HQ + HK:]

    def prompt(self, x, positions, slots, cu, o, ws):
        v = self.heads(x, positions, slots, o, lambda *a, **k: qmm.mmq_q4k(*a, ws=ws, **k))
        qmm.qk_norm_rope(v, q_out=o["v"])                       # the values in 16 bits, as they are
        qmm.attn_prompt(o["q"], o["k"], o["v"], cu, out=o["y"])

    def decode(self, x, positions, slots, table, lens, o, ws):
        self.heads(x, positions, slots, o, qmm.mmvq_q4k)
        B = lens.shape[0]
        qmm.attn_q4(o["q"].view(B, -1, HQ, D), self.cache, table, lens, out=o["y"].view(B, -1, HQ, D), ws=ws)
        qmm.q8_1_quantize(o["y"].view(-1, HQ * D), out=o["yq"])
        qmm.mmvq_q4g(self.od[0], self.od[1], o["yq"], out=o["out"])


def buffers(T):
    e = lambda *s, dtype=F32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    return {"xq": e(T, H // 32, 40, dtype=torch.uint8), "qkv": e(T, N), "q": e(T, HQ, D, dtype=BF16),
            "k": e(T, HK, D, dtype=BF16), "v": e(T, HK, D, dtype=BF16), "y": e(T, HQ, D),
            "yq": e(T, HQ * D // 32, 40, dtype=torch.uint8), "out": e(T, H)}


def rows(seed, T):
    return dev(3 * qmm_synth.activations(qmm_synth.rng(seed), T, H, 0.01)).bfloat16()


LENS = [37, 1, 100]
TABLE = np.random.default_rng(1).permutation(PAGES)[:30].reshape(3, 10).astype(np.int32)


def places(first, count):
    """positions and slots of `count` tokens of each sequence from its first on."""
    pos = np.concatenate([np.arange(f, f + c) for f, c in zip(first, count)])
    seq = np.repeat(np.arange(len(first)), count)
    return dev(pos.astype(np.int32)), dev(TABLE[seq, pos // PAGE].astype(np.int64) * PAGE + pos % PAGE)


def prefill(layer, seed):
    T = sum(LENS)
    o, ws = buffers(T), qmm.workspace(qmm.workspace_bytes(qmm.QMM_OP_MMQ, N, H, T), DEV)
    pos, slots = places([0] * 3, LENS)
    cu = dev(np.concatenate(([0], np.cumsum(LENS))).astype(np.int32))
    args = (rows(seed, T), pos, slots, cu, o, ws)
    layer.prompt(*args)
    return args


def decode_args(layer, seed, n, lens, first):
    B = len(lens)
    pos, slots = places(first, [n] * B)
    need = qmm.attn_q4_workspace_bytes(B, n, HQ, HK, D, 10 * PAGE)
    return (rows(seed, B * n), pos, slots, dev(TABLE), dev(np.array(lens, np.int32)), buffers(B * n),
            torch.empty(max(16, need), dtype=torch.uint8, device=DEV))


def check_attention(y, q, k, v, n, term):
    seen = oracle.visible(n, k.shape[0], True)
    qb = q.double().cpu().numpy()
    ref, spread = oracle.attention(qb, k, v, D**-0.5, seen)
    bad = np.abs(y.double().cpu().numpy() - ref) - allowed(qb, k, D**-0.5, seen, ref, spread, term, F32)
    assert np.all(bad <= 0), (float(bad.max()), np.argwhere(bad > 0)[:8].tolist(), k.shape)


@pytest.mark.parametrize("n", [1, 2])
def test_every_stage_against_the_oracle(n):
    say("attention layer", f"n={n}")
    layer = Layer(3)
    x, pos, slots, cu, o, _ = prefill(layer, 4)
    W = oracle.q4k_dequant(layer.w)

    def check_heads(o, pos, slots):
        X = oracle.q8_1_dequant(host(o["xq"]))
        assert_parity(host(o["qkv"]), oracle.dense(W, X), oracle.abs_bound(W, X), "qkv")
        qkv = o["qkv"].view(-1, HQ + 2 * HK, D)
        for part, w, y in ((qkv[:, :HQ], layer.wq, o["q"]), (qkv[:, HQ:HQ + HK], layer.wk, o["k"])):
            t = oracle.head_norm(host(part), host(w), 1e-6)
            ref = oracle.turn(t, host(layer.rope), host(pos), False)
            size = np.abs(t) + np.abs(np.roll(t, D // 2, -1))            # |a c| + |b s| is at most that
            assert np.all(np.abs(y.double().cpu().numpy() - ref) <= 2.0**-8 * np.abs(ref) + 23 * 2.0**-24 * size)
        want = np.zeros(tuple(layer.cache.shape), np.uint8)
        oracle.cache_store(want, host(slots), o["k"].float().cpu().numpy(), host(qkv[:, HQ + HK:].contiguous()))
        for a, b in zip(oracle.cache_load(host(layer.cache), host(slots)), oracle.cache_load(want, host(slots))):
            assert np.array_equal(a, b)

    check_heads(o, pos, slots)
    assert torch.equal(o["v"], o["qkv"].view(-1, HQ + 2 * HK, D)[:, HQ + HK:].bfloat16())
    for b, L in enumerate(LENS):
        s = slice(int(cu[b]), int(cu[b + 1]))
        check_attention(o["y"][s], o["q"][s], o["k"][s].double().cpu().numpy(), o["v"][s].double().cpu().numpy(), L, 2.0**-8)
    # the new tokens: the cache holds the prompt and, after the append, them
    lens = [L + n for L in LENS]
    x, pos, slots, _, _, o, _ = args = decode_args(layer, 5, n, lens, LENS)
    layer.decode(*args)
    check_heads(o, pos, slots)
    for b, L in enumerate(lens):
        k, v = oracle.cache_load(host(layer.cache), host(places([0] * 3, [L if i == b else 0 for i in range(3)])[1]))
        check_attention(o["y"][b * n:(b + 1) * n], o["q"][b * n:(b + 1) * n], k, v, n, 2.0**-11)
    assert np.array_equal(host(o["yq"]), oracle.quantize_q8_1(host(o["y"]).reshape(-1, HQ * D)))
    Wo, X = oracle.q4g_dequant(*layer.wo), oracle.q8_1_dequant(host(o["yq"]))
    assert_parity(host(o["out"]), oracle.dense(Wo, X), oracle.abs_bound(Wo, X), "out")
    # the cache read back is a prompt's context: the same tokens through attn_prompt
    L = lens[2]
    k, v = qmm.kv_read_q4(layer.cache, places([0] * 3, [0, 0, L])[1], BF16)
    c = lambda *i: torch.tensor(i, dtype=torch.int32, device=DEV)  # noqa: E731
    y = qmm.attn_prompt(o["q"][2 * n:3 * n], k, v, c(0, n), c(0, L), out_dtype=F32)
    check_attention(y, o["q"][2 * n:3 * n], k.double().cpu().numpy(), v.double().cpu().numpy(), n, 2.0**-8)


def test_captured_and_replayed():
    layer, ref = Layer(6), Layer(6)
    pre, pre_ref = prefill(layer, 1), prefill(ref, 1)
    args = decode_args(layer, 2, 2, [L + 2 for L in LENS], LENS)
    ref_args = decode_args(ref, 2, 2, [L + 2 for L in LENS], LENS)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        layer.prompt(*pre)
        layer.decode(*args)
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize()
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        layer.prompt(*pre)
    with torch.cuda.graph(g2):
        layer.decode(*args)
    for r in range(4):
        # other rows, other lengths: all that a graph reads from memory may change between replays
        for a, b in ((pre, pre_ref), (args, ref_args)):
            a[0].copy_(rows(20 + r, a[0].shape[0]))
            b[0].copy_(a[0])
        lens = dev(np.array([L + 2 - r * (L > 30) for L in LENS], np.int32))
        args[4].copy_(lens)
        ref_args[4].copy_(lens)
        ref.prompt(*pre_ref)
        ref.decode(*ref_args)
        torch.cuda.synchronize()
        for o in (pre[4], args[5]):
            for v in o.values():
                v.fill_(1)
        args[6].fill_(0xFF)
        torch.cuda.synchronize()
        g1.replay()
        g2.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.cache, ref.cache), r
        for o, e in ((pre[4], pre_ref[4]), (args[5], ref_args[5])):
            for k in o:
                if k not in (("yq", "out") if o is pre[4] else ("v",)):
                    assert torch.equal(o[k], e[k]), (r, k)
        torch.randn(1000, device=DEV).sum().item()


def test_graphs_that_share_a_workspace():
    # two graphs on one workspace, replayed one after the other, a large call in one and a small in the other
    g = qmm_synth.rng(30)
    cache = dev(g.integers(0, 256, (300, 2, 1, 20 * 64)).astype(np.uint8))
    half = cache.view(F16)
    half[..., 256:320] = torch.rand_like(half[..., 256:320])
    half[..., 576:] = torch.rand_like(half[..., 576:])
    table = dev(g.permutation(300).reshape(1, 300).astype(np.int32))
    lens = [torch.tensor([x], dtype=torch.int32, device=DEV) for x in (4700, 900)]
    q = [dev(qmm_synth.activations(g, n, 8 * 64)).half().view(1, n, 8, 64) for n in (8, 1)]
    ws = torch.empty(max(16, qmm.attn_q4_workspace_bytes(1, 8, 8, 2, 64, 4800)), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(x) for x in q]
    calls = [lambda i=i: qmm.attn_q4(q[i], cache, table, lens[i], out=out[i], ws=ws) for i in (0, 1)]
    want = []
    for c in calls:
        c()
    torch.cuda.synchronize()
    want = [o.clone() for o in out]
    graphs = []
    for c in calls:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            c()
    for _ in range(4):
        for o in out:
            o.fill_(0)
        ws.fill_(0xFF)
        torch.cuda.synchronize()
        for i in (0, 1, 1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    layers = [Layer(7), Layer(8)]
    alone = []
    for i, l in enumerate(layers):
        pre = prefill(l, 10 + i)
        args = decode_args(l, 12 + i, 2, [L + 2 for L in LENS], LENS)
        l.decode(*args)
        alone.append((pre[4], args[5], l.cache.clone()))
    torch.cuda.synchronize()
    again = [(prefill(l, 10 + i), decode_args(l, 12 + i, 2, [L + 2 for L in LENS], LENS)) for i, l in enumerate(layers)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    for _ in range(5):
        for l, s, (pre, args) in zip(layers, streams, again):
            with torch.cuda.stream(s):
                l.prompt(*pre)
                l.decode(*args)
    torch.cuda.synchronize()
    for l, (pre, args), (p0, d0, c0) in zip(layers, again, alone):
        assert torch.equal(l.cache, c0)
        for k in ("xq", "qkv", "q", "k", "y"):
            assert torch.equal(pre[4][k], p0[k]) and torch.equal(args[5][k], d0[k]), k


def test_tensors_used_on_another_stream():
    # the workspace that the call takes by itself belongs to the stream it runs on
    layer = Layer(9)
    prefill(layer, 3)
    x, pos, slots, table, lens, o, ws = decode_args(layer, 4, 1, [L + 1 for L in LENS], LENS)
    layer.decode(x, pos, slots, table, lens, o, ws)
    torch.cuda.synchronize()
    want = o["y"].clone()
    s = torch.cuda.Stream(DEV)
    for _ in range(10):
        with torch.cuda.stream(s):
            y = qmm.attn_q4(o["q"].view(3, 1, HQ, D), layer.cache, table, lens, out_dtype=F32)
            z = qmm.attn_q4(o["q"].view(3, 1, HQ, D), layer.cache, table, lens, out_dtype=F32)
        junk = torch.full((1 << 20,), 255, dtype=torch.uint8, device=DEV)
        s.synchronize()
        assert torch.equal(y.view_as(want), want) and torch.equal(z.view_as(want), want)
        del junk


def test_padded_batch():
    # a batch of fixed size whose last sequences have ended: length 0, slots -1
    layer = Layer(10)
    prefill(layer, 5)
    lens, B = [L + 1 for L in LENS], 5
    x, pos, slots, table, l, o, ws = decode_args(layer, 6, 1, lens, LENS)
    layer.decode(x, pos, slots, table, l, o, ws)
    small, cache = o, layer.cache.clone()
    o5 = buffers(B)
    pad = lambda t, v, n: torch.cat((t, torch.full((n, *t.shape[1:]), v, dtype=t.dtype, device=DEV)))  # noqa: E731
    need = qmm.attn_q4_workspace_bytes(B, 1, HQ, HK, D, 10 * PAGE)
    layer.decode(pad(x, float("nan"), 2), pad(pos, -1, 2), pad(slots, -1, 2), pad(table, -1, 2), pad(l, 0, 2), o5,
                 torch.empty(max(16, need), dtype=torch.uint8, device=DEV))
    assert torch.equal(layer.cache, cache)
    assert torch.equal(o5["y"][:3], small["y"]) and not o5["y"][3:].any() and torch.equal(o5["out"][:3], small["out"])


def test_parts_of_lists():
    # lists of whole numbers from any entry on: a chunk's positions and slots, a batch's last sequences
    g = qmm_synth.rng(40)
    T, n = 70, 1
    x = dev(qmm_synth.activations(g, T, (HQ + 2 * HK) * D)).half().view(T, -1, D)
    q, k, v = x[:, :HQ], x[:, HQ:HQ + HK], x[:, HQ + HK:]
    table = dev(oracle.rope_table(200, D))
    pos, slots = dev(g.integers(0, 200, T).astype(np.int32)), dev(g.permutation(96)[:T].astype(np.int64))
    seqs, lens = dev(g.permutation(6).reshape(3, 2).astype(np.int32)), dev(np.array([5, 31, 17], np.int32))
    cu = dev(np.array([0, 3, 10, 40, 70], np.int32))
    caches = []
    for at in (lambda t, i: t[i:], lambda t, i: t[i:].clone()):
        cache = qmm.kv_cache_q4(6, 16, HK, D, DEV)
        qmm.kv_append_q4(k[1:], v[1:], cache, at(slots, 1), rope=table, positions=at(pos, 1))
        caches.append((cache, *qmm.kv_read_q4(cache, at(slots, 3)), *qmm.qk_norm_rope(q[3:], k[3:], table, at(pos, 3)),
                       qmm.attn_q4(q[:2 * n].view(2, n, HQ, D), cache, at(seqs, 1), at(lens, 1)),
                       qmm.attn_prompt(q, k, v, at(cu, 1))[3:]))
    assert all(torch.equal(a, b) for a, b in zip(*caches))
