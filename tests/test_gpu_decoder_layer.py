"""The norm, the router and the group-scaled matvec together with the products
between them, as a decoder layer calls them: norm -> matvec -> norm with the
residual -> router -> routed FFN -> norm -> output matvec.

Every stage is compared with the oracle on the inputs that the GPU's own
earlier stages gave it, so no error is carried from stage to stage, and the
whole run is captured into a graph and replayed, with the inputs changed in
place and the program's own work between the replays.
"""
import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _gpu import DEV, assert_parity, dev, host, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

H, F, E, TOP_K, V = 512, 256, 16, 4, 640


class Layer:
    def __init__(self, seed):
        g = qmm_synth.rng(seed)
        self.proj = qmm_synth.q4g_weights(g, H, H, 64, True)
        self.head = qmm_synth.q4g_weights(g, V, H, 128)
        self.gate_up = np.stack([qmm_synth.q4k_weights(g, 2 * F, H) for _ in range(E)])
        self.down = np.stack([qmm_synth.q6k_weights(g, H, F) for _ in range(E)])
        self.norms = [1 + 0.1 * g.standard_normal(H).astype(np.float32) for _ in range(3)]
        self.router = (0.05 * g.standard_normal((E, H))).astype(np.float32)
        self.bias = (0.02 * g.standard_normal(E)).astype(np.float32)
        self.d = {k: dev(v) for k, v in (("gate_up", self.gate_up), ("down", self.down), ("router", self.router),
                                         ("bias", self.bias))}
        self.dn = [dev(n) for n in self.norms]
        self.dp = [dev(self.proj[0]), dev(self.proj[1]).half(), dev(self.proj[2])]
        self.dh = [dev(self.head[0]), dev(self.head[1]).bfloat16()]

    def run(self, stream, ws, o):
        """stream: bf16 [T, H], updated in place; every stage's output into o."""
        d = self.d
        qmm.rms_norm_q8_1(stream, self.dn[0], 1e-5, out=o["xq1"])
        qmm.mmvq_q4g(self.dp[0], self.dp[1], o["xq1"], zeros=self.dp[2], out=o["proj"])
        o["before1"].copy_(stream)
        qmm.rms_norm_q8_1(o["proj"], self.dn[1], 1e-5, residual=stream, residual_out=stream, out=o["xq2"], y=o["y"])
        o["after1"].copy_(stream)
        torch.matmul(o["y"], d["router"].t(), out=o["logits"])
        qmm.moe_router(o["logits"], TOP_K, scoring="sigmoid", bias=d["bias"], n_groups=4, topk_groups=2,
                       group_score="top2", renormalize=True, ids=o["ids"], weights=o["w"])
        qmm.moe_ffn(qmm.QMM_Q4_K, d["gate_up"], qmm.QMM_Q6_K, d["down"], o["xq2"], o["ids"], o["w"], out=o["ffn"], ws=ws)
        qmm.rms_norm_q8_1(o["ffn"], self.dn[2], 1e-5, residual=stream, residual_out=stream, out=o["xq3"])
        qmm.q8_1_dequantize(o["xq3"], torch.float16, out=o["x3"])
        qmm.mmvq_q4g(self.dh[0], self.dh[1], o["xq3"], out=o["out"])


def buffers(T):
    e = lambda *s, dtype=torch.float32: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    u = torch.uint8
    return {"xq1": e(T, H // 32, 40, dtype=u), "xq2": e(T, H // 32, 40, dtype=u), "xq3": e(T, H // 32, 40, dtype=u),
            "proj": e(T, H), "before1": e(T, H, dtype=torch.bfloat16), "after1": e(T, H, dtype=torch.bfloat16),
            "y": e(T, H), "logits": e(T, E), "ids": e(T, TOP_K, dtype=torch.int32), "w": e(T, TOP_K), "ffn": e(T, H),
            "x3": e(T, H, dtype=torch.float16), "out": e(T, V)}


def stream_rows(seed, T):
    return dev(3 * qmm_synth.activations(qmm_synth.rng(seed), T, H, 0.01)).bfloat16()


def workspace(T):
    return qmm.workspace(qmm.workspace_bytes(qmm.QMM_OP_MOE_FFN, H, F, T, E, TOP_K), DEV)


@pytest.mark.parametrize("T", [1, 3, 8])
def test_every_stage_against_the_oracle(T):
    say("decoder layer", f"T={T}")
    layer, o, s = Layer(5), buffers(T), stream_rows(9, T)
    start = s.clone()
    layer.run(s, workspace(T), o)
    tol = ((H / 64 + 11) / 2 + 7) * 2.0**-24                # of the norm: see test_gpu_norm

    def norm_bytes(xq, h, w):
        n = oracle.rms_norm(h.double().cpu().numpy(), w, 1e-5)
        got = oracle.q8_1_dequant(host(xq))
        # a value is off by half a step of its block, the scale's f16 rounding and the norm's own error
        step = np.abs(n).reshape(T, -1, 32).max(-1).repeat(32, -1).reshape(T, H) / 127
        assert np.all(np.abs(got - n) <= step * (0.5 + 2.0**-10) + np.abs(n) * (2.0**-10 + 4 * tol))

    norm_bytes(o["xq1"], start, layer.norms[0])
    W, X = oracle.q4g_dequant(*layer.proj), oracle.q8_1_dequant(host(o["xq1"]))
    assert_parity(host(o["proj"]), oracle.dense(W, X), oracle.abs_bound(W, X), "proj")
    assert torch.equal(o["before1"], start)
    assert torch.equal(o["after1"], (o["proj"] + start.float()).bfloat16())
    n = oracle.rms_norm(o["after1"].double().cpu().numpy(), layer.norms[1], 1e-5)
    assert np.all(np.abs(host(o["y"]) - n) <= tol * np.abs(n))
    assert np.array_equal(host(o["xq2"]), oracle.quantize_q8_1(host(o["y"])))
    ids, w = oracle.route(host(o["logits"]), TOP_K, "sigmoid", layer.bias, 4, 2, "top2", True)
    assert np.array_equal(host(o["ids"]), ids)
    assert np.all(np.abs(host(o["w"]) - w) <= (4 + TOP_K + 6) * 2.0**-24 * w)
    # the routed FFN is the separate calls' (which have their own parity tests)
    gu = qmm.moe_grouped_swiglu(qmm.QMM_Q4_K, layer.d["gate_up"], o["xq2"], o["ids"])
    assert torch.equal(o["ffn"], qmm.moe_grouped_mmq(qmm.QMM_Q6_K, layer.d["down"], gu, o["ids"], o["w"]))
    after = (o["ffn"] + o["after1"].float()).bfloat16()
    assert torch.equal(s, after)
    norm_bytes(o["xq3"], after, layer.norms[2])
    X = oracle.q8_1_dequant(host(o["xq3"]))
    assert np.array_equal(host(o["x3"]), X.astype(np.float16))
    W = oracle.q4g_dequant(*layer.head)
    assert_parity(host(o["out"]), oracle.dense(W, X), oracle.abs_bound(W, X), "head")


@pytest.mark.parametrize("T", [1, 5])
def test_captured_and_replayed(T):
    layer, ws = Layer(6), workspace(T)
    s, o = stream_rows(0, T), buffers(T)
    side = torch.cuda.Stream(DEV)
    side.wait_stream(torch.cuda.current_stream(DEV))
    with torch.cuda.stream(side):
        layer.run(s, ws, o)
    torch.cuda.current_stream(DEV).wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.run(s, ws, o)
    eager, ws2 = buffers(T), workspace(T)
    for r in range(4):
        x = stream_rows(20 + r, T)
        s2 = x.clone()
        layer.run(s2, ws2, eager)
        torch.cuda.synchronize()
        for k, v in o.items():
            v.fill_(0 if v.dtype == torch.int32 else 165)
        s.copy_(x)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(s, s2), r
        for k in o:
            assert torch.equal(o[k], eager[k]), (r, k)
        torch.randn(1000, device=DEV).sum().item()


def test_two_streams_at_once():
    # no state is shared between calls: two layers' calls on two streams give what they give alone
    T = 4
    layers, rows = [Layer(7), Layer(8)], [stream_rows(31, T), stream_rows(32, T)]
    alone = []
    for l, x in zip(layers, rows):
        s, o = x.clone(), buffers(T)
        l.run(s, workspace(T), o)
        alone.append((s, o))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV), torch.cuda.Stream(DEV)]
    state = [(x.clone(), workspace(T), buffers(T)) for x in rows]
    torch.cuda.synchronize()
    for _ in range(5):
        for l, st, (s, ws, o), x in zip(layers, streams, state, rows):
            with torch.cuda.stream(st):
                s.copy_(x)
                l.run(s, ws, o)
    torch.cuda.synchronize()
    for (s, _, o), (s0, o0) in zip(state, alone):
        assert torch.equal(s, s0)
        for k in o:
            assert torch.equal(o[k], o0[k]), k


def test_large_calls_captured():
    """Sizes that take the other variants: many tokens for the norm and the router, few rows and long rows for the matvec."""
    g = qmm_synth.rng(40)
    x, r, w = dev(qmm_synth.activations(g, 300, 11008)), dev(qmm_synth.activations(g, 300, 11008)).half(), torch.ones(11008, device=DEV)
    logits = dev(qmm_synth.activations(g, 3000, 384)).bfloat16()
    bias = dev(np.zeros(384, np.float32))            # near ties and equal values everywhere
    q, s, z = qmm_synth.q4g_weights(g, 48, 28672, 128, True)
    q, s, z = dev(q), dev(s).half(), dev(z)
    xq = dev(oracle.quantize_q8_1(qmm_synth.activations(g, 8, 28672)))
    o = {"xq": torch.empty(300, 344, 40, dtype=torch.uint8, device=DEV), "res": torch.empty_like(r),
         "y": torch.empty(300, 11008, dtype=torch.bfloat16, device=DEV),
         "ids": torch.empty(3000, 10, dtype=torch.int32, device=DEV), "w": torch.empty(3000, 10, device=DEV),
         "wide": torch.empty(3000, 40, dtype=torch.int32, device=DEV), "ww": torch.empty(3000, 40, device=DEV),
         "mv": torch.empty(8, 48, device=DEV)}

    def run():
        qmm.rms_norm_q8_1(x, w, residual=r, residual_out=o["res"], out=o["xq"], y=o["y"])
        qmm.moe_router(logits, 10, bias=bias, ids=o["ids"], weights=o["w"])
        qmm.moe_router(logits, 40, scoring="sigmoid", renormalize=True, ids=o["wide"], weights=o["ww"])
        qmm.mmvq_q4g(q, s, xq, zeros=z, out=o["mv"])

    run()
    torch.cuda.synchronize()
    g1 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        run()
    for _ in range(3):
        x.mul_(1.25)
        logits.copy_(logits.roll(1, 0))
        run()
        torch.cuda.synchronize()
        ref = {k: v.clone() for k, v in o.items()}
        for v in o.values():
            v.fill_(1)
        g1.replay()
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], ref[k]), k
    assert np.array_equal(host(o["ids"])[:200], oracle.route(logits[:200].float().cpu().numpy(), 10, bias=np.zeros(384))[0])
