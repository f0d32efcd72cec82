"""GPU: the forms of attn_q4 and attn_prompt that leave partial results in a workspace, on streams of
their own, at once, captured and replayed.  Every case asserts that it needs a workspace."""
import numpy as np
import pytest
import torch

import qmm_synth
from _gpu import DEV, dev, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16


class Cached:
    """attn_q4 over random numbers in the cache: lengths up to `longest` under a table that is as wide."""

    def __init__(self, seed, B, n, Hq, Hk, D, longest):
        g = qmm_synth.rng(seed)
        per = -(-longest // 16)
        self.g, self.longest, self.B = g, longest, B
        self.cache = qmm.kv_cache_q4(B * per, 16, Hk, D, DEV)
        T = B * per * 16
        k, v = (dev(qmm_synth.activations(g, T, Hk * D, 0.01)).view(T, Hk, D) for _ in range(2))
        qmm.kv_append_q4(k, v, self.cache, torch.arange(T, device=DEV))
        self.table = dev(g.permutation(B * per).reshape(B, per).astype(np.int32))
        self.lens = torch.zeros(B, dtype=torch.int32, device=DEV)
        self.q = dev(qmm_synth.activations(g, B * n, Hq * D)).half().view(B, n, Hq, D)
        self.need = qmm.attn_q4_workspace_bytes(B, n, Hq, Hk, D, per * 16)
        self.other_lengths()

    def other_lengths(self):
        now = self.g.integers(0, self.longest + 1, self.B).astype(np.int32)
        now[0] = self.longest
        self.lens.copy_(dev(now))

    def __call__(self, **kw):
        return qmm.attn_q4(self.q, self.cache, self.table, self.lens, **kw)


class Prompts:
    """attn_prompt of few rows behind many keys."""

    def __init__(self, seed, nq, nk, Hq, Hk, D):
        g = qmm_synth.rng(seed)
        self.g, self.nq, self.nk = g, nq, nk
        self.q = dev(qmm_synth.activations(g, nq, Hq * D)).bfloat16().view(nq, Hq, D)
        self.k, self.v = (dev(qmm_synth.activations(g, nk, Hk * D, 0.01)).bfloat16().view(nk, Hk, D) for _ in range(2))
        self.cu_q, self.cu_k = (torch.zeros(3, dtype=torch.int32, device=DEV) for _ in range(2))
        self.need = qmm.attn_prompt_workspace_bytes(2, nq, nk, Hq, Hk, D)
        self.other_lengths()

    def other_lengths(self):
        self.cu_q.copy_(dev(np.array([0, self.g.integers(0, self.nq + 1), self.nq], np.int32)))
        self.cu_k.copy_(dev(np.array([0, self.g.integers(0, self.nk + 1), self.nk], np.int32)))

    def __call__(self, **kw):
        return qmm.attn_prompt(self.q, self.k, self.v, self.cu_q, self.cu_k, **kw)


CASES = {
    "parts": lambda seed: Cached(seed, 2, 1, 8, 2, 128, 3000),
    "parts of many rows": lambda seed: Cached(seed, 3, 8, 16, 2, 64, 2000),
    "runs": lambda seed: Cached(seed, 66, 1, 8, 4, 64, 1100),
    "runs of many rows": lambda seed: Cached(seed, 64, 4, 32, 4, 96, 1100),
    "split prompts": lambda seed: Prompts(seed, 60, 6000, 8, 2, 128),
    "wide split prompts": lambda seed: Prompts(seed, 90, 3000, 4, 1, 256),
}


def scratch(case):
    return torch.full((case.need + 64,), 0xFF, dtype=torch.uint8, device=DEV)


@pytest.fixture(params=list(CASES))
def make(request):
    say("attention with partial results", request.param)

    def one(seed):
        case = CASES[request.param](seed)
        assert case.need > 0
        return case

    return one


def test_a_workspace_taken_on_another_stream(make):
    """The call's own workspace belongs to the stream that it runs on: memory taken elsewhere meanwhile is not it."""
    case = make(1)
    want = case()
    torch.cuda.synchronize()
    s = torch.cuda.Stream(DEV)
    for _ in range(10):
        with torch.cuda.stream(s):
            got = [case() for _ in range(3)]
        junk = [torch.full((case.need,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        s.synchronize()
        assert all(torch.equal(y, want) for y in got)
        del junk, got


@pytest.mark.parametrize("own", [True, False])
def test_two_streams_at_once_with_partial_results(make, own):
    """Workspaces that the calls take by themselves, or one for each stream."""
    cases = [make(2), make(3)]
    want = [c() for c in cases]
    ws = [scratch(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in cases]
    got = [[], []]
    for _ in range(8):
        for c, s, y, w in zip(cases, streams, got, ws):
            with torch.cuda.stream(s):
                y.append(c() if own else c(ws=w[:-64]))
    torch.cuda.synchronize()
    for y, x, w in zip(got, want, ws):
        assert all(torch.equal(z, x) for z in y)
        assert torch.all(w[-64:] == 0xFF)


@pytest.mark.parametrize("own", [True, False])
def test_graphs_with_partial_results_on_two_streams(make, own):
    """Captured with a workspace of the graph's or of the caller's, replayed with other lengths, two graphs at once."""
    cases = [make(4), make(5)]
    ws, out = [scratch(c) for c in cases], [torch.empty_like(c.q) for c in cases]
    graphs, streams = [], [torch.cuda.Stream(DEV) for _ in cases]
    call = lambda i: cases[i](out=out[i]) if own else cases[i](out=out[i], ws=ws[i][:-64])  # noqa: E731
    for i in (0, 1):
        call(i)
    torch.cuda.synchronize()
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            call(i)
    for r in range(5):
        for c in cases:
            c.other_lengths()
        want = [c() for c in cases]
        for o, w in zip(out, ws):
            o.fill_(7)
            w.fill_(0xFF)
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, x) for o, x in zip(out, want)), r
        assert all(torch.all(w[-64:] == 0xFF) for w in ws)


def test_equal_calls_give_equal_bits(make):
    case = make(6)
    want = case()
    ws = scratch(case)
    for fill in (0x00, 0xFF, 0x7F):
        ws.fill_(fill)
        assert torch.equal(case(ws=ws[:-64]), want) and torch.equal(case(), want)
        assert torch.all(ws[-64:] == fill)
