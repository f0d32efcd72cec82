"""GPU: README's attention example runs as it stands, and its calls agree with the oracle."""
import os
import textwrap

import numpy as np
import pytest
import torch

import oracle
import qmm_synth
from _attention import allowed
from _gpu import DEV, dev

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def example(first):
    """The lines of README's Python block from the one that begins with `first` on."""
    lines = open(README, encoding="utf-8").read().splitlines()
    at = next(i for i, x in enumerate(lines) if x.strip().startswith(first))
    end = next(i for i in range(at, len(lines) + 1) if i == len(lines) or lines[i] and not lines[i].startswith("    "))
    return textwrap.dedent("\n".join(lines[at:end]))


def test_attention_example():
    g = qmm_synth.rng(1)
    B, n, Hq, Hk, D, pages = 3, 4, 4, 2, 64, 5
    T = B * n
    slots = np.concatenate([b * 64 + np.arange(n) for b in (4, 0, 2)])
    qkv = dev(qmm_synth.activations(g, T, (Hq + 2 * Hk) * D)).view(T, -1, D)
    names = dict(qmm=qmm, torch=torch, dev=DEV, B=B, n=n, Hq=Hq, Hk=Hk, D=D, pages=pages, qkv=qkv,
                 rope=dev(oracle.rope_table(50, D)), positions=dev(np.tile(np.arange(n, dtype=np.int32), B)),
                 wq=torch.ones(D, device=DEV), wk=torch.ones(D, device=DEV), slots=dev(slots.astype(np.int64)),
                 cu_seqlens=dev((n * np.arange(B + 1)).astype(np.int32)), table=dev(np.array([[4], [0], [2]], np.int32)),
                 lens=dev(np.full(B, n, np.int32)))
    code = example("# attention of a layer")
    assert "attn_prompt" in code and "kv_read_q4" in code
    for line in code.splitlines():
        exec(line, names)                               # noqa: S102
        if "attn_prompt(" in line:
            prompt, k, v = names["y"], names["k"], names["v"]
    q, y = names["q"], names["y"].view(T, Hq, D)
    assert torch.equal(v, qkv[:, -Hk:].bfloat16())
    kept = qmm.kv_read_q4(names["cache"], names["slots"], torch.float32)     # the cache's numbers, exact
    for out, (keys, values), term in ((prompt, (k, v), 2.0**-8), (y, kept, 2.0**-11)):
        for b in range(B):
            s = slice(b * n, b * n + n)
            seen = oracle.visible(n, n, True)
            qb, kb, vb = (t[s].double().cpu().numpy() for t in (q, keys, values))
            ref, spread = oracle.attention(qb, kb, vb, D**-0.5, seen)
            tol = allowed(qb, kb, D**-0.5, seen, ref, spread, term, torch.bfloat16)
            assert np.all(np.abs(out[s].double().cpu().numpy() - ref) <= tol)
