"""GPU: attn_prompt reads and writes the rows of its sequences only, whatever cu_q and cu_k hold.

q, k, v and the output lie inside larger buffers; what is around them holds NaN
(read, it would show in the output) or a mark (written, it would be gone)."""
import numpy as np
import pytest
import torch

import qmm_synth
from _gpu import DEV, dev, say

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F16, BF16 = torch.float16, torch.bfloat16
MOST, LEAST = 2**31 - 1, -2**31
GUARD = 200          # rows on either side: more than a tile of keys or of queries


def inside(g, T, H, D, xt):
    big = torch.full((T + 2 * GUARD, H, D), float("nan"), dtype=xt, device=DEV)
    big[GUARD:GUARD + T] = dev(qmm_synth.activations(g, T, H * D)).view(T, H, D)
    return big[GUARD:GUARD + T]


@pytest.mark.parametrize("Tq,Tk,Hq,Hk,D,xt", [(50, 50, 2, 1, 64, BF16), (50, 1700, 4, 2, 128, F16), (50, 300, 2, 2, 256, BF16)])
@pytest.mark.parametrize("causal", [True, False])
def test_bounds_outside_the_rows(Tq, Tk, Hq, Hk, D, xt, causal):
    g = qmm_synth.rng(Tk + D)
    q, k, v = inside(g, Tq, Hq, D, xt), inside(g, Tk, Hk, D, xt), inside(g, Tk, Hk, D, xt)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def run(cu_q, cu_k):
        big = torch.full((Tq + 2 * GUARD, Hq, D), 7.0, dtype=xt, device=DEV)
        qmm.attn_prompt(q, k, v, i(cu_q), i(cu_k), causal=causal, out=big[GUARD:GUARD + Tq])
        torch.cuda.synchronize()
        assert torch.all(big[:GUARD] == 7) and torch.all(big[GUARD + Tq:] == 7), (cu_q, cu_k)
        assert torch.isfinite(big).all(), (cu_q, cu_k)
        return big[GUARD:GUARD + Tq]

    for cu_q, cu_k, same_q, same_k in (
            ((0, 20, MOST), (0, 20, MOST), (0, 20, Tq), (0, 20, Tk)),                # past the end: as if there
            ((LEAST, 20, Tq), (-1, 20, Tk + 1), (0, 20, Tq), (0, 20, Tk)),           # before the first row
            ((0, 20, Tq), (0, MOST, MOST), (0, 20, Tq), (0, Tk, Tk))):
        say("attn_prompt bounds", cu_q, cu_k)
        assert torch.equal(run(cu_q, cu_k), run(same_q, same_k)), (cu_q, cu_k)
    # sequences that are nowhere within the rows: nothing is written
    for cu_q, cu_k in (((Tq + 10, Tq + 40, MOST), (-40, MOST, 5)), ((LEAST, -7, 0), (0, 5, Tk)), ((Tq, Tq, Tq), (0, 1, Tk))):
        say("attn_prompt bounds", cu_q, cu_k)
        assert torch.all(run(cu_q, cu_k) == 7), (cu_q, cu_k)
    # ends before beginnings: no rows, or no keys, which gives zeros
    say("attn_prompt bounds in reverse")
    assert not run((LEAST, MOST, 10), (MOST, LEAST, 7)).any()
    y = run((0, 30, 10), (0, Tk, 7))
    assert torch.equal(y[:30], run((0, 30, 30), (0, Tk, Tk))[:30]) and torch.all(y[30:] == 7)


def test_sequences_inside_the_rows_read_no_others():
    """Rows of q, k and v between and around the sequences hold NaN."""
    g = qmm_synth.rng(5)
    D, Tq, Tk = 128, 120, 900
    q, k, v = inside(g, Tq, 4, D, BF16), inside(g, Tk, 2, D, BF16), inside(g, Tk, 2, D, BF16)
    c = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    want = qmm.attn_prompt(q, k, v, c(30, 50, 100), c(100, 300, 700))
    for t, rows in ((q, (slice(0, 30), slice(100, Tq))), (k, (slice(0, 100), slice(700, Tk))), (v, (slice(0, 100), slice(700, Tk)))):
        for r in rows:
            t[r] = float("nan")
    y = torch.full_like(want, 7)
    qmm.attn_prompt(q, k, v, c(30, 50, 100), c(100, 300, 700), out=y)
    assert torch.equal(y[30:100], want[30:100]) and torch.all(y[:30] == 7) and torch.all(y[100:] == 7)
