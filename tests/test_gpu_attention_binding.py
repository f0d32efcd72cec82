"""GPU: calls of the attention operators that the binding has to take, or has to refuse."""
import numpy as np
import pytest
import torch

from _gpu import DEV, dev

import quantized_matmul_q8_amd as qmm

pytestmark = pytest.mark.gpu

F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


def test_no_tokens_in_tensors_of_any_strides():
    """What numpy makes of no values has strides of zero."""
    none = lambda *s: torch.empty_strided(s, (0,) * len(s), dtype=F16, device=DEV)  # noqa: E731
    assert dev(np.zeros((0, 2, 64), np.float16)).shape == (0, 2, 64)
    i = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype, device=DEV)  # noqa: E731
    q, k = qmm.qk_norm_rope(none(0, 4, 64), none(0, 2, 64))
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    cache = qmm.kv_cache_q4(2, 16, 2, 64, DEV)
    qmm.kv_append_q4(none(0, 2, 64), none(0, 2, 64), cache, i(0, dtype=torch.int64))
    assert not cache.any()
    assert qmm.attn_q4(none(0, 3, 4, 64), cache, i(0, 2), i(0)).shape == (0, 3, 4, 64)
    assert qmm.attn_q4(none(0, 4, 64), cache, i(0, 2), i(0)).shape == (0, 4, 64)
    assert qmm.attn_prompt(none(0, 4, 64), none(0, 2, 64), none(0, 2, 64), i(1)).shape == (0, 4, 64)
    q = torch.ones(3, 4, 64, dtype=F16, device=DEV)
    assert not qmm.attn_prompt(q, none(0, 2, 64), none(0, 2, 64), torch.tensor([0, 3], dtype=torch.int32, device=DEV), i(2)).any()


def test_outputs_over_an_input_are_refused():
    """Several workgroups read a query, and one may have written its output by then."""
    cache = qmm.kv_cache_q4(2, 16, 2, 64, DEV)
    q, k = torch.ones(3, 4, 64, dtype=F16, device=DEV), torch.ones(3, 4, 64, dtype=F16, device=DEV)
    table, lens = torch.zeros(3, 1, dtype=torch.int32, device=DEV), torch.ones(3, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError, match="out"):
        qmm.attn_q4(q, cache, table, lens, out=q)
    for out in (q, k):
        with pytest.raises(ValueError, match="out"):
            qmm.attn_prompt(q, k, torch.ones_like(k), cu, out=out)
        with pytest.raises(ValueError, match="out"):
            qmm.attn_prompt(q, torch.ones_like(k), k, cu, out=out)
    assert torch.all(q == 1) and torch.all(k == 1)
