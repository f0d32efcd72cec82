"""kv_cache_q4 makes what the calls that take a cache accept, and nothing else (no GPU needed)."""
import pytest
import torch

qmm = pytest.importorskip("quantized_matmul_q8_amd")


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_shapes(D):
    c = qmm.kv_cache_q4(3, 48, 2, D, "cpu")
    assert c.shape == (3, 2, 3, 20 * D) and c.dtype == torch.uint8 and not c.any()
    assert qmm.kv_cache_q4(1, 1 << 20, 1, 64, "meta").shape == (1, 1, 1 << 16, 1280)
    assert qmm.kv_cache_q4(2**31 - 1, 16, 1024, D, "meta").shape == (2**31 - 1, 1024, 1, 20 * D)


@pytest.mark.parametrize("pages,page,Hk,D", [(0, 16, 1, 64), (1, 0, 1, 64), (1, 24, 1, 64), (1, 16, 0, 64), (1, 16, 1, 80),
                                             (1, (1 << 20) + 16, 1, 64), (1, 16, 1025, 64), (2**31, 16, 1, 64)])
def test_refusals(pages, page, Hk, D):
    with pytest.raises(ValueError):
        qmm.kv_cache_q4(pages, page, Hk, D, "meta")
