"""The paged cache's bookkeeping: what it hands out and what it refuses.  No GPU
needed."""
import numpy as np
import pytest

pytest.importorskip("torch")

from bit_tensor_gemm_gb300 import attention_layer as layers  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bld.build()
    L.load()


@pytest.mark.parametrize("rows", [[1], [1, 1, 1], [3, -1], [[1, 2]]])
def test_extend_refuses(rows):
    """Another number of sequences, or fewer than no tokens: nothing changes."""
    cache = layers.PagedCache(2, 20, 2, 64, 16, device="cpu")
    cache.extend([5, 17])
    with pytest.raises(ValueError):
        cache.extend(rows)
    assert cache.lens.tolist() == [5, 17] and len(cache.free) == cache.pages - 3


def test_extend_hands_out_pages():
    cache = layers.PagedCache(2, 40, 2, 64, 16, device="cpu")
    cache.extend([15, 0])
    new = cache.extend([2, 33])
    assert new["positions"].tolist() == [15, 16] + list(range(33))
    assert new["cu_q"].tolist() == [0, 2, 35] and new["lens"].tolist() == [17, 33]
    assert (new["max_q"], new["max_kv"]) == (33, 33)
    slots = new["slots"].numpy()
    assert len(set(slots.tolist())) == 35 and (slots % 16 == np.r_[15, 0, np.arange(33) % 16]).all()
    assert (slots // 16 == np.r_[cache.table[0, [0, 1]], cache.table[1, np.arange(33) // 16]]).all()
