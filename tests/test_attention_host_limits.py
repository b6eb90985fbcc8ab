"""Limits of the attention operators' sizes: refused on the host, before any
device is touched.  No GPU needed."""
import pytest

from bit_tensor_gemm_gb300 import build as bld
from bit_tensor_gemm_gb300 import lbgemm as L
from test_attention_host import attend, refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bld.build()
    L.load()


@pytest.mark.parametrize("batch,max_q,hq", [
    (65535, (1 << 17) + 8, 64),   # 32770 tiles of 256 rows a sequence
    (65535, (1 << 20) + 64, 8),
    (40000, 1 << 21, 16),
])
def test_too_many_tiles(batch, max_q, hq):
    """Tiles of rows are counted in 32 bits by the kernels: 2^31 and more overflowed
    the count."""
    assert batch * -(-max_q * hq // 256) >= 1 << 31
    refused(L.ERR_INVALID_ARG, attend, batch=batch, total=max_q, max_q=max_q, hq=hq, hk=1,
            qs=hq * 128)
    assert b"tiles" in L.load().lbgemm_last_error()
