"""GPU tests of attention with a window over sequences that gave back the pages
before it, within the bounds of attention_tight.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_tight as T  # noqa: E402
import test_gpu_attention as A  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

BF16, F16 = L.BF16, L.F16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


# dtype, dim, heads_q, heads_kv, page, rows, lengths, window
WINDOW = [
    (BF16, 128, 8, 2, 16, [1, 1, 1], [1000, 127, 129], 100),
    (F16, 64, 8, 2, 64, [1, 5, 3], [1000, 700, 64], 64),
    (BF16, 64, 4, 4, 32, [1], [513], 1),
    (F16, 128, 6, 2, 48, [7, 2], [900, 301], 130),
    (BF16, 128, 4, 1, 256, [3], [1900], 500),
    (BF16, 64, 4, 2, 16, [40], [600], 33),
    (F16, 128, 8, 2, 16, [90, 1, 300], [900, 500, 700], 100),
    (BF16, 64, 16, 16, 32, [300], [1500], 257),
    (BF16, 128, 4, 4, 128, [70, 200], [2000, 1000], 1),
]


@pytest.mark.parametrize("case", WINDOW)
def test_pages_before_the_window(case):
    """Pages of which no row sees a token have no entry in the table any more, and
    tokens before the window in a page that is still there hold anything."""
    dtype, dim, hq, hk, page, rows, lens, window = case
    case = (dtype, dim, hq, hk, page, rows, lens, True, window)
    cache, table, width, pages, q = A.attend_inputs(case, 700)
    used = A.U.Cache(pages, page, hk, dim)
    used.codes, used.scales = cache.codes, np.nan_to_num(cache.scales, nan=0.0, posinf=0.0)
    ref = T.attention(q, A.U.DTYPES[dtype], used, lens, rows, table, 0.1, True, window)
    gone = 0
    for b, (n, length) in enumerate(zip(rows, lens)):
        first = max(0, length - n - window + 1)  # the first row's first token
        cache.scales[0, table[b, first // page], :first % page] = np.nan
        cache.scales[1, table[b, first // page], :first % page] = np.inf
        table[b, :first // page] = -1
        gone += first // page
    assert gone > 0
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, 0.1)
    L.lbgemm_device_status()
    T.check(o, lse, ref)
