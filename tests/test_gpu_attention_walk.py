"""GPU tests of attention calls whose CTAs walk from tile to tile: calls with
more tiles than CTAs, with sequences that see nothing among them.

Tolerances as in test_gpu_attention.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

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


def run(case, seed, scale=0.1, repeat=1):
    """One call checked against 64 bits, and its repeats against itself."""
    cache, table, width, pages, q = A.attend_inputs(case, seed)
    buf = A.to_torch(cache)
    o, lse = A.attend(case, q, buf, pages, table, case[6], scale)
    L.lbgemm_device_status()
    A.check_attention(case, cache, table, q, o, lse, scale)
    for _ in range(repeat):
        o2, lse2 = A.attend(case, q, buf, pages, table, case[6], scale)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    L.lbgemm_device_status()


# Runs of tiles without a visible token between ordinary ones, many rows: 8 heads
# of 60 and more sequences on at most one CTA an SM are several such tiles in a row.
EMPTY = [
    (BF16, 64, 8, 8, 16, [100] * 60, [0] * 59 + [700], True, 0),
    (F16, 128, 8, 8, 16, [300] + [70] * 80 + [90, 257], [310] + [0] * 80 + [200, 300], True, 0),
    (BF16, 64, 16, 8, 16, [600, 80, 80, 80, 600, 70] * 6, [20, 0, 300, 0, 5, 0] * 6, True, 0),  # rows before the start
    (F16, 64, 8, 4, 16, [200] * 40, [0, 0, 0, 130] * 10, False, 0),
    (BF16, 128, 4, 4, 16, [500, 66] * 30, [100, 0, 900, 3] * 15, True, 40),
]


@pytest.mark.parametrize("case", EMPTY)
def test_tiles_that_see_nothing(case):
    run(case, 300, repeat=40)
