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


def event_ms(call, repeat=5):
    call()
    times = []
    for _ in range(repeat):
        e = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        e[0].record()
        call()
        e[1].record()
        e[1].synchronize()
        times.append(e[0].elapsed_time(e[1]))
    return sorted(times)[repeat // 2]


def test_long_prompt_beside_single_tokens():
    """One prompt of many rows beside thousands of single tokens: nearly all of the
    call's tiles of rows are empty, and cost next to nothing (each CTA went through
    them one by one)."""
    singles, prompt, hq, dim, page = 2048, 65536, 8, 64, 16
    rows = np.ones(singles + 1, np.int64)
    rows[singles // 2] = prompt
    lens = np.full(singles + 1, 33)
    cache = A.U.Cache(8, page, 1, dim, np.random.default_rng(4))
    buf = A.to_torch(cache)
    table = np.random.default_rng(5).integers(0, 8, (singles + 1, 3))
    q = A.rand(6, (int(rows.sum()), hq, dim), BF16, 0.8)

    def call(case, q):
        return A.attend(case, q, buf, 8, table[:len(case[5])], case[6], 0.1)

    both = (BF16, dim, hq, 1, page, rows.tolist(), lens.tolist(), True, 0)
    alone = (BF16, dim, hq, 1, page, [prompt], [33], True, 0)
    rest = (BF16, dim, hq, 1, page, [1] * singles, [33] * singles, True, 0)
    o, lse = call(both, q)
    L.lbgemm_device_status()
    # every single token, and the prompt's last rows (the others see nothing)
    first = int(rows[:singles // 2].sum())
    keep = np.r_[0:first, first + prompt - 40:int(rows.sum())]
    small = rows.copy()
    small[singles // 2] = 40
    A.check_attention((BF16, dim, hq, 1, page, small.tolist(), lens.tolist(), True, 0), cache, table,
                      q[keep], o[keep], lse[keep], 0.1)
    assert (o[first:first + prompt - 40] == 0).all()
    ms, parts = event_ms(lambda: call(both, q)), (event_ms(lambda: call(alone, q[:prompt])),
                                                  event_ms(lambda: call(rest, q[:singles])))
    print(ms, parts)
    # (the 256-row kernel takes the single tokens too here: a few times their own call)
    assert ms <= 5 * sum(parts)
