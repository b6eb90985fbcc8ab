"""GPU tests of attention within the bounds of attention_tight.py, which a token
left out or counted twice breaks: calls whose CTAs walk over several tiles,
common head layouts, tokens at the edges of steps, pages and runs, and value
scales far apart at many cuts."""
import math

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


def lengths(seed, n, least, most):
    return [int(x) for x in np.random.default_rng(seed).integers(least, most + 1, n)]


def check(case, cache, table, pages, q, scale):
    dtype, dim, hq, hk, page, rows, lens, causal, window = case
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, scale)
    L.lbgemm_device_status()
    T.check(o, lse, T.attention(q, A.U.DTYPES[dtype], cache, lens, rows, table, scale, causal, window))


# dtype, dim, heads_q, heads_kv, page, rows, lengths, causal, window
WALK = [
    (BF16, 128, 32, 8, 64, [1] * 80, lengths(1, 80, 1, 1200), True, 0),
    (F16, 64, 16, 16, 32, lengths(2, 10, 300, 600), lengths(3, 10, 600, 900), True, 0),
    (F16, 64, 16, 4, 16, lengths(4, 60, 1, 5), lengths(5, 60, 5, 2000), True, 256),
    (BF16, 64, 32, 8, 64, lengths(6, 40, 1, 16), lengths(7, 40, 16, 700), True, 0),   # 4 tiles of 16 rows
    (BF16, 128, 24, 8, 48, lengths(8, 20, 20, 200), lengths(9, 20, 1, 500), True, 0),  # rows before the start too
    (F16, 128, 8, 8, 256, [1] * 100, lengths(10, 100, 0, 1500), False, 0),
    (BF16, 128, 16, 4, 64, [700, 1, 1, 90, 1, 1, 1, 300] * 3, lengths(11, 24, 700, 1200), True, 0),
]


@pytest.mark.parametrize("case", WALK)
def test_runs_of_many_tiles(case):
    cache, table, width, pages, q = A.attend_inputs(case, 800, junk=False)
    check(case, cache, table, pages, q, 1 / math.sqrt(case[1]))


@pytest.mark.parametrize("hq,hk", [(32, 8), (24, 8), (16, 4), (8, 8), (16, 16), (12, 1), (64, 2), (10, 5)])
@pytest.mark.parametrize("rows", [[1, 1, 1], [2, 1, 3], [80, 17, 1]])
def test_head_layouts(hq, hk, rows):
    case = (BF16 if hq % 3 else F16, 64 if hk % 5 else 128, hq, hk, 16, rows, [500, 129, 77], True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 810, extra=8, junk=False)
    check(case, cache, table, pages, q, 1 / math.sqrt(case[1]))


@pytest.mark.parametrize("rows,length,page", [
    ([1], 40000, 64), ([5], 20000, 48), ([16], 9000, 16), ([90], 9000, 32), ([300], 3000, 256),
    ([1, 1, 2], 5000, 128)])
def test_tokens_at_every_edge(rows, length, page):
    """The tokens beside the edges of steps (and so of runs and shares) and of the
    quarters of a step, with the last of the cache, have nearly all the weight, and
    large values: each of them counts once."""
    case = (BF16, 128, 4, 2, page, rows, [length] * len(rows), True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 820, junk=False)
    j = np.arange(length)
    edge = (j % 32 == 0) | (j % 32 == 31) | (j >= length - 2)
    q[..., 0] = 4
    cache.codes[0][..., 0] = 0
    for b in range(len(rows)):
        at = table[b, j[edge] // page], j[edge] % page
        cache.codes[0][at[0], at[1], :, 0] = 7
        cache.scales[0][at] = A.U.bf16_round(0.5)
        cache.scales[1][at] *= 8
    check(case, cache, table, pages, q, 1.0)


@pytest.mark.parametrize("batch,hk", [(1, 2), (3, 2), (1, 8), (20, 4)])
@pytest.mark.parametrize("rows", [1, 6, 90])
def test_values_far_apart(rows, batch, hk):
    """Value scales some 50 binades apart and a first token with the weight and tiny
    values, cut in different ways: off by 2^-30 of a row's largest product at most
    for every token."""
    case = (BF16, 128, 4 * hk, hk, 64, [rows] * batch, [1500] * batch, True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 900, junk=False)
    rng = np.random.default_rng(5)
    cache.scales[1] = A.U.bf16_round(np.exp(rng.normal(0, 6, cache.scales[1].shape)))
    cache.scales[1][table[:, 0], 0] = A.U.bf16_round(1e-8)
    cache.scales[0][table[:, 0], 0] *= 8
    q *= 4
    check(case, cache, table, pages, q, 0.3)
