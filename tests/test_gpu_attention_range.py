"""GPU tests of attention over cached values of every size that a bf16 scale can
hold, within the bounds of attention_tight.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_tight as T  # noqa: E402
import test_gpu_attention as A  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

BF16 = L.BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


def value_scales(kind, scales, rng):
    """scales [tokens, heads] of the values, as `kind` has them; and the token that
    takes most of the weight (None: none does)."""
    n = len(scales)
    if kind == "huge":  # values up to 2^127
        scales[:] = 2.0 ** 124
    elif kind == "tiny":
        scales[:] = 1e-36 * np.exp(rng.normal(0, 1, scales.shape))
    elif kind == "below the normal range":
        scales[:] = 2.0 ** -130
    elif kind == "one huge":
        scales[n // 2] = 2.0 ** 124
    elif kind == "one tiny with the weight":
        scales[n // 3] = 1e-36
        return n // 3
    elif kind == "all but one tiny":
        scales[:] = 1e-37
        scales[n - 2] = 1.0
    elif kind == "growing":
        scales[:] = 2.0 ** np.linspace(-125, 124, n)[:, None]
    elif kind == "falling":
        scales[:] = 2.0 ** np.linspace(124, -125, n)[:, None]
    elif kind == "huge, the last ones ordinary with the weight":
        scales[:n - 1] = 2.0 ** 120
        return n - 1
    return None


KINDS = ["huge", "tiny", "below the normal range", "one huge", "one tiny with the weight",
         "all but one tiny", "growing", "falling", "huge, the last ones ordinary with the weight"]


def check_kind(kind, rows, dim, length=700):
    case = (BF16, dim, 4, 2, 16, [rows], [length], True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 640, junk=False)
    rng = np.random.default_rng(12)
    at = table[0, np.arange(length) // 16], np.arange(length) % 16
    s = cache.scales[1][at]
    heavy = value_scales(kind, s, rng)
    cache.scales[1][at] = A.U.bf16_round(s)
    if heavy is not None:  # its key is along every query: they get one more channel of one sign
        q[..., 0] = 4
        cache.codes[0][..., 0] = 0
        cache.codes[0][at[0][heavy], at[1][heavy], :, 0] = 7
        cache.scales[0][at[0][heavy], at[1][heavy]] = 8.0
    scale = 1 / math.sqrt(dim)
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, case[6], scale)
    L.lbgemm_device_status()
    ref = T.attention(q, torch.bfloat16, cache, case[6], case[5], table, scale, True, 0)
    T.check(o, lse, ref)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,dim", [(1, 128), (6, 64), (30, 128)])
def test_value_scales_few_rows(kind, rows, dim):
    check_kind(kind, rows, dim)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,dim", [(90, 64), (400, 128)])
def test_value_scales_many_rows(kind, rows, dim):
    check_kind(kind, rows, dim)


@pytest.mark.parametrize("rows", [1, 6, 30, 90])
def test_shares_of_the_largest_values(rows):
    """Every value near the largest that a bf16 output holds: so is the result, whose
    shares a join must not add up past it."""
    length, dim = 1500, 64
    case = (BF16, dim, 4, 2, 16, [rows], [length], True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 641, junk=False)
    cache.codes[1][:] = 7
    cache.scales[1][:] = 2.0 ** 125  # 7 * 2^125 = 2.98e38
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, case[6], 0.125)
    L.lbgemm_device_status()
    T.check(o, lse, T.attention(q, torch.bfloat16, cache, case[6], case[5], table, 0.125, True, 0))


@pytest.mark.parametrize("above", [100, 126, 127, 130, 140, 147])
@pytest.mark.parametrize("rows", [1, 6, 30, 90])
def test_shares_far_below_the_largest(rows, above):
    """One token's weight 2^above times the others' and its values 2^-above theirs:
    both count, in shares of their own too."""
    length, dim = 1500, 64
    case = (BF16, dim, 4, 2, 16, [rows], [length], True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 642, junk=False)
    at = table[0, np.arange(length) // 16], np.arange(length) % 16
    heavy, scale = length // 3, 0.125
    q[..., 0] = 4
    cache.codes[0][..., 0] = 0
    cache.codes[0][at[0][heavy], at[1][heavy]] = 0
    cache.codes[0][at[0][heavy], at[1][heavy], :, 0] = 7
    # 4 * 7 * ks / 8 = above ln 2, within the rounding of ks
    cache.scales[0][at[0][heavy], at[1][heavy]] = A.U.bf16_round(above * math.log(2) / 3.5)
    cache.scales[1][at[0][heavy], at[1][heavy]] = max(2.0 ** -above, 2.0 ** -126)
    cache.codes[1][at[0][heavy], at[1][heavy]] = np.arange(dim) % 2 * 7
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, case[6], scale)
    L.lbgemm_device_status()
    T.check(o, lse, T.attention(q, torch.bfloat16, cache, case[6], case[5], table, scale, True, 0))


def check_queries(case, q, scale, seed):
    dtype, dim, hq, hk, page, rows, lens, causal, window = case
    cache, table, width, pages, _ = A.attend_inputs(case, seed)
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, scale)
    L.lbgemm_device_status()
    used = A.U.Cache(cache.pages, page, hk, dim)
    used.codes, used.scales = cache.codes, np.nan_to_num(cache.scales, nan=0.0, posinf=0.0)
    T.check(o, lse, T.attention(q, A.U.DTYPES[dtype], used, lens, rows, table, scale, causal, window))


@pytest.mark.parametrize("size", [1e36, 3e37, 1e-36])
@pytest.mark.parametrize("rows,dim", [([1], 128), ([6, 2], 64), ([30], 64), ([90, 300], 128)])
def test_query_sizes(rows, dim, size):
    """Queries near the ends of bf16's range, with a scale that makes ordinary scores."""
    case = (BF16, dim, 4, 2, 16, rows, [700, 400][:len(rows)], True, 0)
    q = A.rand(7, (sum(rows), 4, dim), BF16, 1.0) * size
    check_queries(case, q, 2.0 / math.sqrt(dim) / size, 650)


@pytest.mark.parametrize("apart", [2.0 ** 16, 2.0 ** 30, 2.0 ** 45, 2.0 ** 90])
@pytest.mark.parametrize("rows,dim,hq", [([1], 128, 4), ([6, 2], 64, 4), ([30], 64, 8), ([90, 300], 128, 4)])
def test_queries_beside_larger_ones(rows, dim, hq, apart):
    """A row is what it is whatever its neighbours are: rows of ordinary size beside
    some that are far larger, beside zeros, and rows spread over the whole span."""
    case = (BF16, dim, hq, 2, 16, rows, [700, 400][:len(rows)], True, 0)
    q = A.rand(8, (sum(rows), hq, dim), BF16, 1.0)
    q[0, 1] *= apart
    q[-1, 2] *= 1 / apart
    q[-1, 0] = 0
    if sum(rows) > 30:
        q[5:20] *= apart ** (torch.rand((15, hq, 1), generator=torch.Generator().manual_seed(9)) - 0.5).bfloat16().cuda()
        q[23] = 0
    check_queries(case, q, 1.0 / math.sqrt(dim), 651)


FAR = 2.0 ** -100  # weights below that of a row's largest may count as 0
SHAPES = [
    (64, 8, 8, [1] * 30, [66] * 30, True, 0), (64, 14, 2, [8, 6], [280, 260], False, 0),
    (128, 8, 2, [3] * 20, [35] * 20, True, 0), (64, 12, 3, [90] * 10, [300] * 10, True, 33),
    (128, 6, 3, [278, 90], [285, 100], True, 0), (64, 32, 8, [146, 299], [12, 40], False, 0),
    (128, 14, 2, [2, 1, 5], [700, 33, 300], True, 50)]


@pytest.mark.parametrize("spread", [40, 80])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("keys", [0, 2])
def test_value_scales_over_the_whole_range(shape, spread, keys):
    """Value scales 2^(40 x) and 2^(80 x), x normal, under scores of ordinary and of
    large size: tokens with tiny weights decide rows, one at a time."""
    dim, hq, hk, rows, lens, causal, window = shape
    case = (BF16, dim, hq, hk, 16, rows, lens, causal, window)
    cache, table, width, pages, q = A.attend_inputs(case, 660, junk=False)
    rng = np.random.default_rng(spread + keys)
    cache.scales[1] = A.U.bf16_round(2.0 ** np.clip(rng.normal(0, spread, cache.scales[1].shape), -126, 120))
    if keys:
        cache.scales[0] = A.U.bf16_round(2.0 ** rng.normal(0, keys, cache.scales[0].shape))
    for scale in (0.01, 0.125, 1.0):
        o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, scale)
        L.lbgemm_device_status()
        T.check(o, lse, T.attention(q, torch.bfloat16, cache, lens, rows, table, scale, causal, window, FAR))


@pytest.mark.parametrize("what", ["keys", "queries", "both"])
@pytest.mark.parametrize("shape", SHAPES)
def test_scores_past_the_ulp_of_a_binade(shape, what):
    """Scores from 1e6 to 1e30, where fp32 numbers are more than a binade's exponent
    apart: one token has a row's weight, and the row is its value."""
    dim, hq, hk, rows, lens, causal, window = shape
    case = (BF16, dim, hq, hk, 16, rows, lens, causal, window)
    cache, table, width, pages, q = A.attend_inputs(case, 661, junk=False)
    rng = np.random.default_rng(3)
    if what != "queries":
        cache.scales[0] = A.U.bf16_round(2.0 ** rng.normal(0, 7, cache.scales[0].shape))
    if what != "keys":
        q = q * (2.0 ** torch.from_numpy(np.clip(rng.normal(0, 20, (*q.shape[:2], 1)), -60, 70)).cuda()).bfloat16()
    for scale in (0.01, -1.0):
        o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, scale)
        L.lbgemm_device_status()
        T.check(o, lse, T.attention(q, torch.bfloat16, cache, lens, rows, table, scale, causal, window, FAR))


@pytest.mark.parametrize("size", [2.0 ** 24, 2.0 ** 27, 2.0 ** 30])
@pytest.mark.parametrize("rows,dim,first", [([1], 128, 20), ([6, 2], 64, 33), ([90, 300], 128, 1), ([70], 64, 64)])
def test_lesser_scores_after_huge_negative_ones(rows, dim, first, size):
    """Rows whose first tokens have scores of some -2 `size`: what comes after them,
    scores of some thousands, sets the row as if they were not there."""
    lens = [700, 400][:len(rows)]
    case = (BF16, dim, 4, 2, 16, rows, lens, True, 0)
    cache, table, width, pages, q = A.attend_inputs(case, 662, junk=False)
    j = np.arange(first)
    q[..., 0] = 4
    cache.scales[0] = A.U.bf16_round(cache.scales[0] * 1000)
    for b in range(len(rows)):
        at = table[b, j // 16], j % 16
        cache.codes[0][at] = 0
        cache.codes[0][at[0], at[1], :, 0] = -7
        cache.scales[0][at] = A.U.bf16_round(size)
    scale = 1 / math.sqrt(dim)
    o, lse = A.attend(case, q, A.to_torch(cache), pages, table, lens, scale)
    L.lbgemm_device_status()
    # their own tokens' scores do not count in the bounds: nothing is left of them
    kept = A.U.Cache(cache.pages, 16, 2, dim)
    kept.codes, kept.scales = cache.codes, cache.scales.copy()
    for b in range(len(rows)):
        kept.codes[0][table[b, j // 16], j % 16, :, 0] = -7
        kept.scales[0][table[b, j // 16], j % 16] = 2.0 ** 14
    T.check(o, lse, T.attention(q, torch.bfloat16, kept, lens, rows, table, scale, True, 0, FAR))
