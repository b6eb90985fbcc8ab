"""GPU tests of the 4-bit products on numbers whose sums are exact in fp32 in any order, so
that one lost or doubled element shows, however long the rows: outputs equal the
definition's, rounded once.

Every kernel that a call may take is met here, in both types: few tokens staged or not, with
12 warps or 24, in one round of tiles or several; tiles of every width, cut along k or
not, one wave or more."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

EXACT = 2.0 ** 24  # numbers below it, in units of the smallest, are exact in fp32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(g, shape, low, high):
    return torch.randint(low, high + 1, shape, generator=g, device="cuda")


class Weights:
    """4-bit weights on the GPU from codes (int8 [rows, k]), scales (bytes) and row scales."""

    def __init__(self, codes, scales, row):
        self.scales, self.row, self.group = scales, row, codes.shape[1] // scales.shape[1]
        c = (codes & 15).to(torch.int32).view(codes.shape[0], -1, 8)
        word = c[..., 0]
        for e in range(1, 8):
            word = word | (c[..., e] << (4 * (e // 2) + 16 * (e % 2)))
        self.codes = word.view(torch.uint8)

    def tensors(self):
        return self.codes, self.scales, self.row

    def dense(self, rows=slice(None)):
        """fp64, through the tests' own statement of the layout."""
        codes = torch.from_numpy(U.unpack(self.codes[rows].cpu().numpy()).astype(np.int8)).cuda()
        table = torch.from_numpy(U.e4m3(np.arange(256, dtype=np.uint8))).cuda()
        scales = table[self.scales[rows].long()].repeat_interleave(self.group, 1)
        return codes.double() * scales * self.row[rows].double()[:, None]


HALF, ONE, TWO, EIGHT = 0x30, 0x38, 0x40, 0x50  # e4m3


def powers(g, n, low, high):
    return torch.exp2(ints(g, (n,), low, high).float())


def every_code(g, n, k, group):
    scales = torch.tensor([HALF, ONE, TWO], dtype=torch.uint8, device="cuda")
    return Weights(ints(g, (n, k), -8, 7).to(torch.int8), scales[ints(g, (n, k // group), 0, 2)],
                   powers(g, n, -9, -7))


LINEAR = [  # m, n, k, group
    # few tokens: one round of 64 tiles a CTA, two, three; rows that end inside a step
    (1, 40, 32, 32), (3, 1000, 352, 32), (8, 2000, 4096, 128), (1, 155648, 64, 64), (1, 155649, 64, 32),
    (8, 160001, 96, 32), (5, 170003, 544, 32), (3, 330011, 32, 32), (2, 5001, 8192, 128),
    # tiles of 32 to 256 tokens: cut along k, one wave, several
    (1, 70, 131072, 128), (2, 300, 65536, 64), (7, 300, 8224, 32), (9, 130, 32, 32), (12, 4096, 11008, 64),
    (20, 30000, 544, 32), (31, 129, 20000, 32), (33, 48, 65536, 64), (45, 5003, 4000, 32), (64, 30001, 640, 128),
    (65, 300, 32768, 128), (100, 30001, 544, 32), (128, 2000, 4128, 32), (129, 200, 65536, 128),
    (257, 1031, 2112, 64), (300, 20001, 544, 32), (700, 300, 16416, 32), (2000, 2504, 352, 32),
]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", LINEAR)
def test_linear(case, dtype):
    m, n, k, group = case
    g = gen(m + n + k)
    x, w = ints(g, (m, k), -1, 1).to(U.DTYPES[dtype]), every_code(g, n, k, group)
    assert 16 * 2 * k < EXACT  # |x| <= 1, |code| <= 8, scales from 1/2 to 2
    ys = []
    for stride in (n + -n % 8, n + 1):  # rows that are aligned and rows that are not
        ys.append(torch.full((m, stride), 7.0, dtype=x.dtype, device="cuda"))
        L.lbgemm_w4_linear(dtype, m, n, k, group, x, k, *w.tensors(), ys[-1], stride)
    L.lbgemm_device_status()
    for a in range(0, n, 8192):
        b = min(n, a + 8192)
        want = (x.double() @ w.dense(slice(a, b)).T).to(x.dtype)
        for y in ys:
            assert torch.equal(y[:, a:b], want), (a, (y[:, a:b] != want).nonzero()[:4].tolist())
    assert all((y[:, n:] == 7).all() for y in ys)


@pytest.mark.parametrize("tokens", [1, 12, 40, 100, 300])
def test_linear_beyond_32_bits(tokens):
    """2.3 GB of codes, none of them 0: rows at the ends, around 2^31 bytes and 2^32 weights."""
    n, k, group = 70001, 65536, 128
    g = gen(tokens)
    w = Weights.__new__(Weights)
    w.group, w.row = group, powers(g, n, -9, -7)
    w.codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g, device="cuda")
    w.scales = torch.tensor([HALF, ONE, TWO], dtype=torch.uint8, device="cuda")[ints(g, (n, k // group), 0, 2)]
    x = ints(g, (tokens, k), -1, 1).bfloat16()
    y = torch.empty((tokens, n), dtype=torch.bfloat16, device="cuda")
    L.lbgemm_w4_linear(0, tokens, n, k, group, x, k, *w.tensors(), y, n)
    L.lbgemm_device_status()
    for a, b in ((0, 40), (32740, 32800), (65500, 65570), (69960, n)):
        assert torch.equal(y[:, a:b], (x.double() @ w.dense(slice(a, b)).T).bfloat16()), a


# ---- experts ----------------------------------------------------------------------------------


MOE = [  # tokens, hidden, inter, experts, top, group, picks
    # few picks, 12 warps: staged; from L1 (up, down); several rounds (up, down)
    (1, 32, 32, 1, 1, 32, "any"), (8, 4096, 2048, 3, 2, 128, "any"), (16, 2560, 1344, 5, 1, 64, "holes"),
    (2, 64, 2048, 16, 8, 32, "spread"), (2, 4096, 32, 16, 8, 32, "spread"), (1, 4128, 1888, 16, 16, 32, "spread"),
    (8, 2560, 1888, 16, 2, 32, "spread"),
    # 24 warps: staged; from L1; several rounds (up, down)
    (24, 256, 96, 9, 2, 32, "any"), (24, 2048, 160, 60, 6, 32, "any"), (16, 96, 1312, 64, 4, 32, "spread"),
    (18, 640, 96, 72, 4, 32, "spread"), (50, 64, 640, 200, 8, 64, "any"), (36, 64, 2560, 72, 2, 64, "spread"),
    (40, 1024, 1024, 80, 2, 128, "spread"),
    # tiles of 32, 64, 128 and 256 picks, the second product in as many or 128
    (200, 128, 96, 90, 8, 32, "holes"), (129, 1056, 544, 40, 4, 32, "any"), (400, 256, 160, 20, 3, 32, "any"),
    (300, 256, 160, 5, 2, 32, "any"), (239, 96, 2080, 2, 1, 32, "holes"),
    (300, 256, 2112, 2, 2, 64, "any"), (517, 384, 4096, 3, 1, 128, "holes"), (700, 2080, 2080, 5, 2, 32, "any"),
    (300, 1088, 416, 2, 1, 32, "one"), (1000, 96, 2048, 3, 2, 32, "twice"),
]


def moe_ids(g, tokens, experts, top, kind):
    if kind == "spread":  # every pick an expert of its own
        assert tokens * top <= experts
        return torch.randperm(experts, generator=g, device="cuda")[:tokens * top].view(tokens, top)
    ids = torch.rand((tokens, experts), generator=g, device="cuda").topk(min(top, experts), 1).indices
    if kind == "holes":
        ids[torch.rand((tokens, top), generator=g, device="cuda") < 0.25] = -1
        ids[::5] = -1
    elif kind == "one":
        ids[:] = experts - 1
    elif kind == "twice":
        ids[:, -1] = ids[:, 0]
    return ids


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", MOE)
def test_moe(case, dtype):
    """Every gate's sum is 32, of which silu is 32 itself in fp32 (exp(-32) < 2^-25), so the
    inner vector is 32 times the up row's sum: up to 128 of it are exact in bf16 and fp16."""
    tokens, hidden, inter, experts, top, group, kind = case
    g = gen(tokens + hidden + inter)
    x = ints(g, (tokens, hidden), -1, 1)
    x[:, 0] = 1
    n = experts * inter
    codes = torch.zeros((n, 2, hidden), dtype=torch.int8, device="cuda")
    codes[:, 0, 0] = 4
    some = torch.rand((n, hidden), generator=g, device="cuda") < min(1.0, 24 / hidden)
    codes[:, 1] = (ints(g, (n, hidden), 0, 1) * 2 - 1).to(torch.int8) * some
    scales = torch.full((n, 2, hidden // group), ONE, dtype=torch.uint8, device="cuda")
    scales[:, 0, 0] = EIGHT
    row = torch.ones((n, 2), device="cuda")
    row[:, 1] = powers(g, n, -1, 1)
    up = Weights(codes.view(2 * n, hidden), scales.view(2 * n, -1), row.view(-1))
    down = every_code(g, experts * hidden, inter, group)
    ids = moe_ids(g, tokens, experts, top, kind).to(torch.int32).contiguous()
    share = powers(g, tokens * top, -3, -1).view(tokens, top)
    x = x.to(U.DTYPES[dtype])
    y = torch.full((tokens + 1, hidden), 7.0, dtype=x.dtype, device="cuda")
    L.lbgemm_moe_w4(dtype, tokens, hidden, inter, experts, top, group, x, hidden, ids, share, *up.tensors(),
                    *down.tensors(), y, hidden)
    L.lbgemm_device_status()

    want, size = (torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda") for _ in range(2))
    for e in set(ids.flatten().tolist()) - {-1}:
        who = (ids == e).any(1).nonzero()[:, 0]
        both = (x[who].double() @ up.dense(slice(2 * e * inter, 2 * (e + 1) * inter)).T).view(-1, inter, 2)
        assert (both[..., 0] == 32).all() and both[..., 1].abs().max() <= 128
        d = down.dense(slice(e * hidden, (e + 1) * hidden))
        w = (share[who].double() * (ids[who] == e)).sum(1)[:, None]
        pick = 32 * both[..., 1] @ d.T
        # a pick's sums before their row scale, in units of 32 / 2 of the inner vector times 1/2
        # of the weights; then the sum over the picks, by shares of 2^-3 and more
        scale = down.row[e * hidden:(e + 1) * hidden].double()
        assert (32 * both[..., 1].abs() @ (d.abs() / scale[:, None]).T).max() < EXACT * 8
        want[who] += w * pick
        size[who] += w * (pick / scale).abs()
    # (experts' row scales are within 4 of one another)
    assert size.max() < EXACT / 4
    assert torch.equal(y[:tokens], want.to(x.dtype)), (y[:tokens] != want.to(x.dtype)).nonzero()[:4].tolist()
    assert (y[tokens] == 7).all()
