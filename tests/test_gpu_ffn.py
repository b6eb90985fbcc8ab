"""GPU tests of the feed-forward operators against their 64-bit definitions.

Bounds, from the arithmetic: an output is rounded once (ROUND of itself).  A sum of
products in fp32 along k elements is off by at most 2^-22 of the sum of the
products' sizes for each of the k / 16 steps of the matrix units and 64 more
additions where parts are joined: SUM(k).  Norms: a sum of squares is a tree of
positive numbers, and with the reciprocal root and a handful of products each
factor is off by less than 2^-19 of itself; 2^-18 of the sizes that enter covers
two of them in a row."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

NORM = 2.0 ** -18


def SUM(k):
    return (k / 16 + 64) * 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


def rows(rng, tokens, width, dtype, pad=0, size=1.0):
    """[tokens, width] of a wider buffer, channels of different sizes."""
    x = rng.normal(0, size, (tokens, width + pad)) * np.exp(rng.normal(0, 0.4, width + pad))
    return torch.from_numpy(x).to(U.DTYPES[dtype]).cuda()[:, :width]


def framed(tokens, width, stride, dtype):
    """An output [tokens, width] with a given stride inside a buffer of a known value."""
    buf = torch.full((tokens * stride + 64,), 7.0, dtype=U.DTYPES[dtype], device="cuda")
    out = buf[:tokens * stride].view(tokens, stride)[:, :width] if tokens else buf[:0].view(0, width)
    def untouched():
        mask = torch.ones_like(buf, dtype=torch.bool)
        if tokens:
            mask[:tokens * stride].view(tokens, stride)[:, :width] = False
        return bool((buf[mask] == 7.0).all())
    return out, untouched


# ---- 4-bit weights ---------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (5, 96, 32), (33, 640, 64), (17, 4224, 128)])
def test_quantize(dtype, n, k, group):
    rng = np.random.default_rng(n + k)
    w = rows(rng, n, k, dtype, pad=16)
    w[n // 2, :group] = 0
    codes, cs = torch.full((n, k // 2 + 16), 9, dtype=torch.uint8, device="cuda"), k // 2 + 16
    scales = torch.full((n, k // group + 3), 9, dtype=torch.uint8, device="cuda")
    row = torch.full((n, 2), -1.0, device="cuda")
    L.lbgemm_w4_quantize(dtype, n, k, group, w, k + 16, codes, cs, scales, k // group + 3, row, 2)
    L.lbgemm_device_status()
    want = U.quantise(w.float().cpu().numpy(), group)
    got = U.unpack(codes[:, :k // 2].cpu().numpy())
    assert np.array_equal(row[:, 0].cpu().numpy(), want[2])
    assert np.array_equal(scales[:, :k // group].cpu().numpy(), want[1])
    assert np.array_equal(got, want[0])
    assert (codes[:, k // 2:] == 9).all() and (scales[:, k // group:] == 9).all()
    assert (row[:, 1] == -1).all()


def test_quantize_special_rows():
    w = torch.ones((6, 64), device="cuda")
    w[1], w[2, 5], w[3, 63], w[4] = 0, float("inf"), float("nan"), 1e-44
    w[5] = torch.linspace(-3e38, 3e38, 64)
    codes = torch.empty((6, 32), dtype=torch.uint8, device="cuda")
    scales = torch.empty((6, 2), dtype=torch.uint8, device="cuda")
    row = torch.empty(6, device="cuda")
    L.lbgemm_w4_quantize(L.F32, 6, 64, 32, w, 64, codes, 32, scales, 2, row)
    want = U.quantise(w.cpu().numpy(), 32)
    assert np.array_equal(row.cpu().numpy(), want[2], equal_nan=True)
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(U.unpack(codes.cpu().numpy()), want[0])


LINEAR = [  # dtype, m, n, k, group, x pad, y stride beyond n
    (0, 1, 1, 32, 32, 0, 0), (1, 1, 40, 96, 32, 8, 3), (0, 1, 4096, 4096, 128, 0, 0),
    (0, 2, 333, 1024, 64, 16, 1), (1, 3, 130, 4096, 128, 0, 0), (0, 7, 1000, 352, 32, 8, 0),
    (1, 8, 257, 11008, 64, 0, 7), (0, 9, 511, 2080, 32, 0, 0), (0, 16, 2049, 768, 64, 0, 2),
    (1, 17, 96, 4096, 128, 8, 0), (0, 31, 777, 1312, 32, 0, 0), (0, 33, 128, 640, 128, 0, 0),
    (1, 45, 503, 4000, 32, 0, 1), (0, 64, 1280, 2048, 64, 0, 0), (0, 65, 129, 160, 32, 8, 5),
    (1, 100, 2000, 1024, 128, 0, 0), (0, 128, 640, 8192, 64, 0, 0), (0, 200, 100, 96, 32, 0, 0),
    (1, 255, 384, 1408, 128, 0, 0), (0, 257, 1031, 2112, 64, 8, 1), (0, 700, 2500, 1056, 32, 0, 0),
    (1, 1500, 513, 512, 128, 0, 0), (0, 1, 9, 16384, 128, 0, 0), (0, 16, 9, 16384, 128, 0, 0),
    (1, 5, 20000, 64, 64, 0, 0), (0, 2, 70, 131072, 128, 0, 0), (0, 30, 48, 65536, 64, 0, 0),
]


@pytest.mark.parametrize("case", LINEAR)
def test_linear(case):
    dtype, m, n, k, group, pad, ypad = case
    rng = np.random.default_rng(m * 7 + n)
    x, w = rows(rng, m, k, dtype, pad), U.Weights(rng, n, k, group)
    y, untouched = framed(m, n, n + ypad, dtype)
    L.lbgemm_w4_linear(dtype, m, n, k, group, x, k + pad, *w.tensors(), y, n + ypad)
    L.lbgemm_device_status()
    xd, wd = x.double(), w.dense()
    want = xd @ wd.T
    tol = U.ROUND[dtype] * want.abs() + SUM(k) * (xd.abs() @ wd.abs().T)
    assert ((y.double() - want).abs() <= tol).all()
    assert untouched()


def test_linear_every_scale():
    """Every e4m3 scale but NaN with every code, one product at a time: exact."""
    for dtype in (0, 1):
        scales = np.array([b for b in range(256) if b & 127 != 127], np.uint8)
        rng = np.random.default_rng(3)
        w = U.Weights(rng, len(scales), 32, 32, scales=scales[:, None])
        w.row[:] = 1.0
        x = torch.zeros((32, 32), dtype=U.DTYPES[dtype], device="cuda")
        x[torch.arange(32), torch.arange(32)] = 1.0
        for part in (1, 32):  # few tokens, many
            y = torch.empty((32, 256), dtype=U.DTYPES[dtype], device="cuda")  # (aligned rows)
            for a in range(0, 32, part):
                L.lbgemm_w4_linear(dtype, part, len(scales), 32, 32, x[a:], 32, *w.tensors(), y[a:],
                                   256)
            assert torch.equal(y[:, :len(scales)].double(), w.dense().T)


def test_linear_keeps_to_its_inputs():
    """NaN and infinity of a token, of a weight row and behind the tensors stay there."""
    for m in (3, 40, 300):
        rng = np.random.default_rng(m)
        k, n, group = 160, 150, 32
        x, w = rows(rng, m, k, 0, pad=8), U.Weights(rng, n, k, group)
        x[1, 5], x[2, 0] = float("nan"), float("inf")
        w.row[7] = np.nan
        w.scales[9, 2] = 0x7f
        whole = torch.full((m + 300, k + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
        whole[:m, :k] = x
        y = torch.empty((m, n), dtype=torch.bfloat16, device="cuda")
        L.lbgemm_w4_linear(0, m, n, k, group, whole, k + 8, *w.tensors(), y, n)
        bad = torch.zeros((m, n), dtype=torch.bool, device="cuda")
        bad[1:3], bad[:, 7], bad[:, 9] = True, True, True
        assert (~torch.isfinite(y[bad])).all() and torch.isfinite(y[~bad]).all()


@pytest.mark.parametrize("k", [4096, 8192, 8320, 11008])
def test_linear_one_token_of_any_stride(k):
    """A single row's strides are not looked at, whichever kernel takes it."""
    rng = np.random.default_rng(k)
    x, w = rows(rng, 1, k, 0), U.Weights(rng, 203, k, 64)
    y, again = (torch.empty((1, 203), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    L.lbgemm_w4_linear(0, 1, 203, k, 64, x, k, *w.tensors(), y, 203)
    L.lbgemm_w4_linear(0, 1, 203, k, 64, x, 3, *w.tensors(), again, 1)
    L.lbgemm_device_status()
    want, size = x.double() @ w.dense().T, x.double().abs() @ w.dense().abs().T
    assert ((y.double() - want).abs() <= U.ROUND[0] * want.abs() + SUM(k) * size).all()
    assert torch.equal(y, again)


@pytest.mark.parametrize("m", [7, 8, 9, 16, 31, 33, 64, 65, 95, 97, 128, 129, 161, 224, 255, 257, 290, 513])
def test_linear_around_the_widths_of_tiles(m):
    """Blocks of tokens that a kernel fills, and one more; every token on its own."""
    rng = np.random.default_rng(m)
    n, k, group = 270, 544, 32
    x, w = rows(rng, m, k, 1), U.Weights(rng, n, k, group)
    y, untouched = framed(m, n, n + 2, 1)
    L.lbgemm_w4_linear(1, m, n, k, group, x, k, *w.tensors(), y, n + 2)
    L.lbgemm_device_status()
    want, size = x.double() @ w.dense().T, x.double().abs() @ w.dense().abs().T
    assert ((y.double() - want).abs() <= U.ROUND[1] * want.abs() + SUM(k) * size + 2.0 ** -25).all()
    assert untouched()


# ---- the router ----------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("tokens,experts,top,renormalize,pad", [
    (1, 1, 1, True, 0), (5, 2, 2, False, 1), (33, 60, 4, True, 3), (130, 64, 6, False, 0),
    (7, 128, 8, True, 0), (64, 257, 16, False, 5), (3, 1024, 32, True, 0), (9, 500, 1, False, 0)])
def test_route(dtype, tokens, experts, top, renormalize, pad):
    rng = np.random.default_rng(experts)
    l = rng.normal(0, 1.5, (tokens, experts + pad))
    l = np.round(l * 8) / 8  # many equal ones
    t = torch.from_numpy(l).to(U.DTYPES[dtype]).cuda()
    check_route(dtype, t, experts, top, renormalize)


def check_route(dtype, t, experts, top, renormalize):
    tokens = t.shape[0]
    ids = torch.full((tokens + 1, top), 77, dtype=torch.int32, device="cuda")
    weights = torch.full((tokens + 1, top), 7.0, device="cuda")
    L.lbgemm_moe_route(dtype, tokens, experts, top, t, t.stride(0), renormalize, ids, weights)
    L.lbgemm_device_status()
    l = t[:, :experts].double().cpu().numpy()
    want_ids, want = U.route(l, top, renormalize)
    assert np.array_equal(ids[:tokens].cpu().numpy(), want_ids)
    # exp's own error (2 ulp), its argument's rounding, a sum of up to 1024 numbers
    usable = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    tall = np.where(want_ids >= 0, np.take_along_axis(usable, np.maximum(want_ids, 0), 1), 0)
    span = np.where(want_ids >= 0, tall[:, :1] - tall, 0)
    spread = np.minimum(np.max(np.where(usable > -np.inf, tall[:, :1] - usable, 0), 1), 20)[:, None]
    tol = want * 2.0 ** -24 * (48 + span + spread) + 2.0 ** -149
    got = weights[:tokens].double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        assert (np.abs(got - want) <= tol).all()
    assert (ids[tokens] == 77).all() and (weights[tokens] == 7).all()


@pytest.mark.parametrize("renormalize", [True, False])
def test_route_odd_logits(renormalize):
    inf, nan = float("inf"), float("nan")
    l = torch.zeros((8, 40), device="cuda")
    l[0] = -inf
    l[1] = nan
    l[2, :38] = -inf
    l[3, 11], l[3, 5] = inf, inf
    l[4, ::2] = -0.0
    l[5, 7], l[5, 9], l[5, 3] = nan, 2.0, -inf
    l[6] = torch.linspace(-3e38, 3e38, 40)
    l[7, 1:] = -1e30
    check_route(2, l, 40, 4, renormalize)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("experts", [40, 1024])
def test_route_odd_logits_of_16_bits(dtype, experts):
    """A key holds the expert too: the largest and smallest numbers, signs, subnormals."""
    t = U.DTYPES[dtype]
    inf, nan, most = float("inf"), float("nan"), torch.finfo(t).max
    tiny = torch.finfo(t).smallest_normal * torch.finfo(t).eps
    l = torch.zeros((9, experts), device="cuda").to(t)
    l[0], l[1] = -inf, nan
    l[2, :-2] = -inf
    l[3, 5], l[3, 11], l[3, 3] = most, inf, most
    l[4, ::2] = -0.0
    l[5, 7], l[5, 9], l[5, 3] = nan, 2.0, -inf
    l[6, 1::2], l[6, 20] = -tiny, tiny
    l[7] = -most
    l[7, -1] = -most * (1 - torch.finfo(t).eps)
    l[8, :-3], l[8, -1] = inf, -1.0
    for top, renormalize in ((4, True), (32, False)):
        check_route(dtype, l, experts, top, renormalize)


# ---- experts ----------------------------------------------------------------------------------


def experts_want(x, ids, weights, up, down, hidden, inter, dtype):
    """The definition, and the bound that goes with it."""
    tokens, experts = x.shape[0], up.codes.shape[0] // (2 * inter)
    y = torch.zeros((tokens, hidden), dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    r, xd = U.ROUND[dtype], x.double()
    wu, wd = up.dense(), down.dense()
    for e in range(experts):
        w = (weights.double() * (ids == e)).sum(1)
        who = (ids == e).any(1).nonzero()[:, 0]
        if who.numel() == 0:
            continue
        a = wu[e * 2 * inter:(e + 1) * 2 * inter]
        gu = xd[who] @ a.T
        off = SUM(hidden) * (xd[who].abs() @ a.abs().T)
        g, u = gu[:, ::2], gu[:, 1::2]
        act = g * torch.sigmoid(g)
        h = act * u
        # |silu'| <= 1.1; exp and the division: 2^-21 of the value
        h_off = 1.1 * off[:, ::2] * u.abs() + act.abs() * off[:, 1::2] + off[:, ::2] * off[:, 1::2] * 1.1
        h_off = h_off + (r + 2.0 ** -21) * (h.abs() + h_off)
        if dtype == 1:
            h_off = h_off + 2.0 ** -25  # half a step of fp16's smallest numbers
        d = wd[e * hidden:(e + 1) * hidden]
        y[who] += w[who, None] * (h @ d.T)
        size = (h.abs() + h_off) @ d.abs().T
        tol[who] += w[who, None].abs() * (h_off @ d.abs().T + SUM(inter) * size)
    return y, tol + r * y.abs() + 2.0 ** -22 * y.abs()


def picks(rng, tokens, experts, top, kind):
    ids = np.stack([rng.permutation(experts)[:top] for _ in range(tokens)]) if top <= experts else \
        rng.integers(0, experts, (tokens, top))
    if kind == "holes":
        ids[rng.random((tokens, top)) < 0.3] = -1
        ids[::3] = -1
    elif kind == "one":
        ids[:] = experts - 1
        ids[:, 1:] = -5
    elif kind == "none":
        ids[:] = -1
    elif kind == "twice":
        ids[:, -1] = ids[:, 0]
    weights = rng.random((tokens, top)) + 0.1
    return ids.astype(np.int32), (weights / weights.sum(1, keepdims=True)).astype(np.float32)


MOE = [  # dtype, tokens, hidden, inter, experts, top, group, kind, pad
    (0, 1, 32, 32, 1, 1, 32, "all", 0), (0, 1, 2048, 1024, 16, 6, 128, "all", 0),
    (1, 2, 256, 96, 5, 2, 32, "all", 8), (0, 3, 640, 128, 8, 8, 64, "holes", 0),
    (0, 7, 512, 256, 4, 1, 64, "one", 0), (1, 16, 384, 640, 9, 3, 128, "twice", 0),
    (0, 24, 2048, 512, 32, 6, 64, "all", 0), (0, 33, 96, 160, 60, 4, 32, "holes", 16),
    (1, 64, 1024, 352, 3, 2, 32, "all", 0), (0, 100, 256, 128, 200, 8, 64, "all", 0),
    (0, 129, 128, 64, 2, 2, 64, "none", 0), (0, 257, 512, 192, 6, 2, 64, "all", 8),
    (1, 300, 384, 256, 7, 3, 128, "one", 0), (0, 513, 1088, 416, 10, 4, 32, "holes", 0),
    (0, 1000, 256, 128, 128, 8, 128, "all", 0), (0, 20, 64, 32, 3, 5, 32, "twice", 0),
    (1, 2000, 128, 96, 33, 2, 32, "all", 0), (0, 12, 4096, 2048, 4, 2, 128, "all", 0),
]


@pytest.mark.parametrize("case", MOE)
def test_moe(case):
    dtype, tokens, hidden, inter, experts, top, group, kind, pad = case
    rng = np.random.default_rng(tokens + hidden)
    x = rows(rng, tokens, hidden, dtype, pad)
    up, down = (U.Weights(rng, experts * n, k, group) for n, k in ((2 * inter, hidden), (hidden, inter)))
    ids, weights = (torch.from_numpy(a).cuda() for a in picks(rng, tokens, experts, top, kind))
    y, untouched = framed(tokens, hidden, hidden + pad, dtype)
    L.lbgemm_moe_w4(dtype, tokens, hidden, inter, experts, top, group, x, hidden + pad, ids, weights,
                    *up.tensors(), *down.tensors(), y, hidden + pad)
    L.lbgemm_device_status()
    want, tol = experts_want(x, ids, weights, up, down, hidden, inter, dtype)
    assert ((y.double() - want).abs() <= tol).all()
    assert untouched()
    nothing = (ids < 0).all(1)
    assert (y[nothing] == 0).all()


@pytest.mark.parametrize("tokens", [2, 70])
def test_moe_reports_bad_ids(tokens):
    rng = np.random.default_rng(5)
    hidden, inter, experts, group = 128, 64, 6, 32
    x = rows(rng, tokens, hidden, 0)
    up, down = (U.Weights(rng, experts * n, k, group) for n, k in ((2 * inter, hidden), (hidden, inter)))
    ids, weights = (torch.from_numpy(a).cuda() for a in picks(rng, tokens, experts, 2, "all"))
    ids[1, 0] = experts
    y = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
    call = lambda: L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, 2, group, x, hidden, ids,  # noqa: E731
                                   weights, *up.tensors(), *down.tensors(), y, hidden)
    call()
    with pytest.raises(L.LbgemmError) as e:
        L.lbgemm_device_status()
    assert e.value.status == L.ERR_INVALID_ARG
    want, tol = experts_want(x, ids, weights, up, down, hidden, inter, 0)  # (it adds nothing)
    assert ((y.double() - want).abs() <= tol).all()
    ids[1, 0] = 0
    call()
    L.lbgemm_device_status()


@pytest.mark.parametrize("tokens", [1, 4, 50, 400])
def test_moe_same_bits(tokens):
    """Two calls give the same bits, and a token keeps its result whatever an
    infinity in another token does."""
    rng = np.random.default_rng(tokens)
    hidden, inter, experts, group, top = 256, 128, 8, 64, 3
    x = rows(rng, tokens, hidden, 0)
    up, down = (U.Weights(rng, experts * n, k, group) for n, k in ((2 * inter, hidden), (hidden, inter)))
    ids, weights = (torch.from_numpy(a).cuda() for a in picks(rng, tokens, experts, top, "all"))
    ys = []
    for i in range(3):
        if i == 2 and tokens > 1:
            x[0] = float("inf")
        y = torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda")
        L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, top, group, x, hidden, ids, weights,
                        *up.tensors(), *down.tensors(), y, hidden)
        ys.append(y)
    L.lbgemm_device_status()
    assert torch.equal(ys[0], ys[1])
    if tokens > 1:
        assert torch.equal(ys[0][1:], ys[2][1:]) and not torch.isfinite(ys[2][0]).any()


# ---- norms around a block ----------------------------------------------------------------------


NORMS = [  # dtype, tokens, width, post, gate, next, pad, a, b
    (0, 1, 8, True, "none", True, 0, 1.0, 1.0), (0, 16, 4096, True, "none", True, 0, 1.0, 0.75),
    (1, 33, 256, True, "channel", True, 8, 0.5, 2.0), (2, 1021, 1000, True, "token", True, 0, 1.0, 1.0),
    (0, 700, 264, False, "channel", True, 8, 1.0, -0.25), (2, 65, 72, True, "channel", False, 4, 2.0, 1.0),
    (0, 300, 2048, False, "none", True, 0, 1.0, 1.0), (1, 77, 5120, True, "token", True, 0, 1.0, 0.1),
    (0, 40, 16384, True, "token", True, 0, 1.0, 1.0), (2, 19, 8192, True, "token", True, 0, 1.0, 1.0),
    (0, 1500, 512, True, "token", False, 0, 0.0, 1.0), (1, 5, 1024, False, "none", False, 0, 1.0, 1.0),
    (2, 3001, 128, True, "channel", True, 0, 1.0, 1.0), (0, 2000, 6144, True, "channel", True, 0, 1.0, 1.0),
    (1, 1300, 2064, True, "token", True, 8, 1.0, 1.0), (0, 1700, 4096, True, "channel", True, 0, 1.0, 0.5),
    (2, 1301, 4088, True, "token", True, 0, 1.0, 1.0), (2, 150, 5128, True, "channel", True, 4, 1.0, 1.0),
    (2, 35, 8192, True, "channel", True, 0, 1.0, 1.0), (0, 160, 7176, False, "token", True, 0, 1.0, 1.0),
    (0, 30, 12296, True, "channel", True, 8, 1.0, 1.0), (1, 155, 16384, True, "token", False, 0, 1.0, 1.0),
    (0, 9803, 136, True, "channel", True, 8, 1.0, 1.0), (1, 4999, 504, True, "token", True, 0, 1.0, 1.0),
    (0, 2501, 1016, True, "channel", True, 0, 1.0, 0.5), (2, 9777, 72, False, "none", True, 0, 1.0, 1.0),
]
EPS = 1e-5


def norm_inputs(case):
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    rng = np.random.default_rng(tokens + width)
    one = lambda: (1 + 0.1 * torch.from_numpy(rng.normal(0, 1, width))).to(U.DTYPES[dtype]).cuda()  # noqa: E731
    t = dict(x=rows(rng, tokens, width, dtype, pad), y=rows(rng, tokens, width, dtype, pad),
             post=one() if post else None, next=one() if nxt else None,
             gate=None if gate == "none" else one() if gate == "channel" else
             rows(rng, tokens, width, dtype, pad, 0.5))
    return rng, t, width + pad, (width + pad if gate == "token" else 0)


def sizes(t, a, b):
    """fp64 pieces of the definition, and the sizes that enter x' and xhat."""
    v = {k: None if z is None else z.double() for k, z in t.items()}
    r1 = 1.0 if v["post"] is None else 1 / torch.sqrt((v["y"] ** 2).mean(-1, keepdim=True) + EPS)
    z = v["y"] * r1 * (1.0 if v["post"] is None else v["post"])
    g = torch.ones_like(z) if v["gate"] is None else v["gate"]
    new, n = U.residual_norm(v["x"], v["y"], v["post"], v["gate"], v["next"], a, b, EPS)
    big = (a * v["x"]).abs() + (b * g * z).abs()
    r2 = 1 / torch.sqrt((new ** 2).mean(-1, keepdim=True) + EPS)
    return v, r1, z, g, new, n, big, r2


@pytest.mark.parametrize("case", NORMS)
def test_residual_norm(case):
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    _, t, s, gs = norm_inputs(case)
    xo, clean_x = framed(tokens, width, s, dtype)
    no, clean_n = framed(tokens, width, s, dtype)
    L.lbgemm_residual_norm(dtype, tokens, width, t["x"], s, t["y"], s, t["post"], t["gate"], gs, a, b,
                           t["next"], EPS, xo, s, no if nxt else None, s)
    L.lbgemm_device_status()
    v, r1, z, g, new, n, big, r2 = sizes(t, a, b)
    tiny = 2.0 ** -25 if dtype == 1 else 0.0
    assert ((xo.double() - new).abs() <= U.ROUND[dtype] * new.abs() + NORM * big + tiny).all()
    if nxt:
        tol = U.ROUND[dtype] * n.abs() + NORM * (n.abs() + big * r2 * v["next"].abs())
        # the mean of squares of x' moves by 2 mean(|x'| off): within 2^-18 of the sizes' own
        tol = tol + NORM * n.abs() * (big ** 2).mean(-1, keepdim=True) * r2 ** 2 + tiny
        assert ((no.double() - n).abs() <= tol).all()
    else:
        assert (no == 7).all()
    assert clean_x() and clean_n()


def test_residual_norm_alone_and_in_place():
    """No block before: the norm alone, or with the stream scaled; outputs in place."""
    rng = np.random.default_rng(4)
    for dtype in (0, 1, 2):
        x, w = rows(rng, 50, 768, dtype), rows(rng, 1, 768, dtype)[0]
        n = torch.empty_like(x)
        L.lbgemm_residual_norm(dtype, 50, 768, x, 768, None, 0, None, None, 0, 1.0, 1.0, w, EPS, None, 0,
                               n, 768)
        xd = x.double()
        want = xd / torch.sqrt((xd ** 2).mean(-1, keepdim=True) + EPS) * w.double()
        tiny = 2.0 ** -25 if dtype == 1 else 0.0
        assert ((n.double() - want).abs() <= (U.ROUND[dtype] + NORM) * want.abs() + tiny).all()
        y, m, m2, xo = rows(rng, 50, 768, dtype), torch.empty_like(x), None, torch.empty_like(x)
        args = (None, None, 0, 1.0, 0.5, w, EPS)
        L.lbgemm_residual_norm(dtype, 50, 768, x, 768, y, 768, *args, xo, 768, m, 768)
        L.lbgemm_residual_norm(dtype, 50, 768, x, 768, y, 768, *args, x, 768, y, 768)
        assert torch.equal(x, xo) and torch.equal(y, m)
    L.lbgemm_device_status()


def norm_grads(case, t, s, gs, gx, gn, in_place=False):
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    dx, clean_x = framed(tokens, width, s, dtype)
    dy, clean_y = framed(tokens, width, s, dtype)
    dg, clean_g = framed(tokens, width, s, dtype)
    if gate != "token":
        dg = None if gate == "none" else torch.full((width,), 7.0, device="cuda")
    dpost, dnext = (torch.full((width,), 7.0, device="cuda") if w else None for w in (post, nxt))
    if in_place:
        dx, dy = gx, gn
    L.lbgemm_residual_norm_backward(dtype, tokens, width, gx, s, gn, s, t["x"], s, t["y"], s, t["post"],
                                    t["gate"], gs, a, b, t["next"], EPS, dx, s, dy, s, dg, gs, dpost,
                                    dnext)
    L.lbgemm_device_status()
    assert clean_x() and clean_y() and clean_g()
    return dict(x=dx, y=dy, gate=dg, post=dpost, next=dnext)


@pytest.mark.parametrize("case", NORMS)
@pytest.mark.parametrize("stream", [True, False])
def test_residual_norm_backward(case, stream):
    """Against autograd of the definition in 64 bits."""
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    if not stream and not nxt:
        return
    rng, t, s, gs = norm_inputs(case)
    gx = rows(rng, tokens, width, dtype, pad, 0.1) if stream else None
    gn = rows(rng, tokens, width, dtype, pad, 0.1) if nxt else None
    got = norm_grads(case, t, s, gs, gx, gn)
    v, r1, z, g, new, n, big, r2 = sizes(t, a, b)
    leaf = {k: w.clone().requires_grad_() for k, w in v.items() if w is not None}
    new_, n_ = U.residual_norm(*(leaf.get(k) for k in ("x", "y", "post", "gate", "next")), a, b, EPS)
    loss = 0
    if stream:
        loss = loss + (new_ * gx.double()).sum()
    if nxt:
        loss = loss + (n_ * gn.double()).sum()
    want = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
    # sizes: each term of the formulas with everything positive, xhat by what enters it
    d = gx.double().abs() if stream else torch.zeros_like(z)
    if nxt:
        wdn, xh = (v["next"] * gn.double()).abs(), big * r2
        more = 1 + (xh ** 2).mean(-1, keepdim=True)  # (rstd(x') moves with x')
        d = d + r2 * (wdn + xh * (wdn * xh).mean(-1, keepdim=True)) * more
        tol = {"next": (gn.double().abs() * xh * more).sum(0) * NORM}
    else:
        tol = {}
    tol["x"] = NORM * abs(a) * d
    dz = abs(b) * g.abs() * d
    dg = abs(b) * z.abs() * d
    tol["gate"] = NORM * (dg if gate == "token" else dg.sum(0))
    if post:
        yh, wdz = (v["y"] * r1).abs(), v["post"].abs() * dz
        tol["post"] = NORM * (dz * yh).sum(0)
        tol["y"] = NORM * r1 * (wdz + yh * (wdz * yh).mean(-1, keepdim=True))
    else:
        tol["y"] = NORM * dz
    tiny = 2.0 ** -25 if dtype == 1 else 0.0
    for k, w in want.items():
        once = dtype if k in ("x", "y") or (k == "gate" and gate == "token") else 2
        off = (got[k].double() - w).abs()
        assert (off <= U.ROUND[once] * w.abs() + tol[k] + tiny).all(), k


def test_residual_norm_backward_bits_and_place():
    """The same bits twice, and with the results in place of the gradients."""
    case = (0, 333, 1024, True, "channel", True, 0, 1.0, 0.5)
    rng, t, s, gs = norm_inputs(case)
    gx, gn = rows(rng, 333, 1024, 0), rows(rng, 333, 1024, 0)
    one, two = (norm_grads(case, t, s, gs, gx, gn) for _ in range(2))
    three = norm_grads(case, t, s, gs, gx, gn, in_place=True)
    for k in one:
        assert torch.equal(one[k], two[k]) and torch.equal(one[k], three[k]), k


def test_residual_norm_backward_differences():
    """The gradient along random directions against differences of the library's own
    forward pass in fp32.  A step of 2^-6 in unit directions: the third-order term is
    below 2^-12 of the product of sizes, the forward's rounding (2^-22 of 1 over 2^-5)
    below that; 2^-9 of the sizes covers both."""
    case = (2, 9, 256, True, "channel", True, 0, 1.0, 0.75)
    rng, t, s, gs = norm_inputs(case)
    gx, gn = rows(rng, 9, 256, 2), rows(rng, 9, 256, 2)
    got = norm_grads(case, t, s, gs, gx, gn)

    def loss(v):
        xo, no = torch.empty_like(gx), torch.empty_like(gx)
        L.lbgemm_residual_norm(2, 9, 256, v["x"], s, v["y"], s, v["post"], v["gate"], gs, 1.0, 0.75,
                               v["next"], EPS, xo, s, no, s)
        return ((xo.double() * gx.double()).sum() + (no.double() * gn.double()).sum()).item()

    for k in ("x", "y", "post", "gate", "next"):
        way = torch.from_numpy(rng.normal(0, 1, t[k].shape)).float().cuda()
        way = way / way.norm() * t[k].norm() / 8
        h = 2.0 ** -6
        ends = [loss({**t, k: t[k] + e * way}) for e in (h, -h)]
        slope = (ends[0] - ends[1]) / (2 * h)
        assert abs(slope - (got[k].double() * way.double()).sum().item()) <= \
            2.0 ** -9 * (got[k].double().norm() * way.double().norm()).item(), k


def test_no_tokens():
    """Nothing to do: outputs stay; summed gradients are zeros."""
    z = [torch.full((64,), 7.0, device="cuda") for _ in range(3)]
    w = torch.ones(64, device="cuda")
    L.lbgemm_residual_norm_backward(2, 0, 64, None, 0, None, 0, None, 0, w, 64, w, w, 0, 1.0, 1.0, w, EPS,
                                    None, 0, None, 0, z[0], 0, z[1], z[2])
    L.lbgemm_device_status()
    assert all((v == 0).all() for v in z)
