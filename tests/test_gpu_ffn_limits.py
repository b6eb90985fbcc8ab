"""GPU tests of the feed-forward operators at the limits of their ranges and rules."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
import test_gpu_ffn as F  # noqa: E402
import test_gpu_ffn_exact as X  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import decoder_block as blocks  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


# ---- silu(gate) * up over the range of its factors -------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens", [1, 40, 300])
def test_moe_gates_of_every_size(dtype, tokens):
    """Gates far below 0 with an up that makes an ordinary number of it, one channel each:
    gate, up and the second product are exact, so what is left is silu's own error (an
    exponential of |gate| / 2, squared: up to 2^-16 at the far end) and the rounding."""
    gate = np.array([-170, -130, -104, -103, -100, -95, -92, -90, -89.5, -89, -88.75, -88.5, -88.25, -88, -87.75,
                     -87.5, -87.25, -87, -80, -40, -17, -5, -1, -0.125, 0, 0.25, 1, 9, 30, 88, 89, 1000], np.float32)
    silu = gate.astype(np.float64) / (1 + np.exp(-gate.astype(np.float64)))
    up = np.minimum(1.375 / np.maximum(np.abs(silu), 1e-60), 3e38).astype(np.float32)
    size, eye = 32, np.eye(32, dtype=np.int64)
    ups, down = (U.Weights(np.random.default_rng(1), n, size, 32) for n in (2 * size, size))
    ups.codes[:], ups.scales[:], down.codes[:], down.scales[:], down.row[:] = 0, 0x38, eye, 0x38, 1
    ups.codes[:, 0] = 1
    ups.row[::2], ups.row[1::2] = gate, up
    x = torch.zeros((tokens, size), dtype=U.DTYPES[dtype], device="cuda")
    x[:, 0] = 1
    ids = torch.zeros((tokens, 1), dtype=torch.int32, device="cuda")
    y = torch.empty_like(x)
    L.lbgemm_moe_w4(dtype, tokens, size, size, 1, 1, 32, x, size, ids, torch.ones((tokens, 1), device="cuda"),
                    *ups.tensors(), *down.tensors(), y, size)
    L.lbgemm_device_status()
    want = silu * up.astype(np.float64)
    tol = (U.ROUND[dtype] + 2.0 ** -16) * np.abs(want) + (2.0 ** -25 if dtype else 0)
    off = np.abs(y.double().cpu().numpy() - want)
    assert (off <= tol).all(), [(g, u) for g, u, bad in zip(gate, up, (off > tol).any(0)) if bad]


# ---- few tokens on long rows ------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", [
    # up to 9728 rows of more than 8192 elements go to tiles, more of them stream by rows while the
    # tokens fit shared memory: both sides of each edge
    (1, 9728, 8224, 32), (1, 9729, 8224, 32), (4, 9729, 8192, 64), (4, 9800, 12320, 32), (8, 9800, 8320, 128),
    (1, 11008, 28672, 128), (1, 10001, 49152, 128), (1, 10001, 65536, 64), (2, 20011, 16384, 32),
])
def test_linear_long_rows(case, dtype):
    X.test_linear(case, dtype)


# ---- no tokens --------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("gate", [None, "channel", "token"])
def test_norm_of_no_tokens(dtype, gate):
    """Tensors without elements, weights as ever: summed gradients are zeros."""
    t = U.DTYPES[dtype]
    none, w = torch.empty((0, 96), dtype=t, device="cuda"), torch.ones(96, dtype=t, device="cuda")
    g, stride = {None: (None, 0), "channel": (w, 0), "token": (none, 96)}[gate]
    args = (none, 96, none, 96, w, g, stride, 1.0, 0.5, w, 1e-6)
    L.lbgemm_residual_norm(dtype, 0, 96, *args, none, 96, none, 96)
    sums = [torch.full((96,), 7.0, device="cuda") for _ in range(3)]
    dgate = {None: None, "channel": sums[2], "token": none}[gate]
    L.lbgemm_residual_norm_backward(dtype, 0, 96, none, 96, none, 96, *args, none, 96, none, 96, dgate, stride,
                                    sums[0], sums[1])
    L.lbgemm_device_status()
    assert (sums[0] == 0).all() and (sums[1] == 0).all()
    assert (sums[2] == (0 if gate == "channel" else 7)).all()


def test_block_of_no_tokens():
    block = blocks.random_block(4, 2, 64, 256, 64, 8, 64, 2, 32)
    cache = blocks.PagedCache(2, 64, 2, 64, 16)
    x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    assert block.step(x, cache, cache.extend([0, 0])).shape == (0, 256)
    assert block.experts.step(x).shape == (0, 256)
    L.lbgemm_device_status()


# ---- many experts, many picks, offsets beyond 32 bits ------------------------------------------


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", [
    (60, 32, 32, 1024, 8, 32, "any"), (700, 64, 32, 1024, 4, 32, "holes"), (1000, 32, 64, 1023, 8, 32, "any"),
    (40000, 32, 64, 16, 8, 32, "any"),  # 320000 picks: 64 pieces of the sort
])
def test_moe_many_experts_or_picks(case, dtype):
    X.test_moe(case, dtype)


def test_moe_beyond_32_bits():
    """2^20 picks of 2304 channels: places beyond 2^31 elements of what is gathered and joined."""
    tokens, hidden, inter, experts, top, group = 131072, 2304, 32, 4, 8, 32
    g = X.gen(7)
    x = X.ints(g, (tokens, hidden), -1, 1).bfloat16()
    x[:, 0] = 1
    up, down = X.every_code(g, experts * 2 * inter, hidden, group), X.every_code(g, experts * hidden, inter, group)
    up.codes.view(-1, 2, hidden // 2)[:, 0] = 0  # gates: 32 from the first channel (two codes a byte, bits 0 ..)
    up.codes.view(-1, 2, hidden // 2)[:, 0, 0] = 4
    up.scales.view(-1, 2, hidden // group)[:, 0] = X.EIGHT
    up.codes.view(-1, 2, hidden // 2)[:, 1, 16:] = 0  # up: 32 channels, so that its sums are exact in bf16
    up.scales.view(-1, 2, hidden // group)[:, 1] = X.ONE
    up.row[:] = 1
    up.codes.view(-1, 2, hidden // 2)[:, 1] &= 0x11  # codes 0 and 1
    ids = X.ints(g, (tokens, top), 0, experts - 1).to(torch.int32)
    share = X.powers(g, tokens * top, -3, -1).view(tokens, top)
    y = torch.full((tokens, hidden), 7.0, dtype=torch.bfloat16, device="cuda")
    L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, top, group, x, hidden, ids, share, *up.tensors(),
                    *down.tensors(), y, hidden)
    L.lbgemm_device_status()
    some = torch.cat([torch.arange(40), torch.arange(tokens - 40, tokens), torch.randperm(tokens)[:400]]).cuda()
    both = (x[some].double() @ up.dense().T).view(len(some), experts, inter, 2)
    assert (both[..., 0] == 32).all() and both[..., 1].abs().max() <= 32
    every = torch.einsum("tei,ehi->teh", 32 * both[..., 1], down.dense().view(experts, hidden, inter))
    picked = every.gather(1, ids[some].long()[..., None].expand(-1, -1, hidden))
    want = (picked * share[some].double()[..., None]).sum(1)
    assert torch.equal(y[some], want.bfloat16())


@pytest.mark.parametrize("tokens,n", [(8, 290_000_001), (40_000, 60_000), (90, 24_000_001)])
def test_linear_outputs_beyond_32_bits(tokens, n):
    k, g = 32, X.gen(tokens)
    w = X.Weights.__new__(X.Weights)
    w.group, w.row = 32, torch.ones(n, device="cuda")
    w.codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g, device="cuda")
    w.scales = torch.full((n, 1), X.ONE, dtype=torch.uint8, device="cuda")
    x = X.ints(g, (tokens, k), -1, 1).bfloat16()
    y = torch.empty((tokens, n), dtype=torch.bfloat16, device="cuda")
    L.lbgemm_w4_linear(0, tokens, n, k, 32, x, k, *w.tensors(), y, n)
    L.lbgemm_device_status()
    for a in sorted({0, n // 3, (1 << 27) % n, n - 4096}):
        dense = w.dense(slice(a, a + 4096))
        for rows in (slice(0, 64), slice(max(0, tokens // 2 - 32), tokens // 2 + 32), slice(max(0, tokens - 64), tokens)):
            assert torch.equal(y[rows, a:a + 4096], (x[rows].double() @ dense.T).bfloat16())


def test_route_beyond_32_bits():
    tokens, experts, top = 2_200_003, 1024, 4
    logits = torch.empty((tokens, experts), dtype=torch.bfloat16, device="cuda").normal_(generator=X.gen(1))
    ids = torch.empty((tokens, top), dtype=torch.int32, device="cuda")
    weights = torch.empty((tokens, top), device="cuda")
    L.lbgemm_moe_route(0, tokens, experts, top, logits, experts, True, ids, weights)
    L.lbgemm_device_status()
    some = torch.cat([torch.arange(3), torch.arange(2097150, 2097155), torch.arange(tokens - 5, tokens)]).cuda()
    want_ids, want = U.route(logits[some].double().cpu().numpy(), top, True)
    assert np.array_equal(ids[some].cpu().numpy(), want_ids)
    assert (np.abs(weights[some].double().cpu().numpy() - want) <= 2.0 ** -18 * want).all()


def test_norm_beyond_32_bits():
    """2^31 elements and more, both directions.  An output is off by its rounding and by 2^-18 of
    the sizes that enter, a handful of a row's largest: 2^-14 of that covers them."""
    tokens, width, eps = 300_001, 8192, 1e-6
    g = X.gen(3)
    x, y, dx, dn = (torch.empty((tokens, width), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
                    for _ in range(4))
    post, nxt = ((1 + 0.1 * torch.randn(width, generator=g, device="cuda")).bfloat16() for _ in range(2))
    outs = [torch.empty_like(x) for _ in range(4)]
    sums = [torch.empty(width, device="cuda") for _ in range(2)]
    args = (x, width, y, width, post, None, 0, 1.0, 0.5, nxt, eps)
    L.lbgemm_residual_norm(0, tokens, width, *args, outs[0], width, outs[1], width)
    L.lbgemm_residual_norm_backward(0, tokens, width, dx, width, dn, width, *args, outs[2], width, outs[3], width,
                                    None, 0, *sums)
    L.lbgemm_device_status()
    some = torch.cat([torch.arange(3), torch.arange(262140, 262150), torch.arange(tokens - 5, tokens)]).cuda()
    leaf = [t[some].double().requires_grad_() for t in (x, y)]
    new, n = U.residual_norm(*leaf, post.double(), None, nxt.double(), 1.0, 0.5, eps)
    grads = torch.autograd.grad((new * dx[some].double()).sum() + (n * dn[some].double()).sum(), leaf)
    for got, want in zip(outs, [new.detach(), n.detach(), *grads]):
        top = want.abs().amax(1, keepdim=True)
        assert ((got[some].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -14 * top).all()


# ---- outputs in place of inputs ------------------------------------------------------------------


@pytest.mark.parametrize("case", [
    (0, 1301, 2048, True, "token", True, 0, 1.0, 0.5), (1, 9805, 256, True, "token", True, 0, 1.0, 1.0),
    (0, 1700, 4096, True, "token", True, 0, 1.0, 0.5), (0, 311, 5120, True, "token", True, 8, 1.0, 1.0),
    (2, 29, 8192, True, "token", True, 0, 1.0, 1.0), (0, 160, 16384, True, "token", True, 0, 1.0, 1.0),
    (2, 1021, 1000, True, "token", True, 4, 0.5, 1.0), (0, 33, 136, False, "token", True, 8, 1.0, 1.0)])
def test_norm_in_place(case):
    """Any output on any row-by-row input, the bits of outputs of their own."""
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    rng, t, s, gs = F.norm_inputs(case)
    gx, gn = (F.rows(rng, tokens, width, dtype, pad) for _ in range(2))

    def forward(v, xo, no):
        L.lbgemm_residual_norm(dtype, tokens, width, v["x"], s, v["y"], s, v["post"], v["gate"], gs, a, b,
                               v["next"], F.EPS, xo, s, no, s)
        return xo, no

    def backward(v, dx, dy, dg):
        sums = [torch.empty(width, device="cuda") if v[k] is not None else None for k in ("post", "next")]
        L.lbgemm_residual_norm_backward(dtype, tokens, width, v["gx"], s, v["gn"], s, v["x"], s, v["y"], s,
                                        v["post"], v["gate"], gs, a, b, v["next"], F.EPS, dx, s, dy, s, dg, gs,
                                        *sums)
        return [dx, dy, dg] + [z for z in sums if z is not None]

    def fresh():  # the same numbers with the same strides
        v = {}
        for k, z in dict(t, gx=gx, gn=gn).items():
            if z is not None and z.dim() == 2:
                buf = torch.zeros((tokens, s), dtype=z.dtype, device="cuda")
                buf[:, :width] = z
                v[k] = buf[:, :width]
            else:
                v[k] = z
        return v

    def out():
        return torch.zeros((tokens, s), dtype=U.DTYPES[dtype], device="cuda")[:, :width]

    want = forward(fresh(), out(), out())
    for k, j in (("x", "y"), ("y", "x"), ("gate", "y"), ("x", "gate")):
        v = fresh()
        assert all(torch.equal(p, q) for p, q in zip(forward(v, v[k], v[j]), want)), (k, j)
    want = backward(fresh(), out(), out(), out())
    for k, j, i in (("gx", "gn", "gate"), ("x", "y", "gate"), ("gate", "x", "y"), ("gn", "gate", "gx")):
        v = fresh()
        assert all(torch.equal(p, q) for p, q in zip(backward(v, v[k], v[j], v[i]), want)), (k, j, i)
    L.lbgemm_device_status()
