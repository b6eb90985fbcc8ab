"""GPU tests of the feed-forward operators on odd values, the longest rows, and graphs whose
picks change between replays."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
import test_gpu_ffn as F  # noqa: E402
import test_gpu_ffn_exact as X  # noqa: E402
from test_gpu_ffn import _lib  # noqa: E402,F401
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens", [1, 8, 20, 60, 200])
def test_linear_subnormal_tokens(dtype, tokens):
    """Tokens below the smallest normal number of their type count in full."""
    k, n, g = 544, 300, X.gen(tokens)
    unit = 2.0 ** (-24 if dtype else -133)
    x = X.ints(g, (tokens, k), -3, 3).double().mul(unit).to(U.DTYPES[dtype])
    assert (x.double() / unit).abs().max() == 3
    w = X.every_code(g, n, k, 32)
    w.row.fill_(2.0 ** (20 if dtype else 125))
    y = torch.empty((tokens, n), dtype=x.dtype, device="cuda")
    L.lbgemm_w4_linear(dtype, tokens, n, k, 32, x, k, *w.tensors(), y, n)
    L.lbgemm_device_status()
    assert torch.equal(y, (x.double() @ w.dense().T).to(x.dtype))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("tokens", [1, 9, 130, 300])
def test_linear_longest_rows(dtype, tokens):
    """2^20 elements a row: sums below 2^23, exact."""
    k, n, g = 1 << 20, 133, X.gen(tokens)
    w = X.every_code(g, n, k, 128)
    w.scales.fill_(X.ONE)
    x = X.ints(g, (tokens, k), -1, 1).to(U.DTYPES[dtype])
    y = torch.empty((tokens, n), dtype=x.dtype, device="cuda")
    L.lbgemm_w4_linear(dtype, tokens, n, k, 128, x, k, *w.tensors(), y, n)
    L.lbgemm_device_status()
    want = torch.cat([x.double() @ w.dense(slice(a, a + 19)).T for a in range(0, n, 19)], 1)
    assert torch.equal(y, want.to(x.dtype))


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("case", [
    (1, 65536, 32, 2, 2, 32, "any"), (300, 65536, 32, 2, 1, 32, "any"), (2, 32, 65536, 3, 2, 32, "any"),
    (300, 32, 65536, 2, 1, 32, "any"), (16, 16384, 96, 4, 1, 32, "holes")])
def test_moe_long_rows(case, dtype):
    X.test_moe(case, dtype)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_quantize_groups_of_every_size(dtype, group):
    """Groups from the row's largest down to where their scale is subnormal and then 0."""
    rng = np.random.default_rng(group)
    blocks = 24
    w = rng.normal(0, 1, (40, blocks, group)) * 2.0 ** -np.arange(blocks)[None, rng.permutation(blocks), None]
    w = torch.from_numpy(w.reshape(40, -1) * 2.0 ** rng.integers(-6, 6, (40, 1))).to(U.DTYPES[dtype]).cuda()
    k = w.shape[1]
    codes = torch.empty((40, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((40, k // group), dtype=torch.uint8, device="cuda")
    row = torch.empty(40, device="cuda")
    L.lbgemm_w4_quantize(dtype, 40, k, group, w, k, codes, k // 2, scales, k // group, row)
    L.lbgemm_device_status()
    want = U.quantise(w.float().cpu().numpy(), group)
    assert (want[1] == 0).any() and ((want[1] > 0) & (want[1] < 8)).any()
    assert np.array_equal(row.cpu().numpy(), want[2])
    assert np.array_equal(scales.cpu().numpy(), want[1])
    assert np.array_equal(U.unpack(codes.cpu().numpy()), want[0])


@pytest.mark.parametrize("case", [
    (0, 9, 4096, True, "token", True, 0, 1.0, 1.0), (0, 1301, 2048, True, "token", True, 0, 1.0, 0.5),
    (1, 9805, 256, True, "token", True, 0, 1.0, 1.0), (2, 1303, 1040, True, "channel", True, 0, 1.0, 1.0),
    (0, 1701, 4096, True, "channel", True, 0, 1.0, 0.5), (0, 161, 8192, True, "token", True, 0, 1.0, 1.0)])
@pytest.mark.parametrize("what", ["x", "y", "gx", "gn"])
def test_norm_rows_keep_to_themselves(case, what):
    """NaN and infinity in some rows: every other row has the bits that it had."""
    dtype, tokens, width, post, gate, nxt, pad, a, b = case
    rng, t, s, gs = F.norm_inputs(case)
    t["gx"], t["gn"] = (F.rows(rng, tokens, width, dtype) for _ in range(2))

    def run():
        outs = [torch.empty_like(t["x"]) for _ in range(5)]
        sums = [torch.empty(width, device="cuda") for _ in range(3)]
        args = (t["x"], s, t["y"], s, t["post"], t["gate"], gs, a, b, t["next"], F.EPS)
        L.lbgemm_residual_norm(dtype, tokens, width, *args, outs[0], s, outs[1], s)
        L.lbgemm_residual_norm_backward(dtype, tokens, width, t["gx"], s, t["gn"], s, *args, outs[2], s, outs[3], s,
                                        outs[4] if gs else sums[2], gs, sums[0], sums[1])
        L.lbgemm_device_status()
        return outs[:5 if gs else 4]

    want = run()
    odd = torch.tensor([0, 3, tokens // 2, tokens - 1], device="cuda")
    t[what][odd[:2], 5], t[what][odd[2:], width - 1] = float("nan"), float("inf")
    rest = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rest[odd] = False
    for got, before in zip(run(), want):
        assert torch.equal(got[rest], before[rest])


@pytest.mark.parametrize("tokens", [1, 3, 40, 600])
def test_moe_graph_with_other_picks(tokens):
    """A captured call goes by the picks that stand there when it is replayed."""
    rng = np.random.default_rng(tokens)
    hidden, inter, experts, top, group = 256, 128, 12, 3, 32
    x = F.rows(rng, tokens, hidden, 0)
    up, down = (U.Weights(rng, experts * n, k, group).tensors() for n, k in ((2 * inter, hidden), (hidden, inter)))
    held, weights = (torch.from_numpy(v).cuda() for v in F.picks(rng, tokens, experts, top, "none"))
    y, want = (torch.empty((tokens, hidden), dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def call(ids, share, out, stream=None):
        L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, top, group, x, hidden, ids, share, *up, *down, out,
                        hidden, stream)

    call(held, weights, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(held, weights, y, torch.cuda.current_stream().cuda_stream)
    for kind in ("all", "one", "holes", "none", "twice", "all"):
        ids, share = (torch.from_numpy(v).cuda() for v in F.picks(rng, tokens, experts, top, kind))
        held.copy_(ids)
        weights.copy_(share)
        y.fill_(7)
        graph.replay()
        call(ids, share, want)
        L.lbgemm_device_status()
        assert torch.equal(y, want), kind
        assert kind != "none" or (y == 0).all()
