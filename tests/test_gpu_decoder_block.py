"""GPU tests of the feed-forward operators as they are used together: a block, graphs,
streams, threads, weights beyond 2^31 bytes."""
import threading

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
import test_gpu_ffn as F  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import decoder_block as blocks  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


def dense(w):
    """Weights4 in fp64."""
    codes = torch.from_numpy(U.unpack(w.codes.cpu().numpy()).astype(np.float64)).cuda()
    scales = torch.from_numpy(U.e4m3(w.scales.cpu().numpy())).cuda()
    return codes * scales.repeat_interleave(w.group, 1) * w.row_scales.double()[:, None]


@pytest.mark.parametrize("tokens", [1, 11, 130])
def test_experts_together(tokens):
    """Router's product, router and experts, against the definitions of each on what
    the call before it gave; gate and up end where moe expects them."""
    g = torch.Generator(device="cuda").manual_seed(tokens)
    hidden, inter, experts, top = 256, 96, 8, 3
    gate, up, down, router = (torch.randn(s, generator=g, device="cuda") * 0.06 for s in (
        (experts, inter, hidden), (experts, inter, hidden), (experts, hidden, inter), (experts, hidden)))
    layer = blocks.Experts(router, gate, up, down, top, 32)
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    y = layer.step(x)
    L.lbgemm_device_status()
    # quantised within half a step of a scale of 2^-4 at most
    both = dense(layer.up).view(experts, inter, 2, hidden)
    for got, want in ((both[:, :, 0], gate), (both[:, :, 1], up), (dense(layer.down).view_as(down), down)):
        blocks_of = want.double().abs().view(*want.shape[:-1], -1, 32).amax(-1)
        step = (blocks_of / 7 * (1 + 2.0 ** -4)).repeat_interleave(32, -1)
        assert ((got - want.double()).abs() <= 0.5 * step * (1 + 2.0 ** -3)).all()
    logits = (x.double() @ dense(layer.router).T)
    mine = torch.empty((tokens, experts), dtype=torch.bfloat16, device="cuda")
    L.lbgemm_w4_linear(0, tokens, experts, hidden, 32, x, hidden, *layer.router.tensors(), mine, experts)
    assert ((mine.double() - logits).abs() <= 2.0 ** -8 * logits.abs() + F.SUM(hidden) * (
        x.double().abs() @ dense(layer.router).abs().T)).all()
    ids, weights = (torch.from_numpy(a).cuda() for a in U.route(mine.double().cpu().numpy(), top, True))

    class W:
        def __init__(self, w):
            self.codes, self.w = w.codes, w

        def dense(self):
            return dense(self.w)
    want, tol = F.experts_want(x, ids, weights, W(layer.up), W(layer.down), hidden, inter, 0)
    # (the router's weights are off by 2^-20 of themselves at most)
    assert ((y.double() - want).abs() <= tol + 2.0 ** -20 * want.abs() + 2.0 ** -20 * tol.max()).all()


def test_block_graph():
    """A block's step in a graph gives what its calls give, every time it is replayed."""
    model = 256
    block = blocks.random_block(4, 2, 64, model, 64, 8, 64, 2, 32)
    g = torch.Generator(device="cuda").manual_seed(2)
    caches = [blocks.PagedCache(3, 64, 2, 64, 16) for _ in range(2)]
    x = torch.randn((3 * 20, model), generator=g, device="cuda").bfloat16()
    for c in caches:
        y = block.step(x, c, c.extend([20] * 3))
        assert torch.isfinite(y).all()
    x1 = torch.randn((3, model), generator=g, device="cuda").bfloat16()
    want = block.step(x1, caches[0], caches[0].extend([1] * 3))
    new = caches[1].extend([1] * 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = block.step(x1, caches[1], dict(new, max_kv=64))
    for _ in range(2):
        graph.replay()
        L.lbgemm_device_status()
        assert torch.equal(got, want)


def test_example_runs(capsys):
    assert blocks.main(["--batch", "3", "--prompt", "60", "--steps", "4", "--heads", "4", "--kv-heads",
                        "2", "--dim", "64", "--model", "256", "--experts", "6", "--inter", "128",
                        "--top", "2"]) == 0
    out = capsys.readouterr().out
    assert "step 3, 3 tokens over 65" in out and "nan" not in out


def test_weights4_refuses():
    w = blocks.Weights4(6, 64, 32)
    for shape, first, step in (((7, 64), 0, 1), ((3, 96), 0, 1), ((4, 64), 0, 2), ((2, 64), -1, 1)):
        with pytest.raises(ValueError):
            w.store(torch.zeros(shape, device="cuda"), first, step)


# ---- graphs, streams, threads ---------------------------------------------------------------


def calls(seed, tokens):
    """One call of each kind that takes scratch, on inputs of its own: (run, outputs)."""
    rng = np.random.default_rng(seed)
    k, n, hidden, inter, experts, top = 640, 200, 256, 96, 5, 2
    x, w = F.rows(rng, tokens, k, 0), U.Weights(rng, n, k, 64).tensors()
    h = F.rows(rng, tokens, hidden, 0)
    up, down = (U.Weights(rng, experts * a, b, 32).tensors() for a, b in ((2 * inter, hidden), (hidden, inter)))
    ids, weights = (torch.from_numpy(a).cuda() for a in F.picks(rng, tokens, experts, top, "all"))
    one = torch.ones(hidden, dtype=torch.bfloat16, device="cuda")
    outs = [torch.zeros((tokens, n), dtype=torch.bfloat16, device="cuda"),
            torch.zeros((tokens, hidden), dtype=torch.bfloat16, device="cuda")]
    outs += [torch.zeros_like(h) for _ in range(2)] + [torch.zeros(hidden, device="cuda") for _ in range(3)]

    def run(stream=None):
        L.lbgemm_w4_linear(0, tokens, n, k, 64, x, k, *w, outs[0], n, stream)
        L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, top, 32, h, hidden, ids, weights, *up, *down,
                        outs[1], hidden, stream)
        L.lbgemm_residual_norm_backward(0, tokens, hidden, h, hidden, h, hidden, h, hidden, outs[1],
                                        hidden, one, one, 0, 1.0, 1.0, one, 1e-6, outs[2], hidden,
                                        outs[3], hidden, outs[4], 0, outs[5], outs[6], stream)
    return run, outs, (x, h)


@pytest.mark.parametrize("tokens", [2, 40, 330])
def test_graphs_share_nothing(tokens):
    """Two graphs of different calls, replayed in turn and with new inputs, give what
    the calls give."""
    torch.cuda.synchronize()
    made = [calls(s, tokens) for s in (1, 2)]
    want = []
    for run, outs, _ in made:
        run()
        want.append([o.clone() for o in outs])
    graphs = []
    for run, outs, _ in made:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run()
        graphs.append(graph)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for _, outs, _ in made:
            for o in outs:
                o.zero_()
        for i in order:
            graphs[i].replay()
        L.lbgemm_device_status()
        for i in set(order):
            assert all(torch.equal(a, b) for a, b in zip(made[i][1], want[i]))
    for x in made[0][2]:  # new inputs, half the size
        x.mul_(0.5)
    graphs[0].replay()
    got = [o.clone() for o in made[0][1]]
    made[0][0]()
    L.lbgemm_device_status()
    assert all(torch.equal(a, b) for a, b in zip(got, made[0][1]))


def test_layers_cut_along_k_at_once():
    """Layers of a few tiles, whose parts of k lie in scratch: on two streams at the same
    time and from two graphs in turn, the bits of a call alone."""
    made, want = [], []
    for seed, tokens, k in ((1, 1, 11008), (2, 12, 8192), (3, 45, 4096), (4, 100, 6144)):
        rng = np.random.default_rng(seed)
        x, w = F.rows(rng, tokens, k, 0), U.Weights(rng, 300, k, 128).tensors()
        y = torch.zeros((tokens, 304), dtype=torch.bfloat16, device="cuda")
        made.append((lambda stream=None, a=(tokens, k, x, w, y): L.lbgemm_w4_linear(
            0, a[0], 300, a[1], 128, a[2], a[1], *a[3], a[4], 304, stream), y))
        made[-1][0]()
        want.append(y.clone())

    def check():
        L.lbgemm_device_status()
        for (_, y), z in zip(made, want):
            assert torch.equal(y, z)
            y.zero_()
        torch.cuda.synchronize()

    check()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for i, (run, _) in enumerate(made):
            run(streams[i % 2].cuda_stream)
    torch.cuda.synchronize()
    check()
    graphs = []
    for half in (made[:2], made[2:]):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for run, _ in half:
                run(torch.cuda.current_stream().cuda_stream)
    for order in ((0, 1), (1, 0, 1)):
        for i in order:
            graphs[i].replay()
        made[0][0]()
        check()


def test_streams_and_threads():
    """Calls of several sizes from two threads on two streams, sharing the scratch."""
    sizes = [3, 40, 330, 17]
    made = [[calls(10 * t + i, n) for i, n in enumerate(sizes)] for t in range(2)]
    want = []
    for per in made:
        for run, outs, _ in per:
            run()
        L.lbgemm_device_status()
        want.append([[o.clone() for o in outs] for _, outs, _ in per])
        for _, outs, _ in per:
            for o in outs:
                o.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    errors = []

    def work(t):
        try:
            for _ in range(5):
                for run, _, _ in made[t]:
                    run(streams[t].cuda_stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(t,)) for t in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    L.lbgemm_device_status()
    assert not errors
    for per, good in zip(made, want):
        for (_, outs, _), w in zip(per, good):
            assert all(torch.equal(a, b) for a, b in zip(outs, w))


@pytest.mark.parametrize("tokens", [1, 12, 40, 300])
def test_linear_beyond_32_bits(tokens):
    """Codes of 2.3 GB: the last rows lie beyond 2^31 bytes, and beyond 2^32 weights."""
    n, k, group = 70001, 65536, 128
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.full((n, k // group), 0x38, dtype=torch.uint8, device="cuda")  # 1
    row = torch.ones(n, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    some = torch.tensor([0, 1, 32768, 65535, 65536, 69999, n - 1], device="cuda")
    codes[some] = torch.randint(0, 256, (len(some), k // 2), dtype=torch.uint8, generator=g, device="cuda")
    row[some] = 2.0 ** -8
    x = torch.randn((tokens, k), generator=g, device="cuda").bfloat16()
    y = torch.empty((tokens, n), dtype=torch.bfloat16, device="cuda")
    L.lbgemm_w4_linear(0, tokens, n, k, group, x, k, codes, scales, row, y, n)
    L.lbgemm_device_status()
    w = torch.from_numpy(U.unpack(codes[some].cpu().numpy()).astype(np.float64)).cuda() * 2.0 ** -8
    want = x.double() @ w.T
    tol = 2.0 ** -8 * want.abs() + F.SUM(k) * (x.double().abs() @ w.abs().T)
    assert ((y[:, some].double() - want).abs() <= tol).all()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[some] = False
    assert (y[:, rest] == 0).all()


@pytest.mark.parametrize("tokens", [2, 120])
def test_moe_beyond_32_bits(tokens):
    """Experts of 2.6 GB of codes, the last of them chosen."""
    hidden, inter, experts, group = 4096, 2048, 320, 128
    up, down = (torch.zeros((experts * n, k // 2), dtype=torch.uint8, device="cuda")
                for n, k in ((2 * inter, hidden), (hidden, inter)))
    us, ds = (torch.full((w.shape[0], 2 * w.shape[1] // group), 0x38, dtype=torch.uint8, device="cuda")
              for w in (up, down))
    ur, dr = (torch.full((w.shape[0],), 2.0 ** -7, device="cuda") for w in (up, down))
    g = torch.Generator(device="cuda").manual_seed(4)
    last = experts - 1
    for w, n in ((up, 2 * inter), (down, hidden)):
        w[last * n:] = torch.randint(0, 256, (n, w.shape[1]), dtype=torch.uint8, generator=g, device="cuda")
    x = torch.randn((tokens, hidden), generator=g, device="cuda").bfloat16()
    ids = torch.full((tokens, 2), last, dtype=torch.int32, device="cuda")
    ids[:, 0] = 0  # all zeros
    weights = torch.full((tokens, 2), 0.5, device="cuda")
    y = torch.empty_like(x)
    L.lbgemm_moe_w4(0, tokens, hidden, inter, experts, 2, group, x, hidden, ids, weights, up, us, ur, down,
                    ds, dr, y, hidden)
    L.lbgemm_device_status()

    class One:  # the last expert alone
        def __init__(self, w, n):
            self.w, self.codes = w[last * n:], np.zeros((n, 1))

        def dense(self):
            return torch.from_numpy(U.unpack(self.w.cpu().numpy()).astype(np.float64)).cuda() * 2.0 ** -7
    want, tol = F.experts_want(x, ids - last, weights, One(up, 2 * inter), One(down, hidden), hidden, inter, 0)
    assert ((y.double() - want).abs() <= tol).all()
