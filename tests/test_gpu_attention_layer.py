"""GPU tests of the attention layer that runs the operators together, and of
rotations by a multiple of 8 channels that is none of 16."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_attention as A  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import attention_layer as layers  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


ODD_ROTATIONS = [
    (L.BF16, 70, 5, 3, 128, 24, False, (1, 1), 8),
    (L.F32, 37, 3, 1, 64, 8, False, (1, 1), 0),
    (L.F16, 33, 9, 2, 64, 40, True, (1, 0), 8),
    (L.F32, 21, 2, 1, 256, 200, False, (1, 1), 4),
]


@pytest.mark.parametrize("case", ODD_ROTATIONS)
def test_norm_rope_odd_rotations(case):
    A.test_norm_rope(case)
    A.test_norm_rope_backward_formula(case)


def test_norm_rope_runs_across_tokens():
    """More rows than one pass of the blocks: runs that begin and end inside a
    token, on both sides."""
    case = (L.BF16, 6001, 7, 3, 64, 64, False, (1, 1), 8)
    A.test_norm_rope(case)
    A.test_norm_rope_backward_formula(case)


def read_back(cache, rows):
    """Keys and values of the first rows[b] tokens of every sequence."""
    slots = np.concatenate([
        cache.table[b, np.arange(n) // cache.page_size].astype(np.int64) * cache.page_size +
        np.arange(n) % cache.page_size for b, n in enumerate(rows)])
    k, v = (torch.empty((len(slots), cache.heads, cache.dim), dtype=torch.float32, device="cuda")
            for _ in range(2))
    width = cache.heads * cache.dim
    L.lbgemm_kv4_read(L.F32, len(slots), cache.heads, cache.dim, torch.from_numpy(slots).cuda(),
                      cache.buffer, cache.pages, cache.page_size, k, width, v, width)
    return k, v


@pytest.mark.parametrize("window", [0, 9])
def test_layer_in_pieces(window):
    """A prompt at once, and the same tokens in pieces: the same cache; outputs
    within what the rounding of the attention's result to bf16 and then to 8 bits
    can change: a code of each input of the output projection by one, and by the
    share that its row's scale moves (2^-7 of 127 codes, one more)."""
    model, total = 256, [37, 21, 50]
    layer = layers.random_layer(8, 2, 64, model, 64, 64, window=window)
    g = torch.Generator(device="cuda").manual_seed(3)
    xs = [torch.randn((n, model), generator=g, device="cuda").bfloat16() for n in total]

    whole = layers.PagedCache(3, 64, 2, 64, 16)
    y = layer.step(torch.cat(xs), whole, whole.extend(total)).float()

    pieces = layers.PagedCache(3, 64, 2, 64, 16)
    outs, at = [[] for _ in total], [0] * 3
    for rows in ([30, 1, 20], [0, 15, 29], [7, 4, 0], [0, 1, 1]):
        x = torch.cat([x[a:a + n] for x, a, n in zip(xs, at, rows)])
        part = layer.step(x, pieces, pieces.extend(rows)).float()
        for b, z in enumerate(part.split(rows)):
            outs[b].append(z)
            at[b] += rows[b]
    L.lbgemm_device_status()
    assert at == total
    for a, b in zip(read_back(whole, total), read_back(pieces, total)):
        assert torch.equal(a, b)
    z = torch.cat([torch.cat(o) for o in outs])
    assert torch.isfinite(y).all()
    # |o| is at most the largest cached value; a code is 1 / 127 of a row's largest
    code = read_back(whole, total)[1].abs().max() / 127
    tol = layer.out.float().abs().sum(1) * layer.out_scale * 2 * code + 2.0 ** -7 * y.abs()
    assert ((y - z).abs() <= tol).all()
    # and on the whole much closer than the bound for every single one
    assert (y - z).norm() <= 0.02 * y.norm()


def test_layer_graph_step():
    """A captured step gives what the calls give."""
    layer = layers.random_layer(4, 4, 128, 512, 40, 32, interleaved=True)
    x = torch.randn((2, 512), device="cuda").bfloat16()
    caches = [layers.PagedCache(2, 40, 4, 128, 16) for _ in range(2)]
    prompt = torch.randn((30, 512), device="cuda").bfloat16()
    for c in caches:
        layer.step(prompt, c, c.extend([13, 17]))
    want = layer.step(x, caches[0], caches[0].extend([1, 1]))
    new = caches[1].extend([1, 1])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(x, caches[1], dict(new, max_kv=40))
    graph.replay()
    L.lbgemm_device_status()
    assert torch.equal(got, want)


def test_cache_refuses():
    cache = layers.PagedCache(1, 20, 2, 64, 16)
    cache.extend([32])
    with pytest.raises(ValueError):
        cache.extend([1])
    with pytest.raises(ValueError):
        layers.PagedCache(1, 20, 2, 96, 16)


def test_example_runs(capsys):
    assert layers.main(["--batch", "3", "--prompt", "70", "--steps", "5", "--heads", "8",
                        "--kv-heads", "2", "--dim", "64", "--model", "512", "--page", "16"]) == 0
    out = capsys.readouterr().out
    assert "step 4, 3 tokens over 76" in out and "nan" not in out
