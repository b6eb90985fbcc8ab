"""GPU tests of the feed-forward operators at the limits of their ranges and rules."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import ffn_util as U  # noqa: E402
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
