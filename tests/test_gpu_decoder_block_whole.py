"""GPU tests of a decoder block's step against the definition of a block, norm by norm
and stream by stream.

Bounds as in test_gpu_ffn.py: an output is rounded once, the norms' fp32 arithmetic is off by
2^-18 of the sizes that enter.  The stream after attention is rounded to bf16 before the second
half reads it, so what leaves the block carries that rounding too."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_ffn as F  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import decoder_block as blocks  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

MODEL, EPS, R = 256, 1e-6, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


class Kept:
    """A half of a block that keeps what it was given and what it gave."""

    def __init__(self, half):
        self.half, self.hidden = half, getattr(half, "hidden", None)

    def step(self, x, *rest):
        self.given = x.clone()
        self.gave = self.half.step(x, *rest)
        return self.gave


def norm(v, w):
    """fp64 norm, and what fp32 arithmetic and one rounding may be off by."""
    y = v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS) * w.double()
    return y, (R + F.NORM) * y.abs()


def joined(x, y, w, a, b):
    """a x + b (norm of y, or y), and the sizes that enter."""
    z = y if w is None else norm(y, w)[0]
    return a * x + b * z, (a * x).abs() + (b * z).abs()


@pytest.mark.parametrize("some", [(True, True), (True, False), (False, True), (False, False)])
@pytest.mark.parametrize("rows,pad", [([1, 1, 1], 0), ([37, 0, 91], 8)])
def test_block_is_its_definition(some, rows, pad):
    """Every norm with its own weights, the second and last given or not."""
    block = blocks.random_block(4, 2, 64, MODEL, 128, 8, 64, 2, 32, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    norms = [(1 + 0.3 * torch.randn(MODEL, generator=g, device="cuda")).bfloat16() for _ in range(4)]
    norms[1], norms[3] = (w if there else None for w, there in zip((norms[1], norms[3]), some))
    a, b = 0.875, -0.625
    attention, experts = Kept(block.attention), Kept(block.experts)
    made = blocks.DecoderBlock(attention, experts, norms, a, b, EPS)
    caches = [blocks.PagedCache(3, 128, 2, 64, 16) for _ in range(2)]
    wide = torch.randn((sum(rows), MODEL + pad), generator=g, device="cuda").bfloat16()
    x = wide[:, :MODEL]
    out = made.step(x, caches[0], caches[0].extend(rows))
    L.lbgemm_device_status()
    assert out.shape == x.shape and out.is_contiguous()

    xd = x.double()
    n, tol = norm(xd, norms[0])
    assert ((attention.given.double() - n).abs() <= tol).all()
    y = block.attention.step(attention.given, caches[1], caches[1].extend(rows))
    assert torch.equal(attention.gave, y)

    x1, big = joined(xd, y.double(), norms[1], a, b)
    off = F.NORM * big  # of x1 before its rounding
    n1, tol = norm(x1, norms[2])
    r = 1 / torch.sqrt((x1 * x1).mean(-1, keepdim=True) + EPS)
    tol = tol + F.NORM * (big * r * norms[2].double().abs() +
                          n1.abs() * (big ** 2).mean(-1, keepdim=True) * r ** 2)
    assert ((experts.given.double() - n1).abs() <= tol).all()
    y = block.experts.step(experts.given)
    assert torch.equal(experts.gave, y)

    x2, big = joined(x1, y.double(), norms[3], a, b)
    tol = R * x2.abs() + F.NORM * big + abs(a) * (R * x1.abs() + off) * (1 + R)
    assert ((out.double() - x2).abs() <= tol).all()


def test_rows_of_a_wider_buffer():
    """The bits of the same rows side by side, for the block and for its experts."""
    block = blocks.random_block(4, 2, 64, MODEL, 64, 8, 64, 2, 32)
    wide = torch.randn((90, MODEL + 40), device="cuda").bfloat16()
    x = wide[:, 8:MODEL + 8]
    caches = [blocks.PagedCache(2, 64, 2, 64, 16) for _ in range(2)]
    one, two = (block.step(v, c, c.extend([40, 50])) for v, c in zip((x, x.contiguous()), caches))
    assert torch.equal(one, two)
    assert torch.equal(block.experts.step(x), block.experts.step(x.contiguous()))
    w = torch.randn((6, 96), device="cuda")[:, 16:80]
    one, two = (blocks.Weights4(6, 64, 32).store(v).tensors() for v in (w, w.contiguous()))
    assert all(torch.equal(p, q) for p, q in zip(one, two))
    L.lbgemm_device_status()
