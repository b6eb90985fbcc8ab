"""What the decoder block refuses before a call: the library sees addresses and strides,
not what a tensor is.  No GPU needed."""
import pytest

torch = pytest.importorskip("torch")

from bit_tensor_gemm_gb300 import decoder_block as blocks  # noqa: E402


class Stop(Exception):
    """Raised where a call would have been made."""


@pytest.fixture(autouse=True)
def no_calls(monkeypatch):
    def call(*args):
        raise Stop
    for name in ("lbgemm_w4_quantize", "lbgemm_w4_linear", "lbgemm_residual_norm"):
        monkeypatch.setattr(blocks.L, name, call)


W = torch.zeros((4, 64))


@pytest.mark.parametrize("w", [
    torch.zeros((64, 4)).T,               # channels 4 apart
    torch.zeros((4, 128))[:, ::2], W[:, :32], W[0], W[None], W.double(), W.to(torch.int8), W.to("meta"),
])
def test_store_refuses(w):
    with pytest.raises(ValueError):
        blocks.Weights4(6, 64, 32, "cpu").store(w)


@pytest.mark.parametrize("w", [W, W.bfloat16(), W.half(), torch.zeros((4, 80))[:, :64]])
def test_store_takes(w):
    with pytest.raises(Stop):
        blocks.Weights4(6, 64, 32, "cpu").store(w)


class Experts(blocks.Experts):
    """3 experts of 32 channels, 2 each, on 64, with weights that nobody wrote."""

    def __init__(self):
        self.experts, self.inter, self.hidden, self.top_k, self.group = 3, 32, 64, 2, 32
        self.router = blocks.Weights4(3, 64, 32, "cpu")
        self.up, self.down = blocks.Weights4(3 * 64, 64, 32, "cpu"), blocks.Weights4(3 * 64, 32, 32, "cpu")


@pytest.mark.parametrize("change", [
    dict(up=(3, 16, 64)), dict(up=(2, 32, 64)), dict(down=(3, 32, 64)), dict(down=(3, 64, 16)),
    dict(router=(4, 64)), dict(router=(3, 32))])
def test_experts_refuse_shapes(change):
    shapes = dict(dict(router=(3, 64), gate=(3, 32, 64), up=(3, 32, 64), down=(3, 64, 32)), **change)
    with pytest.raises(ValueError):
        blocks.Experts(*(torch.zeros(shapes[k]) for k in ("router", "gate", "up", "down")), 2, 32)


X = torch.zeros((5, 64), dtype=torch.bfloat16)
BAD_X = [X.float(), X.double(), X[:, :32], X.T.contiguous().T, X[0], X[None], X.to("meta")]


@pytest.mark.parametrize("x", BAD_X)
def test_experts_refuse_tokens(x):
    with pytest.raises(ValueError):
        Experts().step(x)


NORM = torch.zeros(64, dtype=torch.bfloat16)


@pytest.mark.parametrize("x", BAD_X + [X.half()])
def test_block_refuses_tokens(x):
    with pytest.raises(ValueError):
        blocks.DecoderBlock(None, Experts(), [NORM] * 4).step(x, None, None)


@pytest.mark.parametrize("norms", [
    [NORM] * 3, [None, NORM, NORM, NORM], [NORM, NORM, None, NORM], [NORM.float()] * 4,
    [NORM, NORM[:32], NORM, NORM], [NORM, NORM, NORM, torch.zeros(128, dtype=torch.bfloat16)[::2]]])
def test_block_refuses_norms(norms):
    with pytest.raises(ValueError):
        blocks.DecoderBlock(None, Experts(), norms)


@pytest.mark.parametrize("x", [X, torch.zeros((5, 96), dtype=torch.bfloat16)[:, 8:72]])
def test_rows_of_a_wider_buffer_are_taken(x):
    for norms in ([NORM] * 4, [NORM, None, NORM, None]):
        with pytest.raises(Stop):
            blocks.DecoderBlock(None, Experts(), norms).step(x, None, None)
    for y in (x, x.half()):
        with pytest.raises(Stop):
            Experts().step(y)
