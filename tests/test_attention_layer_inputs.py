"""What the attention layer refuses before a call: the library sees addresses, not what a
tensor is.  No GPU needed."""
import pytest

torch = pytest.importorskip("torch")

from bit_tensor_gemm_gb300 import attention_layer as layers  # noqa: E402


class Stop(Exception):
    """Raised where a call would have been made."""


@pytest.fixture(autouse=True)
def no_calls(monkeypatch):
    def call(*args):
        raise Stop
    monkeypatch.setattr(layers.L, "lbgemm_linear_quant", call)


def layer(qkv=(512, 96), out=(96, 256)):  # 4 heads and 2 of 64 on 96 channels
    qkv, out = (torch.zeros(s, dtype=torch.int8) for s in (qkv, out))
    return layers.AttentionLayer(4, 2, 64, qkv, torch.ones(len(qkv)), out, torch.ones(len(out)), None, None,
                                 torch.ones(8, 32), torch.zeros(8, 32))


X = torch.zeros((5, 96), dtype=torch.bfloat16)


@pytest.mark.parametrize("x", [
    X.float(), X.half(), X[:, :64], X.T.contiguous().T, X[0], X[None], X.to("meta"),
    torch.zeros((5, 128), dtype=torch.bfloat16)[:, :96], torch.zeros((5, 128), dtype=torch.bfloat16)])
def test_step_refuses(x):
    with pytest.raises(ValueError):
        layer().step(x, None, None)


def test_step_takes():
    for x in (X, X[2:3], X[:0]):
        with pytest.raises(Stop):
            layer().step(x, None, None)


@pytest.mark.parametrize("change", [dict(qkv=(448, 96)), dict(out=(96, 512)), dict(out=(64, 256)),
                                    dict(qkv=(512, 128))])
def test_layer_refuses_weights(change):
    with pytest.raises(ValueError):
        layer(**change)
