"""Feed-forward operators at the limits of their arguments, on the host.  No GPU needed."""
import pytest

torch = pytest.importorskip("torch")

from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402
from test_ffn_host import BAD, _lib, moe, refused  # noqa: E402,F401


@pytest.mark.parametrize("tokens,top", [
    ((1 << 24) + 1, 1), ((1 << 19) + 1, 32), (1 << 59, 32), (1 << 60, 16), ((1 << 62) + 1, 4),
    ((1 << 63) - 1, 32), ((1 << 63) - 1, 2)])
def test_moe_refuses_too_many_picks(tokens, top):
    """Also where tokens * top_k does not fit 64 bits."""
    refused(BAD, moe, tokens=tokens, top=top, experts=64)


def test_moe_takes_the_most_picks():
    """2^24 picks pass the checks: without a device this is what is left to fail."""
    if torch.cuda.is_available():
        pytest.skip("addresses that nothing may read")
    for tokens, top in ((1 << 24, 1), (1 << 19, 32)):
        with pytest.raises(L.LbgemmError) as e:
            moe(tokens=tokens, top=top, experts=64)
        assert e.value.status != BAD
