"""GPU tests of the norms around a block in every shape (warps and vectors of a row, rows at
once) of every type that test_gpu_ffn.py does not meet; the checks are that file's."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_ffn as F  # noqa: E402
from test_gpu_ffn import _lib  # noqa: E402,F401

# dtype, tokens, width, post, gate, next, pad, a, b; token counts are odd, so that where rows go two
# at once the last pair holds one
CASES = [
    # 8 warps, two rows: widths 1032 to 2048
    (0, 1301, 2048, True, "channel", True, 0, 1.0, 0.5), (0, 1403, 1040, True, "token", True, 8, 1.0, 1.0),
    (1, 1501, 1032, True, "token", True, 0, 1.0, -0.5), (1, 1303, 2040, False, "channel", True, 0, 0.5, 1.0),
    (2, 1303, 1040, True, "channel", True, 4, 1.0, 1.0), (2, 1401, 1304, True, "token", True, 0, 1.0, 1.0),
    (0, 1777, 1536, True, "none", True, 0, 1.0, 1.0),
    # two rows of one to four warps and of sixteen
    (1, 9805, 256, True, "token", True, 0, 1.0, 1.0), (1, 10001, 104, True, "channel", True, 8, 1.0, 0.5),
    (0, 5001, 400, True, "token", True, 0, 1.0, 1.0), (2, 4999, 264, True, "channel", True, 4, 1.0, 1.0),
    (1, 2503, 1024, True, "channel", True, 0, 1.0, 1.0), (2, 2501, 520, False, "token", True, 0, 1.0, -1.0),
    (2, 1305, 2056, True, "none", True, 0, 1.0, 1.0), (2, 1305, 2560, True, "channel", True, 0, 1.0, 0.5),
    # a row at once: few rows, or wide ones
    (1, 33, 504, True, "channel", True, 8, 1.0, 1.0), (0, 37, 600, True, "token", True, 0, 1.0, 1.0),
    (2, 41, 264, True, "channel", True, 0, 1.0, 1.0), (1, 45, 1200, True, "token", True, 0, 0.5, 1.0),
    (2, 47, 2000, True, "channel", True, 4, 1.0, 1.0), (1, 51, 3000, True, "channel", True, 0, 1.0, 1.0),
    (1, 311, 7000, True, "token", True, 8, 1.0, 0.25), (1, 29, 8192, True, "none", True, 0, 1.0, 1.0),
]


@pytest.mark.parametrize("case", CASES)
def test_residual_norm(case):
    F.test_residual_norm(case)


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("stream", [True, False])
def test_residual_norm_backward(case, stream):
    F.test_residual_norm_backward(case, stream)
