"""GPU test of the attention layer on a stream of its own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from bit_tensor_gemm_gb300 import attention_layer as layers  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


@pytest.mark.parametrize("handle", [False, True])
def test_step_on_another_stream(handle):
    """While a step waits on its stream, the current stream gets memory of the sizes
    that the step has let go of, and writes to it: nothing of the step is in there."""
    layer = layers.random_layer(8, 2, 64, 512, 64, 64)
    x = torch.randn((3 * 40, 512), device="cuda").bfloat16()
    caches = [layers.PagedCache(3, 64, 2, 64, 16) for _ in range(2)]
    want = layer.step(x, caches[0], caches[0].extend([40] * 3))
    new = caches[1].extend([40] * 3)
    side = torch.cuda.Stream()
    torch.full((8,), float("nan"), dtype=torch.bfloat16, device="cuda")  # (loads its kernel)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)  # (cycles: some 100 ms)
    got = layer.step(x, caches[1], new, side.cuda_stream if handle else side)
    waits = not side.query()
    for _ in range(4):  # the joint projection's and the attention's sizes
        junk = [torch.full((3 * 40, n), float("nan"), dtype=torch.bfloat16, device="cuda")
                for n in (12 * 64, 8 * 64, 512)]
    torch.cuda.current_stream().synchronize()
    assert waits and not side.query()  # (or the memory was not in use yet)
    side.synchronize()
    del junk
    L.lbgemm_device_status()
    assert torch.equal(got, want)
