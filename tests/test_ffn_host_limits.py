"""Feed-forward operators at the limits of their arguments, on the host.  No GPU needed."""
import os
import re

import pytest

torch = pytest.importorskip("torch")

from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402
from test_ffn_host import ALIGN, BAD, P, _lib, back, moe, norm, refused  # noqa: E402,F401


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


# ---- no tokens ------------------------------------------------------------------------------


@pytest.mark.parametrize("gate", [P, None])
@pytest.mark.parametrize("post", [P, None])
def test_norm_of_no_tokens_takes_no_rows(post, gate):
    """Tensors without elements have no address: weights may be given all the same."""
    norm(tokens=0, X=None, Y=None, post=post, gate=gate, Xo=None, No=None)
    rows = dict(dXo=None, dN=None, X=None, Y=None, dX=None, dY=None)
    if post or gate or torch.cuda.is_available():
        if torch.cuda.is_available():
            pytest.skip("addresses that nothing may write")
        with pytest.raises(L.LbgemmError) as e:  # (their gradients are zeros, which takes a device)
            back(tokens=0, post=post, gate=gate, dpost=post, dgate=gate, **rows)
        assert e.value.status not in (BAD, ALIGN)
    else:
        back(tokens=0, post=None, gate=None, nxt=None, dpost=None, dgate=None, dnext=None, **rows)
    # a token needs its rows
    refused(BAD, norm, Y=None, post=P, gate=None)
    refused(BAD, back, Y=None, post=P, gate=None, dgate=None, dY=None)


# ---- what a dependent launch may take for constant ---------------------------------------


def kernels(name):
    """(name, parameters, body) of a source file's kernels."""
    with open(os.path.join(bld.CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    for m in re.finditer(r"__global__ void (?:__launch_bounds__\([^{;]*?\)\s*)?(\w+)\(([^{;]*)\)\s*\{", text):
        end = text.find("\n}", m.end())
        yield m.group(1), m.group(2), text[m.end():end]


# What is older than the whole chain of launches of a call: its own inputs.
INPUTS = {"x", "weights", "scales", "row_scales", "scale_ptr"}


@pytest.mark.parametrize("name", ["w4_tiles.cu", "w4_rows.cu"])
def test_dependents_take_inputs_only_for_constant(name):
    """A kernel that waits for the launch before it may stand on the GPU while that launch
    writes: only inputs of the call are __restrict__ or loaded by __ldg in it."""
    waiting = 0
    for kernel, parameters, body in kernels(name):
        if "griddepcontrol.wait" not in body:
            continue
        waiting += 1
        for p in re.findall(r"__restrict__\s+(\w+)", parameters):
            assert p in INPUTS, f"{kernel}: {p}"
        for p in re.findall(r"__ldg\(\s*([\w.]+)", body):
            assert p.split(".")[-1] in INPUTS, f"{kernel}: {p}"
    assert waiting == {"w4_tiles.cu": 5, "w4_rows.cu": 1}[name]


@pytest.mark.parametrize("name,kernel,written", [
    ("simt.cu", "skinny_s8_kernel", {"A", "sx"}), ("stream_mma.cu", "stream_mma_kernel", {"X", "sx"}),
    ("hmma_skinny.cu", "hmma_skinny_kernel", {"X", "sx"}),
    ("simt.cu", "cvt_s8_f16_flat_kernel", {"a", "b"}), ("simt.cu", "cvt_s8_f16_kernel", {"src"})])
def test_quantised_activations_are_not_constant(name, kernel, written):
    """What the activations' quantiser may still be writing when the 8-bit kernel behind it
    starts: neither __restrict__ nor loaded by __ldg there."""
    found = [(p, body) for k, p, body in kernels(name) if k == kernel]
    assert len(found) == 1
    parameters, body = found[0]
    assert not written & set(re.findall(r"__restrict__\s+(\w+)", parameters))
    loads = re.findall(r"__ldg\((?:reinterpret_cast<[^>]*>\()?\s*(\w+)", body)
    assert not written & set(loads)
