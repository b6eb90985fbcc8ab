"""Limits of the attention operators' sizes: refused on the host, before any
device is touched.  No GPU needed."""
import os
import re
import subprocess

import pytest

from bit_tensor_gemm_gb300 import build as bld
from bit_tensor_gemm_gb300 import lbgemm as L
from test_attention_host import attend, refused


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bld.build()
    L.load()


@pytest.mark.parametrize("batch,max_q,hq", [
    (65535, (1 << 17) + 8, 64),   # 32770 tiles of 256 rows a sequence
    (65535, (1 << 20) + 64, 8),
    (40000, 1 << 21, 16),
])
def test_too_many_tiles(batch, max_q, hq):
    """Tiles of rows are counted in 32 bits by the kernels: 2^31 and more overflowed
    the count."""
    assert batch * -(-max_q * hq // 256) >= 1 << 31
    refused(L.ERR_INVALID_ARG, attend, batch=batch, total=max_q, max_q=max_q, hq=hq, hk=1,
            qs=hq * 128)
    assert b"tiles" in L.load().lbgemm_last_error()


def test_registers_of_the_many_row_kernel(tmp_path):
    """Its warps share out 128 registers a thread after the launch, and would wait
    for ever for what a launch with fewer does not have: the compiler gives every
    form of it 128, and the launch checks that."""
    src = os.path.join(bld.CSRC, "kv4_tiles.cu")
    r = subprocess.run([bld.nvcc(), *bld.ARCH, *bld.CFLAGS, "-Xptxas", "-v", "-c", src, "-o",
                        str(tmp_path / "t.o")], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    kernels = re.findall(r"entry function .*kv4_tiles_kernel(?:.*\n)+?.*Used (\d+) registers", r.stderr)
    assert kernels == ["128"] * 4, r.stderr
    with open(src) as f:
        code = f.read()
    assert re.search(r"numRegs < kLaunchRegs\) return cudaError", code)
    # the split is in the constants that the launch and the static check use
    assert len(re.findall(r"setmaxnreg", code)) == 2 and not re.search(r"setmaxnreg[^%]*u32 \d", code)
