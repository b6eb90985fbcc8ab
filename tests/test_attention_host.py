"""Argument checks of the attention operators: refused on the host, before any
device is touched.  No GPU needed."""
import math

import pytest

from bit_tensor_gemm_gb300 import build as bld
from bit_tensor_gemm_gb300 import lbgemm as L

P = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bld.build()
    L.load()


def refused(status, call, **change):
    with pytest.raises(L.LbgemmError) as e:
        call(**change)
    assert e.value.status == status, str(e.value)
    assert L.lbgemm_last_error()


def rope(dtype=L.BF16, tokens=4, hq=2, hk=1, dim=128, Q=P, qs=256, K=P, ks=128, wq=P, wk=P,
         eps=1e-6, cos=P, sin=P, rows=16, pos=P, rot=128, inter=False, Qo=P, qos=256, Ko=P, kos=128):
    L.lbgemm_qk_norm_rope(dtype, tokens, hq, hk, dim, Q, qs, K, ks, wq, wk, eps, cos, sin, rows,
                          pos, rot, inter, Qo, qos, Ko, kos, 0)


ROPE_BAD = [
    (dict(dtype=3), L.ERR_INVALID_ARG), (dict(dtype=-1), L.ERR_INVALID_ARG),
    (dict(tokens=-1), L.ERR_INVALID_ARG), (dict(hq=-1), L.ERR_INVALID_ARG),
    (dict(hq=0, hk=0), L.ERR_INVALID_ARG), (dict(dim=0), L.ERR_INVALID_ARG),
    (dict(dim=12), L.ERR_INVALID_ARG), (dict(dim=520), L.ERR_INVALID_ARG),
    (dict(rot=130), L.ERR_INVALID_ARG), (dict(rot=3), L.ERR_INVALID_ARG),
    (dict(rot=-2), L.ERR_INVALID_ARG), (dict(eps=-1.0), L.ERR_INVALID_ARG),
    (dict(eps=math.nan), L.ERR_INVALID_ARG), (dict(Q=None), L.ERR_INVALID_ARG),
    (dict(Ko=None), L.ERR_INVALID_ARG), (dict(qs=248), L.ERR_INVALID_ARG),
    (dict(qs=260), L.ERR_ALIGNMENT), (dict(K=P + 8), L.ERR_ALIGNMENT),
    (dict(wq=P + 4), L.ERR_ALIGNMENT), (dict(cos=None), L.ERR_INVALID_ARG),
    (dict(pos=None), L.ERR_INVALID_ARG), (dict(rows=0), L.ERR_INVALID_ARG),
    (dict(sin=P + 4), L.ERR_ALIGNMENT), (dict(pos=P + 4), L.ERR_ALIGNMENT),
]


@pytest.mark.parametrize("change,status", ROPE_BAD)
def test_norm_rope_refusals(change, status):
    refused(status, rope, **change)


def rope_back(dwq=P, dwk=P, wq=P, wk=P, dQ=P, dQo=P, Q=P, dtype=L.F32, dqs=256):
    L.lbgemm_qk_norm_rope_backward(dtype, 4, 2, 1, 128, dQo, 256, P, 128, Q, 256, P, 128, wq, wk,
                                   1e-6, P, P, 16, P, 128, False, dQ, dqs, P, 128, dwq, dwk, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dwq=None), L.ERR_INVALID_ARG), (dict(wk=None), L.ERR_INVALID_ARG),
    (dict(dwk=P + 4), L.ERR_ALIGNMENT), (dict(dQ=None), L.ERR_INVALID_ARG),
    (dict(dQo=None), L.ERR_INVALID_ARG), (dict(Q=None), L.ERR_INVALID_ARG),
    (dict(dtype=7), L.ERR_INVALID_ARG), (dict(dqs=100), L.ERR_INVALID_ARG),
])
def test_norm_rope_backward_refusals(change, status):
    refused(status, rope_back, **change)


def write(dtype=L.BF16, tokens=4, heads=2, dim=128, K=P, ks=256, V=P, vs=256, slots=P, cache=P,
          pages=4, page=16):
    L.lbgemm_kv4_write(dtype, tokens, heads, dim, K, ks, V, vs, slots, cache, pages, page, 0)


def read(dtype=L.BF16, tokens=4, heads=2, dim=128, K=P, ks=256, V=P, vs=256, slots=P, cache=P,
         pages=4, page=16):
    L.lbgemm_kv4_read(dtype, tokens, heads, dim, slots, cache, pages, page, K, ks, V, vs, 0)


@pytest.mark.parametrize("call", [write, read])
@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), L.ERR_INVALID_ARG), (dict(tokens=-1), L.ERR_INVALID_ARG),
    (dict(heads=0), L.ERR_INVALID_ARG), (dict(dim=96), L.ERR_INVALID_ARG),
    (dict(page=24), L.ERR_INVALID_ARG), (dict(page=0), L.ERR_INVALID_ARG),
    (dict(pages=0), L.ERR_INVALID_ARG), (dict(K=None), L.ERR_INVALID_ARG),
    (dict(V=P + 2), L.ERR_ALIGNMENT), (dict(vs=252), L.ERR_INVALID_ARG),
    (dict(ks=258), L.ERR_ALIGNMENT), (dict(slots=None), L.ERR_INVALID_ARG),
    (dict(slots=P + 4), L.ERR_ALIGNMENT), (dict(cache=None), L.ERR_INVALID_ARG),
    (dict(cache=P + 8), L.ERR_ALIGNMENT),
])
def test_cache_refusals(call, change, status):
    refused(status, call, **change)


def attend(dtype=L.BF16, batch=2, total=6, max_q=4, hq=8, hk=2, dim=128, Q=P, qs=1024, cu=P, cache=P,
           pages=8, page=16, table=P, width=4, lens=P, max_kv=64, scale=0.1, causal=True, window=0,
           O=P, lse=P):
    L.lbgemm_kv4_attention(dtype, batch, total, max_q, hq, hk, dim, Q, qs, cu, cache, pages, page,
                           table, width, lens, max_kv, scale, causal, window, O, lse, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=L.F32), L.ERR_INVALID_ARG), (dict(batch=-1), L.ERR_INVALID_ARG),
    (dict(batch=0), L.ERR_INVALID_ARG), (dict(max_q=0), L.ERR_INVALID_ARG),
    (dict(max_q=7), L.ERR_INVALID_ARG), (dict(hq=7), L.ERR_INVALID_ARG),
    (dict(hq=0), L.ERR_INVALID_ARG), (dict(dim=80), L.ERR_INVALID_ARG),
    (dict(page=8), L.ERR_INVALID_ARG), (dict(max_kv=65), L.ERR_INVALID_ARG),
    (dict(max_kv=-1), L.ERR_INVALID_ARG), (dict(window=-1), L.ERR_INVALID_ARG),
    (dict(window=8, causal=False), L.ERR_INVALID_ARG), (dict(scale=math.inf), L.ERR_INVALID_ARG),
    (dict(Q=None), L.ERR_INVALID_ARG), (dict(qs=1000), L.ERR_INVALID_ARG),
    (dict(qs=1028), L.ERR_ALIGNMENT), (dict(cu=None), L.ERR_INVALID_ARG),
    (dict(lens=None), L.ERR_INVALID_ARG), (dict(table=None), L.ERR_INVALID_ARG),
    (dict(O=None), L.ERR_INVALID_ARG), (dict(O=P + 8), L.ERR_ALIGNMENT),
    (dict(lse=P + 2), L.ERR_ALIGNMENT), (dict(cu=P + 2), L.ERR_ALIGNMENT),
    (dict(cache=None), L.ERR_INVALID_ARG),
])
def test_attention_refusals(change, status):
    refused(status, attend, **change)


def test_nothing_to_do_needs_no_device():
    rope(tokens=0, Q=None, K=None, Qo=None, Ko=None)
    write(tokens=0, K=None, V=None, slots=None)
    read(tokens=0, K=None, V=None, slots=None)
    attend(batch=0, total=0, max_q=0, Q=None, O=None, cu=None)


def test_page_bytes():
    assert L.lbgemm_kv4_page_bytes(8, 128, 64) == 8 * 64 * 132
    assert L.lbgemm_kv4_page_bytes(1, 64, 16) == 16 * 68
    for bad in ((0, 128, 64), (8, 96, 64), (8, 128, 40), (8, 128, 0), (70000, 64, 16)):
        assert L.lbgemm_kv4_page_bytes(*bad) == 0
