"""Argument checks of the feed-forward operators: refused on the host, before any
device is touched; and the tests' own statement of the 4-bit layout.  No GPU needed."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import ffn_util as U  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

P = 4096  # an aligned address that nothing reads
BAD, ALIGN = L.ERR_INVALID_ARG, L.ERR_ALIGNMENT


@pytest.fixture(scope="module", autouse=True)
def _lib():
    bld.build()
    L.load()


def refused(status, call, **change):
    with pytest.raises(L.LbgemmError) as e:
        call(**change)
    assert e.value.status == status, str(e.value)
    assert L.lbgemm_last_error()


def quantize(dtype=L.BF16, N=4, K=256, group=64, W=P, ws=256, codes=P, cs=128, scales=P, ss=4,
             rows=P, rs=1):
    L.lbgemm_w4_quantize(dtype, N, K, group, W, ws, codes, cs, scales, ss, rows, rs, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), BAD), (dict(N=-1), BAD), (dict(K=0), BAD), (dict(K=96), BAD),
    (dict(group=16), BAD), (dict(group=96, K=192), BAD), (dict(K=(1 << 20) + 64), BAD),
    (dict(W=None), BAD), (dict(ws=248), BAD), (dict(ws=260), ALIGN), (dict(W=P + 8), ALIGN),
    (dict(codes=None), BAD), (dict(cs=112), BAD), (dict(cs=136), ALIGN), (dict(scales=None), BAD),
    (dict(ss=3), BAD), (dict(rows=None), BAD), (dict(rows=P + 2), ALIGN), (dict(rs=0), BAD),
])
def test_quantize_refusals(change, status):
    refused(status, quantize, **change)


def linear(dtype=L.BF16, M=4, N=6, K=256, group=64, X=P, xs=256, codes=P, scales=P, rows=P, Y=P,
           ys=6):
    L.lbgemm_w4_linear(dtype, M, N, K, group, X, xs, codes, scales, rows, Y, ys, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=L.F32), BAD), (dict(dtype=-1), BAD), (dict(M=-1), BAD), (dict(N=-1), BAD),
    (dict(M=(1 << 30) + 1), BAD), (dict(K=0), BAD), (dict(K=100), BAD), (dict(group=48), BAD),
    (dict(X=None), BAD), (dict(xs=128), BAD), (dict(xs=260), ALIGN), (dict(X=P + 2), ALIGN),
    (dict(codes=None), BAD), (dict(codes=P + 8), ALIGN), (dict(scales=None), BAD),
    (dict(scales=P + 4), ALIGN), (dict(rows=None), BAD), (dict(rows=P + 4), ALIGN),
    (dict(Y=None), BAD), (dict(Y=P + 8), ALIGN), (dict(ys=5), BAD),
])
def test_linear_refusals(change, status):
    refused(status, linear, **change)


def route(dtype=L.F32, tokens=4, experts=8, top=2, logits=P, stride=8, ids=P, weights=P):
    L.lbgemm_moe_route(dtype, tokens, experts, top, logits, stride, True, ids, weights, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=5), BAD), (dict(tokens=-1), BAD), (dict(experts=0), BAD), (dict(experts=1025), BAD),
    (dict(top=0), BAD), (dict(top=9), BAD), (dict(top=33, experts=64, stride=64), BAD),
    (dict(logits=None), BAD), (dict(stride=7), BAD), (dict(logits=P + 2), ALIGN),
    (dict(ids=None), BAD), (dict(ids=P + 2), ALIGN), (dict(weights=None), BAD),
    (dict(weights=P + 1), ALIGN),
])
def test_route_refusals(change, status):
    refused(status, route, **change)


def moe(dtype=L.BF16, tokens=4, hidden=128, inter=64, experts=8, top=2, group=64, X=P, xs=128, ids=P,
        weights=P, uc=P, us=P, ur=P, dc=P, ds=P, dr=P, Y=P, ys=128):
    L.lbgemm_moe_w4(dtype, tokens, hidden, inter, experts, top, group, X, xs, ids, weights, uc, us,
                    ur, dc, ds, dr, Y, ys, 0)


@pytest.mark.parametrize("change,status", [
    (dict(dtype=L.F32), BAD), (dict(tokens=-1), BAD), (dict(tokens=1 << 24), BAD),
    (dict(hidden=96), BAD), (dict(inter=32), BAD), (dict(group=8), BAD), (dict(experts=0), BAD),
    (dict(experts=2000), BAD), (dict(top=0), BAD), (dict(top=33), BAD),
    (dict(inter=1 << 20, experts=1024), BAD), (dict(X=None), BAD), (dict(xs=120), BAD),
    (dict(xs=132), ALIGN), (dict(ids=None), BAD), (dict(ids=P + 2), ALIGN),
    (dict(weights=None), BAD), (dict(uc=None), BAD), (dict(us=None), BAD), (dict(ur=P + 4), ALIGN),
    (dict(dc=P + 8), ALIGN), (dict(dr=None), BAD), (dict(Y=None), BAD), (dict(ys=64), BAD),
    (dict(Y=P + 2), ALIGN),
])
def test_moe_refusals(change, status):
    refused(status, moe, **change)


def norm(dtype=L.BF16, tokens=4, width=64, X=P, xs=64, Y=P, ys=64, post=P, gate=P, gs=0, a=1.0, b=1.0,
         nxt=P, eps=1e-6, Xo=P, xos=64, No=P, nos=64):
    L.lbgemm_residual_norm(dtype, tokens, width, X, xs, Y, ys, post, gate, gs, a, b, nxt, eps, Xo,
                           xos, No, nos, 0)


SHARED = [
    (dict(dtype=3), BAD), (dict(tokens=-1), BAD), (dict(width=0), BAD), (dict(width=60), BAD),
    (dict(width=16392, xs=16392, ys=16392), BAD), (dict(dtype=L.F32, width=8200), BAD),
    (dict(X=None), BAD), (dict(xs=56), BAD), (dict(xs=68), ALIGN), (dict(Y=None), BAD),
    (dict(Y=P + 8), ALIGN), (dict(post=P + 2), ALIGN), (dict(gate=P + 2), ALIGN),
    (dict(gs=32), BAD), (dict(gs=-64), BAD), (dict(gs=68), ALIGN), (dict(a=math.inf), BAD),
    (dict(b=math.nan), BAD), (dict(eps=-1.0), BAD), (dict(eps=math.nan), BAD),
    (dict(nxt=P + 4), ALIGN),
]


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(nxt=None), BAD), (dict(No=None), BAD), (dict(Xo=None), BAD), (dict(xos=32), BAD),
    (dict(No=P + 2), ALIGN), (dict(Y=None, post=None, gate=None, Xo=None, nxt=None, No=None), BAD),
])
def test_norm_refusals(change, status):
    refused(status, norm, **change)


def back(dtype=L.BF16, tokens=4, width=64, dXo=P, dxos=64, dN=P, dns=64, X=P, xs=64, Y=P, ys=64,
         post=P, gate=P, gs=0, a=1.0, b=1.0, nxt=P, eps=1e-6, dX=P, dxs=64, dY=P, dys=64, dgate=P,
         dgs=0, dpost=P, dnext=P):
    L.lbgemm_residual_norm_backward(dtype, tokens, width, dXo, dxos, dN, dns, X, xs, Y, ys, post,
                                    gate, gs, a, b, nxt, eps, dX, dxs, dY, dys, dgate, dgs, dpost,
                                    dnext, 0)


@pytest.mark.parametrize("change,status", SHARED + [
    (dict(dN=None), BAD), (dict(dXo=None, dN=None, nxt=None, dnext=None), BAD),
    (dict(dXo=P + 2), ALIGN), (dict(dX=None), BAD), (dict(dY=None), BAD), (dict(dxs=60), BAD),
    (dict(dgate=None), BAD), (dict(gate=None), BAD), (dict(dgate=P + 4), ALIGN),
    (dict(gs=64, dgs=0), BAD), (dict(gs=64, dgs=72), None), (dict(dpost=None), BAD),
    (dict(dnext=None), BAD), (dict(dnext=P + 8), ALIGN), (dict(post=None), BAD),
])
def test_norm_backward_refusals(change, status):
    if status is None:  # taken: without a device this is what is left to fail
        if torch.cuda.is_available():
            pytest.skip("addresses that nothing may read")
        with pytest.raises(L.LbgemmError) as e:
            back(**change)
        assert e.value.status not in (BAD, ALIGN)
        return
    refused(status, back, **change)


def test_nothing_to_do_needs_no_device():
    quantize(N=0, W=None, codes=None, scales=None, rows=None)
    linear(M=0, X=None, Y=None, codes=None)
    linear(N=0, X=None, Y=None, codes=None)
    route(tokens=0, logits=None, ids=None, weights=None)
    moe(tokens=0, X=None, Y=None, ids=None, weights=None)
    norm(tokens=0, X=None, Y=P, Xo=None, No=None)


# ---- the tests' own statement of the layout ------------------------------------------


def test_layout_by_hand():
    """Elements 0 .. 7 = 1 2 3 4 5 6 7 -8: the even ones in the low half-word."""
    codes = np.zeros((1, 32), np.int64)
    codes[0, :8] = [1, 2, 3, 4, 5, 6, 7, -8]
    assert U.pack(codes)[0, :4].tolist() == [0x31, 0x75, 0x42, 0x86]
    rng = np.random.default_rng(1)
    codes = rng.integers(-8, 8, (5, 64))
    assert (U.unpack(U.pack(codes)) == codes).all()


def test_e4m3_by_hand():
    got = U.e4m3(np.array([0x00, 0x01, 0x08, 0x38, 0x39, 0x7e, 0xb8], np.uint8))
    assert got.tolist() == [0.0, 2.0 ** -9, 2.0 ** -6, 1.0, 1.125, 448.0, -1.0]
    x = np.array([0.0, 2.0 ** -10, 3 * 2.0 ** -10, 1.0, 1.0625, 1.1875, 448.0, 460.0, 9999.0])
    assert U.to_e4m3(x).tolist() == [0, 0, 2, 0x38, 0x38, 0x3a, 0x7e, 0x7e, 0x7e]
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mine = U.e4m3(np.arange(256, dtype=np.uint8))
    assert np.array_equal(mine, every, equal_nan=True)


def test_quantise_reads_back():
    """A weight comes back within half a step, the largest of a group within what
    the scale's own rounding (2^-4) leaves above 7 steps."""
    rng = np.random.default_rng(2)
    w = rng.normal(0, 1, (7, 256)).astype(np.float32)
    codes, scales, row = U.quantise(w, 64)
    step = np.repeat(U.e4m3(scales) * row[:, None].astype(np.float64), 64, 1)
    assert np.abs(codes).max() == 7
    assert (np.abs(w - codes * step) <= 0.5 * step * (1 + 1e-6)).all()
