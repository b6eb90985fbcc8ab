"""GPU tests of the attention operators (norm with rotation, the 4-bit paged
cache, attention over it) against their definitions in 64 bits.

Tolerances, fixed from the arithmetic:
  norm and rotation   one rounding to the output type (half an ulp of |y|) plus
                      fp32 steps: 32 * 2^-24 of the rotated pair's magnitude
                      (rsqrt 2 ulp, the sum of up to 512 squares, products);
  weight gradients    fp32 sums: 2^-18 of sum |g xhat| (any order of up to a
                      few thousand terms a lane stays far inside);
  cache               exact, bytes and values;
  attention           with p rounded to 11 significant bits for the value
                      product and scores held in fp32 around a bias of up to
                      136 code units: dt = 2^-20 * 136 * scale * ks * sum|q|,
                      o within half an ulp + (2^-11 + 2 dt) * sum p |v|,
                      lse within dt + 2^-20 * (1 + |lse|).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_util as U  # noqa: E402
from bit_tensor_gemm_gb300 import build as bld  # noqa: E402
from bit_tensor_gemm_gb300 import lbgemm as L  # noqa: E402

BF16, F16, F32 = L.BF16, L.F16, L.F32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bld.build()
    L.load()


def rand(seed, shape, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(U.DTYPES[dtype]).cuda()


def strided(x, extra):
    """x [tokens, heads, dim] as a view of wider rows."""
    t, h, d = x.shape
    wide = torch.full((t, h * d + extra), float("nan"), dtype=x.dtype, device=x.device)
    wide[:, :h * d] = x.reshape(t, -1)
    return wide[:, :h * d].unflatten(1, (h, d))


# ---- norm and rotation -----------------------------------------------------------

# dtype, tokens, heads_q, heads_k, dim, rot, interleaved, weights (q, k), extra columns
ROPE = [
    (BF16, 1, 32, 8, 128, 128, False, (1, 1), 0),
    (BF16, 77, 5, 1, 128, 128, True, (1, 1), 64),
    (F16, 33, 7, 3, 64, 32, False, (1, 1), 8),
    (F32, 19, 4, 2, 64, 64, True, (1, 0), 4),
    (F32, 130, 1, 1, 256, 64, False, (0, 1), 0),
    (BF16, 9, 3, 0, 256, 256, True, (1, 0), 0),
    (F16, 12, 0, 6, 128, 0, False, (0, 1), 0),     # norm only, keys only
    (BF16, 21, 6, 2, 128, 16, False, (0, 0), 16),  # rotation only
    (F32, 40, 2, 2, 72, 20, False, (1, 1), 4),     # sizes of the any-size kernel
    (BF16, 41, 3, 1, 80, 80, True, (1, 1), 8),
    (F16, 5, 2, 1, 512, 34, False, (1, 1), 0),
    (F32, 3, 1, 1, 8, 2, True, (1, 1), 0),
    (BF16, 1000, 13, 5, 128, 96, False, (1, 1), 0),
]


def rope_case(case, seed):
    dtype, n, hq, hk, dim, rot, inter, norms, extra = case
    d = {"q": rand(seed, (n, hq, dim), dtype), "k": rand(seed + 1, (n, hk, dim), dtype)}
    d["q"] *= 3
    d = {k: strided(v, extra) for k, v in d.items()}
    g = torch.Generator().manual_seed(seed + 2)
    w = [(1 + 0.3 * torch.randn(dim, generator=g)).to(U.DTYPES[dtype]).cuda() if on else None
         for on in norms]
    rows = n + 50
    ang = torch.rand((rows, max(rot // 2, 1)), generator=g, dtype=torch.float64) * 6.3
    cos, sin = ang.cos().float().cuda(), ang.sin().float().cuda()
    pos = torch.randint(0, rows, (n,), generator=g).cuda()
    return d, w, cos, sin, rows, pos


def rope_call(case, d, w, cos, sin, rows, pos, eps, q_out, k_out, stream=None):
    dtype, n, hq, hk, dim, rot, inter, _, _ = case
    L.lbgemm_qk_norm_rope(dtype, n, hq, hk, dim, d["q"], d["q"].stride(0), d["k"], d["k"].stride(0),
                          w[0], w[1], eps, cos, sin, rows, pos, rot, inter, q_out,
                          q_out.stride(0), k_out, k_out.stride(0), stream)


@pytest.mark.parametrize("case", ROPE)
def test_norm_rope(case):
    dtype, n, hq, hk, dim, rot, inter, norms, extra = case
    d, w, cos, sin, rows, pos = rope_case(case, 100)
    out = [torch.full((n, h, dim), float("nan"), dtype=U.DTYPES[dtype], device="cuda")
           for h in (hq, hk)]
    rope_call(case, d, w, cos, sin, rows, pos, 1e-5, *out)
    L.lbgemm_device_status()
    c, s = (z[pos][:, :rot // 2].double() for z in (cos, sin))
    for x, wi, y in zip((d["q"], d["k"]), w, out):
        if x.shape[1] == 0:
            continue
        wd = wi.double() if wi is not None else None
        ref = U.norm_rope(x.double(), wd, 1e-5, c, s, rot, inter)
        flat = U.norm_rope(x.double(), wd, 1e-5, c, s, 0, inter).abs()  # before the rotation
        size = U.rotate(flat, c.abs(), -s.abs(), rot, inter).abs() + U.rotate(
            flat, c.abs(), s.abs(), rot, inter).abs()
        tol = U.ROUND[dtype] * ref.abs() + 32 * 2.0 ** -24 * size + 2.0 ** -25
        assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() / tol).max()
    # in place gives the same bits
    rope_call(case, d, w, cos, sin, rows, pos, 1e-5, d["q"], d["k"])
    torch.cuda.synchronize()
    assert torch.equal(d["q"], out[0]) and torch.equal(d["k"], out[1])


def grad_call(case, dy, d, w, cos, sin, rows, pos, eps, dx, dw):
    dtype, n, hq, hk, dim, rot, inter, _, _ = case
    L.lbgemm_qk_norm_rope_backward(
        dtype, n, hq, hk, dim, dy[0], dy[0].stride(0), dy[1], dy[1].stride(0), d["q"],
        d["q"].stride(0), d["k"], d["k"].stride(0), w[0], w[1], eps, cos, sin, rows, pos, rot,
        inter, dx[0], dx[0].stride(0), dx[1], dx[1].stride(0), dw[0], dw[1])


def run_grad(case, seed, eps=1e-5):
    dtype, n, hq, hk, dim, rot, inter, norms, extra = case
    d, w, cos, sin, rows, pos = rope_case(case, seed)
    dy = [strided(rand(seed + 5 + i, (n, h, dim), dtype), extra) for i, h in enumerate((hq, hk))]
    dx = [torch.full((n, h, dim), float("nan"), dtype=U.DTYPES[dtype], device="cuda")
          for h in (hq, hk)]
    dw = [torch.full((dim,), float("nan"), device="cuda") if on else None for on in norms]
    grad_call(case, dy, d, w, cos, sin, rows, pos, eps, dx, dw)
    L.lbgemm_device_status()
    return d, w, cos, sin, rows, pos, dy, dx, dw


@pytest.mark.parametrize("case", ROPE)
def test_norm_rope_backward_formula(case):
    dtype, n, hq, hk, dim, rot, inter, norms, extra = case
    d, w, cos, sin, rows, pos, dy, dx, dw = run_grad(case, 200)
    c, s = (z[pos][:, :rot // 2].double() for z in (cos, sin))
    for x, wi, g, got, gw in zip((d["q"], d["k"]), w, dy, dx, dw):
        if x.shape[1] == 0:
            if gw is not None:
                assert (gw == 0).all()
            continue
        wd = wi.double() if wi is not None else None
        ref, refw = U.norm_rope_grad(x.double(), wd, 1e-5, g.double(), c, s, rot, inter)
        # magnitudes entering each channel: two terms of the rotation, the projection
        size = U.rotate(g.double().abs(), c.abs(), -s.abs(), rot, inter).abs() + U.rotate(
            g.double().abs(), c.abs(), s.abs(), rot, inter).abs()
        if wd is not None:
            r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-5)
            xh = (x.double() * r).abs()
            size = r * (wd.abs() * size + xh * (wd.abs() * size * xh).mean(-1, keepdim=True))
        tol = U.ROUND[dtype] * ref.abs() + 32 * 2.0 ** -24 * size + 2.0 ** -25
        assert ((got.double() - ref).abs() <= tol).all(), ((got.double() - ref).abs() / tol).max()
        if gw is not None:
            rot_g = U.rotate(g.double(), c, -s, rot, inter)
            total = (rot_g.abs() * xh).sum((0, 1))
            assert ((gw.double() - refw).abs() <= 2.0 ** -18 * total + 1e-12).all()
    again = [torch.empty_like(v) if v is not None else None for v in dw]
    grad_call(case, dy, d, w, cos, sin, rows, pos, 1e-5, dx, again)
    for a, b in zip(dw, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("case", [c for c in ROPE if c[0] == F32 and all(c[7])])
def test_norm_rope_backward_differences(case):
    """<grad, direction> against central differences of the fp64 forward."""
    dtype, n, hq, hk, dim, rot, inter, norms, extra = case
    d, w, cos, sin, rows, pos, dy, dx, dw = run_grad(case, 300)
    c, s = (z[pos][:, :rot // 2].double() for z in (cos, sin))
    for x, wi, g, got, gw in zip((d["q"], d["k"]), w, dy, dx, dw):
        gen = torch.Generator().manual_seed(9)
        vx = torch.randn(x.shape, generator=gen, dtype=torch.float64).cuda()
        vw = torch.randn(wi.shape, generator=gen, dtype=torch.float64).cuda()

        def loss(e):
            return (U.norm_rope(x.double() + e * vx, wi.double() + e * vw, 1e-5, c, s, rot, inter)
                    * g.double()).sum().item()

        h = 1e-5
        want = (loss(h) - loss(-h)) / (2 * h)
        parts = torch.cat([(got.double() * vx).flatten(), (gw.double() * vw).flatten()])
        # fp32 gradients: 2^-18 of the summed magnitudes; differences: h^2 of a smooth loss
        assert abs(parts.sum().item() - want) <= (2.0 ** -18 + 1e-8) * parts.abs().sum().item()


def test_norm_rope_zero_rows_and_tokens():
    """All-zero heads stay zero with finite gradients; no tokens: weight
    gradients are zero."""
    x = torch.zeros((2, 1, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw = torch.full((64,), 7.0, device="cuda")
    dy = torch.ones_like(x)
    L.lbgemm_qk_norm_rope(F32, 2, 1, 0, 64, x, 64, None, 0, w, None, 1e-6, None, None, 0, None, 0,
                          False, y, 64, None, 0)
    L.lbgemm_qk_norm_rope_backward(F32, 2, 1, 0, 64, dy, 64, None, 0, x, 64, None, 0, w, None, 1e-6,
                                   None, None, 0, None, 0, False, dx, 64, None, 0, dw, None)
    assert (y == 0).all() and torch.isfinite(dx).all() and (dw == 0).all()
    dw.fill_(7.0)
    L.lbgemm_qk_norm_rope_backward(F32, 0, 1, 0, 64, None, 64, None, 0, None, 64, None, 0, w, None,
                                   1e-6, None, None, 0, None, 0, False, None, 64, None, 0, dw,
                                   None)
    assert (dw == 0).all()


@pytest.mark.parametrize("dim", [128, 72])
def test_norm_rope_position_out_of_range(dim):
    q = rand(1, (4, 1, dim), F32)
    table = torch.zeros((10, dim // 2), device="cuda")
    for bad in (-1, 10, 1 << 40):
        pos = torch.tensor([0, bad, 9, 3], device="cuda")
        L.lbgemm_qk_norm_rope(F32, 4, 1, 0, dim, q, dim, None, 0, None, None, 0.0, table, table, 10,
                              pos, dim, False, torch.empty_like(q), dim, None, 0)
        with pytest.raises(L.LbgemmError) as e:
            L.lbgemm_device_status()
        assert e.value.status == L.ERR_INVALID_ARG
    L.lbgemm_device_status()


# ---- the cache --------------------------------------------------------------------


def to_torch(cache):
    return torch.from_numpy(cache.bytes()).cuda()


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("dim,heads,page,tokens,extra", [
    (64, 1, 16, 1, 0), (128, 3, 48, 70, 8), (64, 5, 64, 333, 16), (128, 8, 256, 1000, 0)])
def test_cache_write_and_read(dtype, dim, heads, page, tokens, extra):
    rng = np.random.default_rng(dim + tokens)
    pages = tokens // page + 3
    k, v = (rand(40 + i, (tokens, heads, dim), dtype) for i in range(2))
    k *= torch.exp(torch.randn((1, heads, dim), generator=torch.Generator().manual_seed(3))).to(
        k.dtype).cuda()
    if tokens > 60:  # vectors that an ordinary one never shows
        k[3], v[4] = 0, 0
        k[5, 0, 7], v[6, 0, 9] = math.inf, math.nan
        k[7, 0, 1], k[7, 0, 2] = -math.inf, math.nan
        v[8] *= 1e-7 if dtype == F16 else 1e-30
        v[9] = 6e-8 if dtype == F16 else 1e-40  # below the normal range of the type
        k[10] = v[10] = 60000.0 if dtype == F16 else 3e38
        k[11] = (torch.arange(dim) % 15 - 7).to(k.dtype).cuda() * 0.5  # ties of the rounding
        v[11] = (torch.arange(dim) % 29 - 14).to(k.dtype).cuda() * 0.5
    slots = rng.permutation(pages * page)[:tokens]
    drop = rng.random(tokens) < 0.1
    drop[:12] = False
    slots = np.where(drop, -1 - rng.integers(0, 5, tokens), slots)
    cache = U.Cache(pages, page, heads, dim, rng)
    buf = to_torch(cache)
    k, v = strided(k, extra), strided(v, extra)
    ds = torch.from_numpy(slots).cuda()
    L.lbgemm_kv4_write(dtype, tokens, heads, dim, k, k.stride(0), v, v.stride(0), ds, buf, pages,
                       page)
    L.lbgemm_device_status()
    keep = slots >= 0
    for i, x in enumerate((k, v)):
        codes, scale = U.quantise(x.double().cpu().numpy())
        cache.codes[i].reshape(-1, heads, dim)[slots[keep]] = codes[keep]
        cache.scales[i].reshape(-1, heads)[slots[keep]] = scale[keep]
    got, want = buf.cpu().numpy(), cache.bytes()
    # (a NaN scale may have any payload)
    sg, sw = (torch.from_numpy(z[..., page * dim:].copy()).view(torch.bfloat16).float().numpy()
              for z in (got, want))
    assert np.array_equal(got[..., :page * dim], want[..., :page * dim])
    assert np.array_equal(sg, sw, equal_nan=True)
    # read back
    ko, vo = (strided(torch.zeros_like(x), extra) for x in (k, v))
    L.lbgemm_kv4_read(dtype, tokens, heads, dim, ds, buf, pages, page, ko, ko.stride(0), vo,
                      vo.stride(0))
    L.lbgemm_device_status()
    for i, x in enumerate((ko, vo)):
        ref = np.zeros((tokens, heads, dim))
        with np.errstate(all="ignore"):
            ref[keep] = (cache.codes[i].reshape(-1, heads, dim)[slots[keep]] *
                         cache.scales[i].reshape(-1, heads)[slots[keep]][..., None])
        ref = torch.from_numpy(ref).float().to(x.dtype)
        assert torch.equal(torch.nan_to_num(x.cpu().float(), nan=123.0),
                           torch.nan_to_num(ref.float(), nan=123.0))


def test_cache_slot_out_of_range():
    k = rand(1, (3, 2, 64), BF16)
    buf = torch.zeros((2, 2, 16 * 68), dtype=torch.uint8, device="cuda")
    out = torch.full_like(k, 5.0)
    for bad in (32, 1 << 50):
        slots = torch.tensor([0, bad, 31], device="cuda")
        L.lbgemm_kv4_write(BF16, 3, 2, 64, k, 128, k, 128, slots, buf, 2, 16)
        with pytest.raises(L.LbgemmError) as e:
            L.lbgemm_device_status()
        assert e.value.status == L.ERR_INVALID_ARG
        L.lbgemm_kv4_read(BF16, 3, 2, 64, slots, buf, 2, 16, out, 128, out, 128)
        with pytest.raises(L.LbgemmError):
            L.lbgemm_device_status()
    L.lbgemm_device_status()


# ---- attention ----------------------------------------------------------------------

# dtype, dim, heads_q, heads_kv, page, rows per sequence, lengths, causal, window
ATTEND = [
    (BF16, 128, 32, 8, 64, [1], [77], True, 0),
    (BF16, 128, 8, 8, 16, [1, 1, 1], [1, 16, 17], True, 0),
    (F16, 64, 7, 1, 16, [1, 1, 1, 1], [0, 1, 33, 250], True, 0),           # an empty cache
    (BF16, 64, 16, 2, 48, [1] * 5, [2000, 1, 130, 64, 65], True, 0),
    (F16, 128, 12, 4, 256, [1, 1], [5000, 4097], False, 0),
    (BF16, 128, 4, 1, 32, [3, 5, 1], [100, 5, 700], True, 0),              # drafted tokens
    (F16, 64, 8, 2, 16, [5, 2, 7], [3, 600, 90], True, 64),                # rows before the start
    (BF16, 128, 2, 2, 64, [1, 1], [3000, 200], True, 128),                 # a window of one token's row
    (BF16, 64, 40, 8, 64, [9, 1], [1000, 1000], True, 0),
    (F16, 128, 6, 2, 16, [130, 1, 67], [130, 900, 500], True, 0),          # prompts
    (BF16, 128, 8, 2, 64, [257], [1000], True, 0),
    (BF16, 64, 3, 3, 32, [300, 5], [300, 2], True, 100),
    (F16, 128, 5, 1, 48, [129, 40], [700, 129], False, 0),
    (F16, 64, 16, 16, 128, [200, 33, 0, 64], [333, 33, 50, 64], True, 0),  # a sequence without rows
    (BF16, 128, 16, 1, 64, [70], [5000], True, 300),
    (BF16, 128, 1, 1, 16, [1], [40000], True, 0),
    (F16, 128, 64, 1, 64, [2], [513], True, 0),                            # 64 heads on one
]


def attend_inputs(case, seed, extra=0, junk=True):
    dtype, dim, hq, hk, page, rows, lens, causal, window = case
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    width = max(max(need), 1) + 2
    cache = U.Cache(pages, page, hk, dim, rng)
    order = rng.permutation(pages)
    table = np.full((len(lens), width), -1, np.int64)  # entries beyond the length: no page
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if junk:  # tokens past the length in the last page hold anything
        for b, n in enumerate(lens):
            if n % page:
                for s, v in ((0, np.nan), (1, np.inf)):
                    cache.scales[s, table[b, need[b] - 1], n % page:] = v
    q = strided(rand(seed + 1, (sum(rows), hq, dim), dtype, 0.8), extra)
    return cache, table, width, pages, q


def attend(case, q, buf, pages, table, lens, scale, with_lse=True, stream=None, max_kv=None):
    dtype, dim, hq, hk, page, rows, _, causal, window = case
    total = sum(rows)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device="cuda")
    o = torch.full((total, hq, dim), float("nan"), dtype=U.DTYPES[dtype], device="cuda")
    lse = torch.full((total, hq), float("nan"), device="cuda") if with_lse else None
    L.lbgemm_kv4_attention(dtype, len(rows), total, max(rows), hq, hk, dim, q, q.stride(0), cu, buf,
                           pages, page, torch.as_tensor(table, dtype=torch.int32).cuda(),
                           table.shape[1], torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           max(lens) if max_kv is None else max_kv, scale, causal, window, o, lse,
                           stream)
    return o, lse


def check_attention(case, cache, table, q, o, lse, scale):
    dtype, dim, hq, hk, page, rows, lens, causal, window = case
    ref, rlse, spread, reach = U.attention(
        q.double(), torch.from_numpy(cache.codes).double().cuda(),
        torch.from_numpy(cache.scales).cuda(), lens, rows, torch.from_numpy(table), page, scale,
        causal, window)
    dt = 2.0 ** -20 * 136 * reach
    tol = U.ROUND[dtype] * ref.abs() + (2.0 ** -11 + 2 * dt[..., None]) * spread + 2.0 ** -25
    err = (o.double() - ref).abs()
    assert torch.isfinite(o).all()
    assert (err <= tol).all(), (err / tol).max()
    if lse is not None:
        empty = torch.isinf(rlse)
        assert torch.equal(torch.isinf(lse), empty) and (o[empty] == 0).all()
        e = (lse.double() - rlse)[~empty].abs()
        assert (e <= (dt + 2.0 ** -20 * (1 + rlse.abs()))[~empty]).all()


@pytest.mark.parametrize("case", ATTEND)
def test_attention(case):
    dtype, dim = case[:2]
    cache, table, width, pages, q = attend_inputs(case, 500, extra=8 * (case[2] % 3))
    buf = to_torch(cache)
    scale = 1.0 / math.sqrt(dim)
    o, lse = attend(case, q, buf, pages, table, case[6], scale)
    L.lbgemm_device_status()
    check_attention(case, cache, table, q, o, lse, scale)
    # the same call gives the same bits, with and without lse, and with a
    # looser bound on the length
    o2, _ = attend(case, q, buf, pages, table, case[6], scale, with_lse=False)
    assert torch.equal(o, o2)
    o3, lse3 = attend(case, q, buf, pages, table, case[6], scale, max_kv=width * case[4])
    L.lbgemm_device_status()
    check_attention(case, cache, table, q, o3, lse3, scale)


@pytest.mark.parametrize("rows", [1, 6, 90])
def test_attention_values_far_apart(rows):
    """Scores that dwarf one another, scales of very different sizes, a first
    token that takes nearly all the weight with a tiny value."""
    case = (BF16, 128, 8, 2, 64, [rows], [1500], True, 0)
    cache, table, width, pages, q = attend_inputs(case, 900)
    rng = np.random.default_rng(5)
    cache.scales[1] = U.bf16_round(np.exp(rng.normal(0, 6, cache.scales[1].shape)))
    cache.scales[1][table[0, 0], 0] = U.bf16_round(1e-8)
    cache.scales[0][table[0, 0], 0] *= 8
    q *= 4
    o, lse = attend(case, q, to_torch(cache), pages, table, case[6], 0.3)
    L.lbgemm_device_status()
    check_attention(case, cache, table, q, o, lse, 0.3)


@pytest.mark.parametrize("rows,length", [(1, 300), (4, 300), (200, 300)])
def test_attention_poisoned_tokens(rows, length):
    """A token whose scale is not finite makes the rows that see it NaN and
    leaves the others as they were."""
    case = (F16, 64, 4, 2, 16, [rows], [length], True, 32)
    cache, table, width, pages, q = attend_inputs(case, 31)
    scale = 0.125
    o, lse = attend(case, q, to_torch(cache), pages, table, case[6], scale)
    poisoned = length - 20
    for which, value in ((0, np.nan), (1, np.inf), (1, np.nan)):
        old = cache.scales[which].copy()
        cache.scales[which][table[0, poisoned // 16], poisoned % 16, 1] = value
        cache.codes[which][table[0, poisoned // 16], poisoned % 16, 1] = 0
        o2, lse2 = attend(case, q, to_torch(cache), pages, table, case[6], scale)
        L.lbgemm_device_status()
        pos = length - rows + np.arange(rows)
        sees = torch.from_numpy((pos >= poisoned) & (pos - 32 < poisoned)).cuda()
        assert torch.isnan(o2[sees][:, 2:]).all()
        assert torch.equal(o2[:, :2], o[:, :2])
        assert torch.equal(o2[~sees], o[~sees])
        cache.scales[which] = old


def test_attention_no_keys_at_all():
    case = (BF16, 64, 4, 2, 16, [2, 70], [0, 0], True, 0)
    cache, table, width, pages, q = attend_inputs(case, 77)
    o, lse = attend(case, q, to_torch(cache), pages, table, [0, 0], 1.0)
    L.lbgemm_device_status()
    assert (o == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("rows", [1, 100])
def test_attention_past_32_bit_offsets(rows):
    """Pages beyond 4 GB of cache."""
    page, heads, dim = 256, 8, 128
    per = page * (dim + 4)
    pages = (5 << 30) // (heads * per)
    buf = torch.empty((pages, heads, per), dtype=torch.uint8, device="cuda")
    case = (BF16, dim, 8, heads, page, [rows], [700], True, 0)
    cache, _, _, small, q = attend_inputs(case, 61)
    table = np.array([[pages - 1, 2, pages - 7]])
    cache2 = U.Cache(3, page, heads, dim, np.random.default_rng(8))
    for i, at in enumerate(table[0]):
        buf[at] = to_torch(cache2)[i]
    scale = 0.1
    o, lse = attend(case, q, buf, pages, table, case[6], scale)
    L.lbgemm_device_status()
    check_attention(case, cache2, np.array([[0, 1, 2]]), q, o, lse, scale)
    # the write and read side
    k = rand(3, (2, heads, dim), BF16)
    slots = torch.tensor([(pages - 1) * page + 255, 5], device="cuda")
    L.lbgemm_kv4_write(BF16, 2, heads, dim, k, heads * dim, k, heads * dim, slots, buf, pages, page)
    back = torch.zeros_like(k), torch.zeros_like(k)
    L.lbgemm_kv4_read(BF16, 2, heads, dim, slots, buf, pages, page, back[0], heads * dim, back[1],
                      heads * dim)
    L.lbgemm_device_status()
    codes, s = U.quantise(k.double().cpu().numpy())
    want = torch.from_numpy(codes * s[..., None]).to(torch.bfloat16)
    assert torch.equal(back[0].cpu(), want) and torch.equal(back[1].cpu(), want)


@pytest.mark.parametrize("rows", [1, 100])
def test_attention_bad_indexes(rows):
    """Page numbers and lengths out of range are reported and touch nothing."""
    case = (BF16, 128, 4, 2, 16, [rows], [120], True, 0)
    cache, table, width, pages, q = attend_inputs(case, 91)
    buf = to_torch(cache)
    for bad in (-1, pages, 1 << 30):
        t = table.copy()
        t[0, 3] = bad
        attend(case, q, buf, pages, t, case[6], 0.1)
        with pytest.raises(L.LbgemmError) as e:
            L.lbgemm_device_status()
        assert e.value.status == L.ERR_INVALID_ARG
    for lens in ([121], [-1]):
        attend(case, q, buf, pages, table, lens, 0.1, max_kv=120)
        with pytest.raises(L.LbgemmError) as e:
            L.lbgemm_device_status()
        assert e.value.status == L.ERR_INVALID_ARG
    o, lse = attend(case, q, buf, pages, table, case[6], 0.1)
    L.lbgemm_device_status()
    check_attention(case, cache, table, q, o, lse, 0.1)


def test_graph_and_streams():
    """Write, norm, attention captured into one graph on a side stream, and
    replayed on changed inputs; two streams at once on the shared scratch."""
    case = (BF16, 128, 8, 2, 64, [1, 1], [5000, 300], True, 0)
    cache, table, width, pages, q = attend_inputs(case, 15, junk=False)
    buf = to_torch(cache)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    dtab = torch.as_tensor(table, dtype=torch.int32).cuda()
    lens = torch.tensor(case[6], dtype=torch.int32, device="cuda")
    scale = 0.09
    o = torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 8), device="cuda")
    k, v = rand(1, (2, 2, 128), BF16), rand(2, (2, 2, 128), BF16)
    slots_np = np.array([table[0, 4999 // 64] * 64 + 4999 % 64, table[1, 299 // 64] * 64 + 299 % 64])
    slots = torch.from_numpy(slots_np).cuda()

    def step(stream, q, o, lse):
        L.lbgemm_kv4_write(BF16, 2, 2, 128, k, 256, v, 256, slots, buf, pages, 64, stream)
        L.lbgemm_kv4_attention(BF16, 2, 2, 1, 8, 2, 128, q, q.stride(0), cu, buf, pages, 64, dtab,
                               dtab.shape[1], lens, 5000, scale, True, 0, o, lse, stream)

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    step(side, q, o, lse)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step(side.cuda_stream, q, o, lse)
    for seed in (50, 60):
        q.copy_(rand(seed, tuple(q.shape), BF16))
        k.copy_(rand(seed + 1, tuple(k.shape), BF16))
        v.copy_(rand(seed + 2, tuple(v.shape), BF16))
        o.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, x in enumerate((k, v)):
            codes, s = U.quantise(x.double().cpu().numpy())
            cache.codes[i].reshape(-1, 2, 128)[slots_np] = codes
            cache.scales[i].reshape(-1, 2)[slots_np] = s
        check_attention(case, cache, table, q, o, lse, scale)
    others = [torch.cuda.Stream() for _ in range(2)]
    qs = [rand(70 + i, tuple(q.shape), BF16) for i in range(2)]
    os = [[torch.empty_like(o) for _ in range(4)] for _ in range(2)]
    ls = [torch.empty_like(lse) for _ in range(2)]
    torch.cuda.synchronize()
    for rep in range(4):
        for i in range(2):
            L.lbgemm_kv4_attention(BF16, 2, 2, 1, 8, 2, 128, qs[i], qs[i].stride(0), cu, buf, pages,
                                   64, dtab, dtab.shape[1], lens, 5000, scale, True, 0, os[i][rep],
                                   ls[i], others[i])
    torch.cuda.synchronize()
    for i in range(2):
        for rep in range(4):
            check_attention(case, cache, table, qs[i], os[i][rep], ls[i], scale)
