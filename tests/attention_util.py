"""The attention operators in 64 bits, for the tests: written from the
formulas in include/lbgemm.h, sharing no code with the library."""
import math

import numpy as np
import torch

DTYPES = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
# half a unit in the last place of an output rounded once, relative to the
# output: 8, 11 and 24 significant bits
ROUND = {0: 2.0 ** -8, 1: 2.0 ** -11, 2: 2.0 ** -24}


def rotate(x, cos, sin, rot, interleaved):
    """x [tokens, heads, dim] in fp64; cos, sin [tokens, rot / 2]."""
    y = x.clone()
    if rot == 0:
        return y
    c, s = cos[:, None, :], sin[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, a * s + b * c
    return y


def norm_rope(x, w, eps, cos, sin, rot, interleaved):
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return rotate(x, cos, sin, rot, interleaved)


def norm_rope_grad(x, w, eps, dy, cos, sin, rot, interleaved):
    """(dx, dw) of sum(dy * norm_rope(x, w)) by the formula."""
    g = rotate(dy, cos, -sin, rot, interleaved)
    if w is None:
        return g, None
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xhat = x * r
    wg = w * g
    return r * (wg - xhat * (wg * xhat).mean(-1, keepdim=True)), (g * xhat).sum((0, 1))


def bf16_round(x):
    """float64 array -> the nearest bf16 (half to even), as float64."""
    return torch.from_numpy(np.asarray(x, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def quantise(x):
    """[..., dim] -> (codes int64, scale float64), in the fp32 steps that the
    header names."""
    with np.errstate(all="ignore"):
        x = x.astype(np.float32)
        top = np.where(np.isnan(x).any(-1), np.float32(np.nan), np.abs(x).max(-1))
        scale = bf16_round(top.astype(np.float32) * np.float32(1.0 / 7.0))
        ok = (scale > 0) & np.isfinite(scale)
        q = x / np.where(ok, scale, 1.0).astype(np.float32)[..., None]
        q = np.rint(np.where(ok[..., None], q, np.float32(0.0)))
    return np.clip(q, -7, 7).astype(np.int64), scale


class Cache:
    """A 4-bit paged cache in numpy, and its bytes."""

    def __init__(self, pages, page, heads, dim, rng=None):
        self.pages, self.page, self.heads, self.dim = pages, page, heads, dim
        self.codes = np.zeros((2, pages, page, heads, dim), np.int64)
        self.scales = np.zeros((2, pages, page, heads), np.float64)
        if rng is not None:
            self.codes[:] = rng.integers(-8, 8, self.codes.shape)
            self.scales[:] = bf16_round(np.exp(rng.normal(-1.5, 0.7, self.scales.shape)))

    def bytes(self):
        out = np.empty((self.pages, self.heads, self.page * (self.dim + 4)), np.uint8)
        half = self.page * self.dim // 2
        for i in range(2):
            n = (self.codes[i] & 15).transpose(0, 2, 1, 3)  # [pages, heads, page, dim]
            packed = (n[..., 0::2] | (n[..., 1::2] << 4)).astype(np.uint8)
            out[:, :, i * half:(i + 1) * half] = packed.reshape(self.pages, self.heads, half)
            s = torch.from_numpy(self.scales[i].transpose(0, 2, 1).copy()).to(torch.bfloat16)
            at = 2 * half + 2 * i * self.page
            out[:, :, at:at + 2 * self.page] = s.view(torch.uint8).numpy()
        return out


def attention(q, cache_codes, cache_scales, lens, rows, table, page, scale, causal, window):
    """q [total, heads_q, dim] fp64; cache_codes [2, pages, page, heads, dim],
    cache_scales [2, pages, page, heads] (torch fp64, same device).  Returns o,
    lse, spread = sum_j p_j |v_j| and reach = the largest scale * ks_j * sum_d
    |q_d| of the tokens a row sees."""
    total, hq, dim = q.shape
    hk = cache_codes.shape[3]
    group = hq // hk
    dev = q.device
    o = torch.zeros_like(q)
    spread = torch.zeros_like(q)
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device=dev)
    reach = torch.zeros((total, hq), dtype=torch.float64, device=dev)
    first = 0
    for b, (n, length) in enumerate(zip(rows, lens)):
        if n and length:
            j = torch.arange(length, device=dev)
            pg = table[b][(j // page).cpu()].to(dev).long()
            at = j % page
            pos = length - n + torch.arange(n, device=dev)
            seen = torch.ones((n, length), dtype=torch.bool, device=dev)
            if causal:
                seen &= j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
            for h in range(hk):
                ks, vs = cache_scales[0, pg, at, h], cache_scales[1, pg, at, h]
                kc, vc = cache_codes[0, pg, at, h], cache_codes[1, pg, at, h]
                used = seen.any(0)
                # what no row sees has no effect, whatever it holds
                ks, vs = (torch.where(used, z, 0.0) for z in (ks, vs))
                k, v = kc * ks[:, None], vc * vs[:, None]
                for g in range(h * group, (h + 1) * group):
                    x = q[first:first + n, g]
                    t = torch.where(seen, (x @ k.T) * scale, -math.inf)
                    lse[first:first + n, g] = torch.logsumexp(t, -1)
                    any_ = seen.any(-1)
                    p = torch.where(any_[:, None], torch.softmax(t, -1), 0.0)
                    o[first:first + n, g] = p @ v
                    spread[first:first + n, g] = p @ v.abs()
                    reach[first:first + n, g] = (
                        (seen * ks[None]).amax(-1) * abs(scale) * x.abs().sum(-1))
        first += n
    return o, lse, spread, reach
