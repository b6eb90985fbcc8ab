"""Attention over the 4-bit cache in 64 bits with the error that the arithmetic
of lbgemm_kv4_attention allows, for the tests; written from the formulas in
include/lbgemm.h, sharing no code with the library.

With A = the largest scale * sum_d |q_d k_jd| of a row's tokens j, everything in
natural logarithms:
  scores      codes and queries are exact in fp16; their products' sums go
              through dim / 16 matrix instructions of fp32 sums, each off by at
              most 2^-22 of A (operands lined up, digits dropped), then three
              roundings and the exponential's: dt = (dim / 16 + 6) 2^-22 A
  sums        of n tokens' weights in steps of 128, in fp32:
              (n / 128 + 60) 2^-24 of themselves
  lse         dt + sums + 2^-22 |lse|
  o           a weight times a value scale is rounded to fp16: 2^-11 of itself or
              2^-30 of the row's largest, whichever is more; then the output's
              rounding, or half its smallest number
"""
import math

import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def attention(q, dtype, cache, lens, rows, table, scale, causal, window, lost=0.0):
    """q [total, heads_q, dim]; cache: attention_util.Cache.  Returns o, lse and
    what each may be off by, in fp64; weights below `lost` of a row's largest may
    count as 0."""
    q = q.double()
    dev, (total, hq, dim) = q.device, q.shape
    hk, page = cache.heads, cache.page
    codes = torch.from_numpy(cache.codes).to(dev).double()
    scales = torch.from_numpy(cache.scales).to(dev)
    o, tol = torch.zeros_like(q), torch.zeros_like(q)
    lse = torch.full((total, hq), -math.inf, dtype=torch.float64, device=dev)
    tol_lse = torch.zeros((total, hq), dtype=torch.float64, device=dev)
    group, first = hq // hk, 0
    for b, (n, length) in enumerate(zip(rows, lens)):
        if n and length:
            j = torch.arange(length, device=dev)
            pages, at = torch.as_tensor(table[b], device=dev).long()[j // page], j % page
            pos = length - n + torch.arange(n, device=dev)
            seen = torch.ones((n, length), dtype=torch.bool, device=dev)
            if causal:
                seen &= j[None] <= pos[:, None]
            if window:
                seen &= j[None] > pos[:, None] - window
            some = seen.any(-1)[None, :, None]
            for h in range(hk):
                k, v = ((codes[i, pages, at, h] * scales[i, pages, at, h][:, None]) for i in (0, 1))
                heads = slice(h * group, (h + 1) * group)
                x = q[first:first + n, heads].transpose(0, 1)  # [group, n, dim]
                t = torch.where(seen, scale * (x @ k.T), -math.inf)
                big = torch.where(seen, abs(scale) * (x.abs() @ k.abs().T), 0.0).amax(-1, keepdim=True)
                p = torch.where(some, torch.softmax(t, -1), 0.0)
                z = torch.logsumexp(t, -1, keepdim=True)
                y, spread = p @ v, p @ v.abs()
                # the largest weight x value scale of a row, and a code of at most 8
                least = 2.0 ** -30 * 8 * (p * scales[1, pages, at, h].abs()).amax(-1, keepdim=True)
                dt = (dim / 16 + 6) * 2.0 ** -22 * big
                sums = (length / 128 + 60) * 2.0 ** -24
                e = (ROUND[dtype] * y.abs() + (2.0 ** -11 + 2 * dt + sums) * spread +
                     seen.sum(-1)[:, None] * least + LEAST[dtype])
                if lost:
                    e += torch.where(p < lost * p.amax(-1, keepdim=True), p, 0.0) @ v.abs()
                o[first:first + n, heads] = y.transpose(0, 1)
                tol[first:first + n, heads] = e.transpose(0, 1)
                lse[first:first + n, heads] = z[..., 0].T
                tol_lse[first:first + n, heads] = (dt + sums + 2.0 ** -22 * z.abs())[..., 0].T
        first += n
    return o, lse, tol, tol_lse


def check(o, lse, ref):
    want, want_lse, tol, tol_lse = ref
    assert torch.isfinite(o).all()
    empty = torch.isinf(want_lse)
    err = (o.double() - want).abs()
    assert (o[empty] == 0).all() and (err <= tol)[~empty].all(), (err / tol)[~empty].max().item()
    assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
    off = ((lse.double() - want_lse).abs() / tol_lse)[~empty]
    assert (off <= 1).all(), off.max().item()
