"""The feed-forward operators in 64 bits, for the tests: written from the formulas
in include/lbgemm.h, sharing no code with the library."""
import numpy as np
import torch

DTYPES = {0: torch.bfloat16, 1: torch.float16, 2: torch.float32}
# half a unit in the last place of an output rounded once, relative to the output
ROUND = {0: 2.0 ** -8, 1: 2.0 ** -11, 2: 2.0 ** -24}


def e4m3(byte):
    """The numbers that e4m3 bytes stand for (numpy uint8 -> float64)."""
    byte = byte.astype(np.int64)
    exponent, digits = (byte >> 3) & 15, byte & 7
    size = np.where(exponent > 0, (8 + digits) * 2.0 ** (exponent - 10.0), digits * 2.0 ** -9)
    size = np.where((byte & 127) == 127, np.nan, size)
    return np.where(byte >= 128, -size, size)


def to_e4m3(x):
    """The nearest e4m3 bytes of x >= 0, half to even, saturating (numpy)."""
    values = e4m3(np.arange(127, dtype=np.uint8))  # ascending
    hi = np.clip(np.searchsorted(values, x), 1, 126)
    lo = hi - 1
    a, b = x - values[lo], values[hi] - x
    up = (b < a) | ((a == b) & (hi % 2 == 0))
    return np.where(up, hi, lo).astype(np.uint8)


def pack(codes):
    """int codes [rows, k] -> bytes [rows, k / 2]."""
    c = (codes & 15).astype(np.uint32).reshape(codes.shape[0], -1, 8)
    word = np.zeros(c.shape[:2], np.uint32)
    for e in range(8):
        word |= c[..., e] << np.uint32(4 * (e // 2) + 16 * (e % 2))
    return word.view(np.uint8).reshape(codes.shape[0], -1)


def unpack(packed):
    word = np.ascontiguousarray(packed).view(np.uint32)
    c = np.stack([(word >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & 15 for e in range(8)], -1)
    c = c.reshape(packed.shape[0], -1).astype(np.int64)
    return np.where(c >= 8, c - 16, c)


def quantise(w, group):
    """fp32 [rows, k] -> codes, e4m3 bytes, row scales, in the header's fp32 steps."""
    rows, k = w.shape
    f = np.float32
    with np.errstate(all="ignore"):
        row = np.abs(w).max(1) * f(1.0 / 3136.0)
        ok = np.isfinite(np.abs(w).sum(1, dtype=np.float64)) & (row > 0)
        row = np.where(np.isfinite(np.abs(w).sum(1, dtype=np.float64)), row, f(np.nan)).astype(f)
        blocks = w.reshape(rows, -1, group)
        t = np.abs(blocks).max(2) * f(1.0 / 7.0) / np.where(ok, row, f(1))[:, None]
        scale = np.where(ok[:, None], to_e4m3(np.where(ok[:, None], t, 0).astype(np.float64)), 0)
        scale = scale.astype(np.uint8)
        step = (e4m3(scale).astype(f) * np.where(ok, row, f(0))[:, None]).astype(f)
        q = np.rint(blocks / np.where(step > 0, step, f(1))[..., None])
        codes = np.where(step[..., None] > 0, np.clip(q, -7, 7), 0)
    return codes.reshape(rows, k).astype(np.int64), scale, row


class Weights:
    """Random 4-bit rows of every code and ordinary scales, and their tensors."""

    def __init__(self, rng, rows, k, group, size=None, scales=None):
        self.codes = rng.integers(-8, 8, (rows, k))
        self.scales = rng.integers(0x28, 0x50, (rows, k // group)).astype(np.uint8) \
            if scales is None else scales
        size = k ** -0.5 if size is None else size
        self.row = (size * np.exp(rng.normal(0, 0.3, rows))).astype(np.float32)
        self.group = group

    def dense(self):
        """fp64 on the GPU."""
        w = torch.from_numpy(self.codes.astype(np.float64)).cuda()
        s = torch.from_numpy(e4m3(self.scales)).cuda().repeat_interleave(self.group, 1)
        return w * s * torch.from_numpy(self.row.astype(np.float64)).cuda()[:, None]

    def tensors(self):
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return up(pack(self.codes)), up(self.scales), up(self.row)


def route(logits, top_k, renormalize):
    """numpy fp64 [tokens, experts] -> ids, weights."""
    l = np.where(np.isnan(logits), -np.inf, np.minimum(logits, np.finfo(np.float32).max))
    tokens, experts = l.shape
    ids = np.full((tokens, top_k), -1, np.int32)
    weights = np.zeros((tokens, top_k))
    for t in range(tokens):
        order = sorted((e for e in range(experts) if l[t, e] > -np.inf), key=lambda e: (-l[t, e], e))
        chosen = order[:top_k]
        if not chosen:
            continue
        p = np.exp(l[t] - l[t, chosen[0]])
        ids[t, :len(chosen)] = chosen
        weights[t, :len(chosen)] = p[chosen] / p[chosen if renormalize else order].sum()
    return ids, weights


def residual_norm(x, y, post, gate, nxt, a, b, eps):
    """fp64 tensors -> x', n (None without a weight)."""
    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w
    new = a * x
    if y is not None:
        z = y if post is None else norm(y, post)
        new = new + b * (z if gate is None else gate * z)
    return new, None if nxt is None else norm(new, nxt)
