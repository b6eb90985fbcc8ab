"""One attention layer on the library's calls: 8-bit linear layers around norm,
rotation and attention over a cache held in 4 bits.

A step of new tokens (a prompt, a chunk of one, or one token of each sequence)
goes through

    lbgemm_linear_quant     x -> queries, keys and values, one projection
    lbgemm_qk_norm_rope     norm and rotation of the query and key heads, read
                            out of the projection and written back into it
    lbgemm_kv4_write        keys and values into the sequences' pages
    lbgemm_kv4_attention    the new tokens' attention over all pages
    lbgemm_linear_quant     the output projection

with nothing copied in between.  The example feeds random hidden states to one
layer with random weights: a prompt for every sequence, then single tokens, the
latter as one CUDA graph, and prints the CUDA-event time of each.

    python -m bit_tensor_gemm_gb300.attention_layer --batch 16 --prompt 1000 --steps 32
"""
from __future__ import annotations

import argparse
import sys

import numpy as np

from . import lbgemm as L


class PagedCache:
    """Pages of a 4-bit cache for `batch` sequences, handed out as they grow."""

    def __init__(self, batch, tokens, heads, dim, page_size, device="cuda"):
        import torch  # noqa: PLC0415  (device memory and streams only)
        self.torch, self.device = torch, device
        self.heads, self.dim, self.page_size = heads, dim, page_size
        self.width = -(-tokens // page_size)
        self.pages = batch * self.width
        self.bytes = L.lbgemm_kv4_page_bytes(heads, dim, page_size)
        if self.bytes == 0:
            raise ValueError("no 4-bit cache for these sizes")
        self.buffer = torch.empty(self.pages * self.bytes, dtype=torch.uint8, device=device)
        self.free = list(range(self.pages - 1, -1, -1))
        self.table = np.full((batch, self.width), -1, dtype=np.int32)
        self.lens = np.zeros(batch, dtype=np.int32)

    def extend(self, rows):
        """Room for rows[b] more tokens of every sequence b.  Returns the step's
        device arrays: positions and slots of the new tokens, their cu_q, the page
        table and the lengths; and the longest row count and length."""
        rows = np.asarray(rows)
        if rows.shape != self.lens.shape or (rows < 0).any():
            raise ValueError("a row count, 0 or more, is needed for every sequence")
        if (self.lens + rows > self.width * self.page_size).any():
            raise ValueError("a sequence outgrows the cache")
        positions, slots = [], []
        for b, n in enumerate(rows):
            at = np.arange(self.lens[b], self.lens[b] + n)
            for page in range(-(-int(self.lens[b]) // self.page_size),
                              -(-int(self.lens[b] + n) // self.page_size)):
                self.table[b, page] = self.free.pop()
            positions.append(at)
            slots.append(self.table[b, at // self.page_size].astype(np.int64) * self.page_size +
                         at % self.page_size)
        self.lens += rows.astype(np.int32)
        up = lambda x, kind: self.torch.from_numpy(np.ascontiguousarray(x, dtype=kind)).to(self.device)  # noqa: E731
        return dict(positions=up(np.concatenate(positions), np.int64),
                    slots=up(np.concatenate(slots), np.int64),
                    cu_q=up(np.concatenate([[0], np.cumsum(rows)]), np.int32),
                    table=up(self.table, np.int32), lens=up(self.lens, np.int32),
                    max_q=int(rows.max()), max_kv=int(self.lens.max()))


class AttentionLayer:
    """The layer's weights: `qkv` int8 [(heads_q + 2 heads_kv) dim, model], `out`
    int8 [model, heads_q dim], their fp32 scales by row, the norm weights of query
    and key heads (bf16, or None) and the rotation tables (fp32 [positions,
    rot / 2])."""

    def __init__(self, heads_q, heads_kv, dim, qkv, qkv_scale, out, out_scale, q_norm, k_norm,
                 cosines, sines, eps=1e-6, interleaved=False, window=0):
        self.heads_q, self.heads_kv, self.dim = heads_q, heads_kv, dim
        self.qkv, self.qkv_scale, self.out, self.out_scale = qkv, qkv_scale, out, out_scale
        self.q_norm, self.k_norm, self.cosines, self.sines = q_norm, k_norm, cosines, sines
        self.eps, self.interleaved, self.window = eps, interleaved, window

    def step(self, x, cache, new, stream=None):
        """x: bf16 [tokens, model], the new tokens' hidden states, sequence after
        sequence; new: what cache.extend() gave for them.  Returns [tokens, model].
        stream: as lbgemm takes it; what the step allocates, its result among it, then
        belongs to that stream (torch hands memory out again in the order of the
        stream that it belongs to)."""
        import torch  # noqa: PLC0415
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), x.device)
            with torch.cuda.stream(stream):
                return self.step(x, cache, new)
        tokens, model = x.shape
        hq, hk, dim = self.heads_q, self.heads_kv, self.dim
        width = (hq + 2 * hk) * dim
        joint = torch.empty((tokens, width), dtype=torch.bfloat16, device=x.device)
        L.lbgemm_linear_quant(tokens, width, model, x, self.qkv, self.qkv_scale, joint)
        q, k, v = joint[:, :hq * dim], joint[:, hq * dim:(hq + hk) * dim], joint[:, (hq + hk) * dim:]
        L.lbgemm_qk_norm_rope(L.BF16, tokens, hq, hk, dim, q, width, k, width, self.q_norm,
                              self.k_norm, self.eps, self.cosines, self.sines,
                              self.cosines.shape[0], new["positions"], 2 * self.cosines.shape[1],
                              self.interleaved, q, width, k, width)
        L.lbgemm_kv4_write(L.BF16, tokens, hk, dim, k, width, v, width, new["slots"], cache.buffer,
                           cache.pages, cache.page_size)
        o = torch.empty((tokens, hq * dim), dtype=torch.bfloat16, device=x.device)
        L.lbgemm_kv4_attention(L.BF16, len(cache.lens), tokens, new["max_q"], hq, hk, dim, q, width,
                               new["cu_q"], cache.buffer, cache.pages, cache.page_size,
                               new["table"], cache.width, new["lens"], new["max_kv"], dim ** -0.5,
                               True, self.window, o, None)
        y = torch.empty((tokens, model), dtype=torch.bfloat16, device=x.device)
        L.lbgemm_linear_quant(tokens, model, hq * dim, o, self.out, self.out_scale, y)
        return y


def random_layer(heads_q, heads_kv, dim, model, positions, rot, seed=1, device="cuda", **kw):
    """A layer with random weights that keep activations near unit size."""
    import torch  # noqa: PLC0415
    g = torch.Generator(device=device).manual_seed(seed)
    width = (heads_q + 2 * heads_kv) * dim

    def weights(n, k):
        w = torch.randint(-127, 128, (n, k), dtype=torch.int8, generator=g, device=device)
        return w, torch.full((n,), 1.0 / (73.5 * k ** 0.5), device=device)  # 73.5: their rms

    def norm():
        return (1 + 0.1 * torch.randn(dim, generator=g, device=device)).bfloat16()

    angle = torch.arange(positions, device=device)[:, None] * 10000.0 ** (
        -torch.arange(0, rot, 2, device=device) / max(rot, 1))
    return AttentionLayer(heads_q, heads_kv, dim, *weights(width, model),
                          *weights(model, heads_q * dim), norm(), norm(),
                          torch.cos(angle).float().contiguous(),
                          torch.sin(angle).float().contiguous(), **kw)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000, help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=32, help="single tokens after it")
    ap.add_argument("--heads", type=int, default=32)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--dim", type=int, default=128, choices=(64, 128))
    ap.add_argument("--model", type=int, default=4096)
    ap.add_argument("--page", type=int, default=64)
    ap.add_argument("--window", type=int, default=0)
    a = ap.parse_args(argv)
    import torch  # noqa: PLC0415

    L.load()
    total = a.prompt + a.steps + 1
    layer = random_layer(a.heads, a.kv_heads, a.dim, a.model, total, a.dim, window=a.window)
    cache = PagedCache(a.batch, total, a.kv_heads, a.dim, a.page)
    stream = torch.cuda.current_stream()

    def timed(word, call):
        e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        e0.record(stream)
        y = call()
        e1.record(stream)
        e1.synchronize()
        print(f"{word}: {e0.elapsed_time(e1) * 1e3:.1f} us, rms {y.float().square().mean().sqrt():.4f}",
              flush=True)

    x = torch.randn((a.batch * a.prompt, a.model), device="cuda").bfloat16()
    new = cache.extend([a.prompt] * a.batch)
    timed(f"prompts, {a.batch} x {a.prompt} tokens", lambda: layer.step(x, cache, new))

    # Single tokens: the calls are captured once with the longest length as the
    # bound; every step then copies its indexes into the graph's own and replays.
    x1 = torch.randn((a.batch, a.model), device="cuda").bfloat16()
    held = cache.extend([1] * a.batch)
    layer.step(x1, cache, held)  # (the library has met this device outside the capture)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = layer.step(x1, cache, dict(held, max_kv=total))
    for s in range(a.steps):
        for name, value in cache.extend([1] * a.batch).items():
            if isinstance(value, torch.Tensor):
                held[name].copy_(value)

        def call():
            graph.replay()
            return y1
        if s in (0, a.steps - 1):
            timed(f"step {s}, {a.batch} tokens over {cache.lens.max()}", call)
        else:
            graph.replay()
    L.lbgemm_device_status()
    return 0


if __name__ == "__main__":
    sys.exit(main())
