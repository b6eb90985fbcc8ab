"""One decoder block on the library's calls: the attention layer of attention_layer.py
and a mixture of experts over 4-bit weights, with the norms around both.

A step of new tokens goes through

    lbgemm_residual_norm    the norm before attention
    AttentionLayer.step     attention over the 4-bit cache
    lbgemm_residual_norm    the norm after it, the residual stream, the next norm
    lbgemm_w4_linear        the router's logits (its weights too are in 4 bits here: the
                            library has no product of two 16-bit operands)
    lbgemm_moe_route        the experts of every token
    lbgemm_moe_w4           their products
    lbgemm_residual_norm    the norm after them and the residual stream

The example feeds random hidden states to one block with random weights: a prompt
for every sequence, then single tokens, the latter as one CUDA graph, and prints
the CUDA-event time of each.

    python -m bit_tensor_gemm_gb300.decoder_block --batch 16 --prompt 500 --steps 16
"""
from __future__ import annotations

import argparse
import sys

from . import lbgemm as L
from .attention_layer import PagedCache, random_layer

_KINDS = {"torch.bfloat16": L.BF16, "torch.float16": L.F16, "torch.float32": L.F32}


def _rows(name, x, width, kinds, device):
    """The library's number for the type of x, rows of `width` elements side by side.
    (It sees addresses and strides only, so what a tensor is gets checked here.)"""
    kind = _KINDS.get(str(x.dtype))
    if kind not in kinds or x.dim() != 2 or x.shape[1] != width or x.stride(1) != 1 or \
            x.device != device:
        raise ValueError(f"{name}: rows of {width} elements side by side are needed on {device}, not "
                         f"{x.dtype} {tuple(x.shape)} with strides {x.stride()} on {x.device}")
    return kind


class Weights4:
    """4-bit weights [rows, k] with a scale for every `group` elements and row."""

    def __init__(self, rows, k, group, device="cuda"):
        import torch  # noqa: PLC0415  (device memory and streams only)
        self.rows, self.k, self.group = rows, k, group
        self.codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=device)
        self.scales = torch.empty((rows, k // group), dtype=torch.uint8, device=device)
        self.row_scales = torch.empty(rows, dtype=torch.float32, device=device)

    def store(self, w, first=0, step=1):
        """Quantises w [n, k] into the rows first, first + step, ..."""
        kind = _rows("weights", w, self.k, (L.BF16, L.F16, L.F32), self.codes.device)
        n, k = w.shape
        if first < 0 or step < 1 or (n and first + (n - 1) * step >= self.rows):
            raise ValueError("these rows are not among the weights")
        L.lbgemm_w4_quantize(kind, n, k, self.group, w, w.stride(0),
                             self.codes[first:], step * k // 2, self.scales[first:],
                             step * (k // self.group), self.row_scales[first:], step)
        return self

    def tensors(self):
        return self.codes, self.scales, self.row_scales


class Experts:
    """A router and `experts` gated layers of `inter` channels: gate, up [experts,
    inter, hidden], down [experts, hidden, inter], router [experts, hidden]."""

    def __init__(self, router, gate, up, down, top_k, group=64):
        experts, inter, hidden = gate.shape
        if up.shape != gate.shape or down.shape != (experts, hidden, inter) or \
                router.shape != (experts, hidden):
            raise ValueError("router, gate, up and down are not of the same experts")
        self.experts, self.inter, self.hidden, self.top_k, self.group = experts, inter, hidden, top_k, group
        self.router = Weights4(experts, hidden, group, gate.device).store(router)
        self.up = Weights4(experts * 2 * inter, hidden, group, gate.device)
        self.up.store(gate.reshape(-1, hidden), 0, 2).store(up.reshape(-1, hidden), 1, 2)
        self.down = Weights4(experts * hidden, inter, group, gate.device)
        self.down.store(down.reshape(-1, inter))

    def step(self, x):
        """x: bf16 or fp16 [tokens, hidden]; on torch's current stream."""
        import torch  # noqa: PLC0415
        kind = _rows("x", x, self.hidden, (L.BF16, L.F16), self.up.codes.device)
        tokens, hidden = x.shape
        logits = torch.empty((tokens, self.experts), dtype=x.dtype, device=x.device)
        L.lbgemm_w4_linear(kind, tokens, self.experts, hidden, self.group, x, x.stride(0),
                           *self.router.tensors(), logits, self.experts)
        ids = torch.empty((tokens, self.top_k), dtype=torch.int32, device=x.device)
        weights = torch.empty((tokens, self.top_k), dtype=torch.float32, device=x.device)
        L.lbgemm_moe_route(kind, tokens, self.experts, self.top_k, logits, self.experts, True, ids,
                           weights)
        y = torch.empty((tokens, hidden), dtype=x.dtype, device=x.device)
        L.lbgemm_moe_w4(kind, tokens, hidden, self.inter, self.experts, self.top_k, self.group, x,
                        x.stride(0), ids, weights, *self.up.tensors(), *self.down.tensors(), y,
                        hidden)
        return y


class DecoderBlock:
    """norms: bf16 [model] weights of the norms before attention, after it, before the
    experts and after them (the second and last may be None)."""

    def __init__(self, attention, experts, norms, residual_scale=1.0, block_scale=1.0, eps=1e-6):
        if len(norms) != 4 or norms[0] is None or norms[2] is None:
            raise ValueError("norms: four, the first and third of them not None")
        for w in norms:
            if w is not None:
                _rows("norm weights", w[None], experts.hidden, (L.BF16,), norms[0].device)
        self.attention, self.experts, self.norms = attention, experts, norms
        self.residual_scale, self.block_scale, self.eps = residual_scale, block_scale, eps

    def step(self, x, cache, new):
        """x: bf16 [tokens, model]; new: what cache.extend() gave for them; on torch's
        current stream.  Returns the residual stream after the block."""
        import torch  # noqa: PLC0415
        _rows("x", x, self.experts.hidden, (L.BF16,), self.norms[0].device)
        tokens, model = x.shape
        n, x1, n1, x2 = (torch.empty((tokens, model), dtype=x.dtype, device=x.device)
                         for _ in range(4))
        before, after, before_experts, after_experts = self.norms
        a, b, eps = self.residual_scale, self.block_scale, self.eps
        L.lbgemm_residual_norm(L.BF16, tokens, model, x, x.stride(0), None, 0, None, None, 0,
                               1.0, 1.0, before, eps, None, 0, n, model)
        y = self.attention.step(n, cache, new)
        L.lbgemm_residual_norm(L.BF16, tokens, model, x, x.stride(0), y, model, after, None, 0,
                               a, b, before_experts, eps, x1, model, n1, model)
        y = self.experts.step(n1)
        L.lbgemm_residual_norm(L.BF16, tokens, model, x1, model, y, model, after_experts, None, 0, a,
                               b, None, eps, x2, model, None, 0)
        return x2


def random_block(heads_q, heads_kv, dim, model, positions, experts, inter, top_k, group=64, seed=1,
                 device="cuda"):
    """A block with random weights that keep activations near unit size."""
    import torch  # noqa: PLC0415
    g = torch.Generator(device=device).manual_seed(seed + 1)
    rand = lambda *shape: torch.randn(shape, generator=g, device=device)  # noqa: E731
    norms = [(1 + 0.1 * rand(model)).bfloat16() for _ in range(4)]
    layer = Experts(rand(experts, model) * model ** -0.5, *(
        (rand(experts, n, k) * k ** -0.5).bfloat16()
        for n, k in ((inter, model), (inter, model), (model, inter))), top_k, group)
    return DecoderBlock(random_layer(heads_q, heads_kv, dim, model, positions, dim, seed, device),
                        layer, norms)


def main(argv=None) -> int:
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=500, help="tokens of each prompt")
    ap.add_argument("--steps", type=int, default=16, help="single tokens after it")
    ap.add_argument("--heads", type=int, default=16)
    ap.add_argument("--kv-heads", type=int, default=4)
    ap.add_argument("--dim", type=int, default=128, choices=(64, 128))
    ap.add_argument("--model", type=int, default=2048)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--inter", type=int, default=1024)
    ap.add_argument("--top", type=int, default=6)
    a = ap.parse_args(argv)
    import torch  # noqa: PLC0415

    L.load()
    total = a.prompt + a.steps + 1
    block = random_block(a.heads, a.kv_heads, a.dim, a.model, total, a.experts, a.inter, a.top)
    cache = PagedCache(a.batch, total, a.kv_heads, a.dim, 64)
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
    timed(f"prompts, {a.batch} x {a.prompt} tokens", lambda: block.step(x, cache, new))

    x1 = torch.randn((a.batch, a.model), device="cuda").bfloat16()
    held = cache.extend([1] * a.batch)
    block.step(x1, cache, held)  # (the library has met this device outside the capture)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y1 = block.step(x1, cache, dict(held, max_kv=total))

    def replay():
        graph.replay()
        return y1

    for s in range(a.steps):
        for name, value in cache.extend([1] * a.batch).items():
            if isinstance(value, torch.Tensor):
                held[name].copy_(value)
        if s in (0, a.steps - 1):
            timed(f"step {s}, {a.batch} tokens over {cache.lens.max()}", replay)
        else:
            replay()
    L.lbgemm_device_status()
    return 0


if __name__ == "__main__":
    sys.exit(main())
