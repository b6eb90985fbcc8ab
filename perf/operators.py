"""Measured cases of the attention operators around a cache held in 4 bits.

Three operators, as one serving or training step of an attention layer uses
them next to the low-bit linear layers:

- ``rope`` / ``train``: RMS norm of each query and key head with the position
  rotation in the same pass, alone or followed by its backward pass;
- ``cache``: keys and values quantised to 4 bits as they are written into a
  paged cache, and read back;
- ``attend``: attention of new tokens over that cache.

With ``own`` false ``run`` computes them by elementary torch operations in
fp32; with ``own`` true it makes the library's calls.  ``exact`` gives the
same outputs from the definitions in fp64.

Cache layout (one block of heads x page_size x (dim + 4) bytes a page): for
each head the page's key codes [page_size, dim / 2], its value codes, then
its key scales and value scales (bf16, [page_size] each).  A code is a signed
nibble, element 2j in the low half of byte j; a value is code * scale, with
scale = bf16(max|x| / 7) over the head's vector and code = round(x / scale)
clamped to [-7, 7].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}


def listed():
    return [
        # one new token of one sequence: a decoding step's norm and rotation, bound by latency
        {"name": "rope_token", "op": "rope", "dtype": "bf16", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "table": 32768},
        # a long prompt through a layer with 32 query and 8 key heads, read out of the joint projection
        {"name": "rope_prompt", "op": "rope", "dtype": "bf16", "tokens": 16384, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "table": 32768},
        # a training step: the pass and its gradients, weights' gradients among them
        {"name": "rope_train", "op": "train", "dtype": "bf16", "tokens": 8192, "heads": 32, "kv_heads": 8, "dim": 128, "rot": 128,
         "interleaved": False, "norm": True, "table": 8192},
        # a small model trained in fp32: an odd number of tokens, neighbouring pairs rotated, half of each head
        {"name": "rope_train_fp32", "op": "train", "dtype": "fp32", "tokens": 1021, "heads": 12, "kv_heads": 3, "dim": 64, "rot": 32,
         "interleaved": True, "norm": True, "table": 2048},
        # a decoding step of 64 sequences: one token each into its page
        {"name": "cache_step", "op": "cache", "dtype": "bf16", "tokens": 64, "heads": 8, "dim": 128, "page": 64},
        # prompts of 30011 tokens written, and read back for a part that needs them in 16 bits
        {"name": "cache_prompt", "op": "cache", "dtype": "bf16", "tokens": 30011, "heads": 8, "dim": 128, "page": 64},
        # the first tokens of a chat: one token over a cache that ends inside its second page
        {"name": "attend_short", "op": "attend", "dtype": "bf16", "batch": 1, "new": 1, "context": 77, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "causal": True, "window": 0},
        # one user with a very long document
        {"name": "attend_long", "op": "attend", "dtype": "bf16", "batch": 1, "new": 1, "context": 131072, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "causal": True, "window": 0},
        # a full serving batch, every sequence of another length
        {"name": "attend_batch", "op": "attend", "dtype": "bf16", "batch": 64, "new": 1, "context": 8192, "ragged": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "causal": True, "window": 0},
        # drafted tokens checked together, in a layer with a sliding window
        {"name": "attend_draft", "op": "attend", "dtype": "fp16", "batch": 24, "new": 5, "context": 4001, "ragged": True, "heads": 16,
         "kv_heads": 4, "dim": 64, "page": 16, "causal": True, "window": 1024},
        # prompts of many lengths on top of shared prefixes, one key head for each query head
        {"name": "attend_prompts", "op": "attend", "dtype": "fp16", "batch": 7, "new": 1100, "context": 3001, "ragged": True, "heads": 16,
         "kv_heads": 16, "dim": 64, "page": 32, "causal": True, "window": 0},
        # one chunk of a long prompt over what came before it
        {"name": "attend_chunk", "op": "attend", "dtype": "bf16", "batch": 1, "new": 4096, "context": 16384, "ragged": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 64, "causal": True, "window": 0},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: _cost(op) for op in ("rope", "train", "cache", "attend")}
    while True:
        op = rng.choice(["rope", "train", "cache", "attend", "attend", "attend"])
        dim = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
        heads = kv * rng.choice([1, 2, 3, 4, 4, 5, 6, 7, 8])
        if heads > 64 or (heads + 2 * kv) % 24 == 0 or heads % 24 == 0:  # widths that nothing here has
            continue
        if op in ("rope", "train"):
            tokens = _log(rng, 1, 16384)
            case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "tokens": tokens, "heads": heads, "kv_heads": kv,
                    "dim": dim, "rot": rng.choice([dim, dim, dim // 2, dim // 4]), "interleaved": rng.random() < 0.4,
                    "norm": rng.random() < 0.8, "table": tokens + rng.randrange(1, 20000)}
        elif op == "cache":
            case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "tokens": _log(rng, 1, 32768), "heads": kv,
                    "dim": dim, "page": rng.choice([16, 32, 48, 64, 128, 256])}
        else:
            new = 1 if rng.random() < 0.4 else _log(rng, 1, 4096)
            context = _log(rng, new, 131072)
            causal = rng.random() < 0.85
            case = {"op": op, "dtype": rng.choice(["bf16", "fp16"]), "batch": _log(rng, 1, 128), "new": new, "context": context,
                    "ragged": rng.random() < 0.7, "heads": heads, "kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 48, 64, 128, 256]),
                    "causal": causal, "window": _log(rng, 16, 8192) if causal and rng.random() < 0.25 else 0}
            # what the plain form holds: every score at once, and the cache in fp32
            if case["batch"] * heads * new * context > 1 << 31 or case["batch"] * context * kv * dim > 1 << 29:
                continue
        w = work(case)
        if w["bytes"] <= most[op]["bytes"] and w["flops"] <= most[op]["flops"]:
            return case


def _cost(op):
    works = [work(c) for c in listed() if c["op"] == op]
    return {k: max(w[k] for w in works) for k in ("bytes", "flops")}


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the longest first, the others spread when ragged."""
    rng = random.Random(case["batch"] * 7919 + case["context"])
    out = [(case["new"], case["context"])]
    for _ in range(case["batch"] - 1):
        if case["ragged"]:
            n = rng.randint(max(1, case["new"] // 4), case["new"])
            out.append((n, rng.randint(n, case["context"])))
        else:
            out.append(out[0])
    return out


def work(case):
    if case["op"] in ("rope", "train"):
        x = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        side = case["tokens"] * (8 + 4 * case["rot"])
        passes = 2 if case["op"] == "rope" else 4  # x in, y out; for training also dy in, dx out
        return {"bytes": passes * x * SIZES[case["dtype"]] + side, "flops": (8 if case["op"] == "rope" else 24) * x}
    if case["op"] == "cache":
        x = 2 * case["tokens"] * case["heads"]
        return {"bytes": x * (2 * case["dim"] * SIZES[case["dtype"]] + case["dim"] // 2 + 2) + 8 * case["tokens"], "flops": 5 * x * case["dim"]}
    pairs = tokens = rows = 0
    for n, length in _lengths(case):
        first = length - n  # position of the first new token
        w = case["window"]
        rows += n
        if not case["causal"]:
            pairs += n * length
            tokens += length
            continue
        if w and first >= w:
            pairs += n * w
        elif w:
            pairs += sum(min(first + i + 1, w) for i in range(n))
        else:
            pairs += n * first + n * (n + 1) // 2
        tokens += length - (max(0, first - w + 1) if w else 0)
    d = case["dim"]
    return {"bytes": tokens * case["kv_heads"] * (d + 4) + rows * case["heads"] * (2 * d * 2 + 4) + 4 * (tokens // case["page"] + 1),
            "flops": 4 * d * case["heads"] * pairs}


# ---- inputs ---------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _activations(g, tokens, heads, dim, dtype, spread=1.0):
    """Queries, keys or values as projections give them: every channel with a size and an offset of its own, a few large."""
    size = torch.exp(0.4 * torch.randn((heads, dim), generator=g, device="cuda"))
    offset = 0.5 * torch.randn((heads, dim), generator=g, device="cuda") * size
    x = torch.randn((tokens, heads, dim), generator=g, device="cuda").mul_(size * spread).add_(offset * spread)
    return x.to(dtype)


def _joint(parts):
    """The parts side by side in one buffer of a row per token, as a joint projection leaves them: views of it."""
    tokens = parts[0].shape[0]
    whole = torch.cat([p.reshape(tokens, -1) for p in parts], dim=1)
    views, at = [], 0
    for p in parts:
        n = p.shape[1] * p.shape[2]
        views.append(whole[:, at:at + n].unflatten(1, (p.shape[1], p.shape[2])))
        at += n
    return views


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case}
    dtype, dim = DTYPES[case["dtype"]], case["dim"]
    s["stream"] = torch.cuda.current_stream().cuda_stream
    if case["op"] in ("rope", "train"):
        n, hq, hk = case["tokens"], case["heads"], case["kv_heads"]
        s["q"], s["k"], _ = _joint([_activations(g, n, h, dim, dtype) for h in (hq, hk, hk)])
        s["wq"], s["wk"] = ((1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if case["norm"] else None for _ in range(2))
        angle = torch.arange(case["table"], device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (
            -torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / case["rot"])
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
        start = int(torch.randint(0, case["table"] - n + 1, (1,), generator=g, device="cuda"))
        s["positions"] = torch.arange(start, start + n, device="cuda")
        s["q_out"], s["k_out"] = (torch.empty((n, h, dim), dtype=dtype, device="cuda") for h in (hq, hk))
        if case["op"] == "train":
            s["q_grad"], s["k_grad"] = ((0.1 * torch.randn((n, h, dim), generator=g, device="cuda")).to(dtype) for h in (hq, hk))
            s["dq"], s["dk"] = torch.empty_like(s["q_out"]), torch.empty_like(s["k_out"])
            s["dwq"], s["dwk"] = (torch.empty(dim, dtype=torch.float32, device="cuda") if case["norm"] else None for _ in range(2))
        return s
    page = case["page"]
    if case["op"] == "cache":
        n, h = case["tokens"], case["heads"]
        s["k"], s["v"] = _joint([_activations(g, n, h, dim, dtype) for _ in range(2)])
        pages = -(-n // page) + 3
        s["cache"] = torch.zeros((pages, h, page * (dim + 4)), dtype=torch.uint8, device="cuda")
        order = torch.randperm(pages, generator=g, device="cuda")[: -(-n // page)]
        at = torch.arange(n, device="cuda")
        s["slots"] = order[at // page] * page + at % page
        if n <= 256:  # a decoding step: tokens of different sequences, each in a page of its own
            s["slots"] = torch.randperm(pages * page, generator=g, device="cuda")[:n]
        s["k_out"], s["v_out"] = (torch.empty((n, h, dim), dtype=dtype, device="cuda") for _ in range(2))
        return s
    lengths = _lengths(case)
    hq, hk, batch = case["heads"], case["kv_heads"], case["batch"]
    need = [-(-length // page) for _, length in lengths]
    pages, width = sum(need) + 2, max(need)
    cache = torch.empty((pages, hk, page * (dim + 4)), dtype=torch.uint8, device="cuda")
    half = page * dim // 2
    step = max(1, (1 << 26) // (page * hk * dim))
    size = torch.exp(0.4 * torch.randn((2, hk, 1, dim), generator=g, device="cuda"))
    offset = 0.5 * torch.randn((2, hk, 1, dim), generator=g, device="cuda") * size
    for p0 in range(0, pages, step):
        p1 = min(pages, p0 + step)
        for which in (0, 1):
            x = torch.randn((p1 - p0, hk, page, dim), generator=g, device="cuda").mul_(size[which]).add_(offset[which])
            codes, scale = _quantise(x.to(dtype).float())
            cache[p0:p1, :, which * half:(which + 1) * half] = _pack(codes).reshape(p1 - p0, hk, half)
            at = 2 * half + which * 2 * page
            cache[p0:p1, :, at:at + 2 * page] = scale.to(torch.bfloat16).view(torch.uint8).reshape(p1 - p0, hk, 2 * page)
    s["cache"] = cache
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((batch, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["kv_lens"] = torch.tensor([length for _, length in lengths], dtype=torch.int32, device="cuda")
    cu = [0]
    for n, _ in lengths:
        cu.append(cu[-1] + n)
    s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["rows"], s["scale"] = cu[-1], 1.0 / math.sqrt(dim)
    s["q"] = _activations(g, cu[-1], hq, dim, dtype, spread=0.7)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty((cu[-1], hq), dtype=torch.float32, device="cuda")
    return s


# ---- the plain forms --------------------------------------------------------------


def _quantise(x):
    """fp32 vectors -> (codes as fp32 whole numbers, scale as fp32 holding a bf16)."""
    scale = (x.abs().amax(-1, keepdim=True) * (1.0 / 7.0)).to(torch.bfloat16).float()
    codes = (x / scale).round().clamp(-7, 7)
    return torch.where((scale > 0) & scale.isfinite(), codes, 0.0), scale


def _pack(codes):
    n = codes.to(torch.int16) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8)


def _unpack(packed):
    n = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)
    return ((n ^ 8).to(torch.int16) - 8).float()


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] channels of x rotated in pairs, the others as they are."""
    rot = 2 * cos.shape[-1]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


EPS = 1e-6


def _plain_rope(s, x, w, cos, sin):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()
    return _rotate(x, cos, sin, s["case"]["interleaved"]).to(DTYPES[s["case"]["dtype"]])


def _plain_rope_grad(s, x, w, dy, cos, sin):
    dtype = x.dtype
    x, g = x.float(), _rotate(dy.float(), cos, -sin, s["case"]["interleaved"])
    if w is None:
        return g.to(dtype), None
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    n = x * r
    dw = (g * n).sum((0, 1))
    g = g * w.float()
    return (r * (g - n * (g * n).mean(-1, keepdim=True))).to(dtype), dw


def _plain_store(s, x, which):
    """Keys (which 0) or values (1) into the cache, and back from it."""
    page, d, half = s["case"]["page"], s["case"]["dim"], s["case"]["page"] * s["case"]["dim"] // 2
    at, inside = s["slots"] // page, s["slots"] % page
    codes, scale = _quantise(x.float())
    rows = s["cache"][..., which * half:(which + 1) * half].unflatten(-1, (page, d // 2))
    rows[at, :, inside] = _pack(codes)
    first = 2 * half + which * 2 * page
    scales = s["cache"][..., first:first + 2 * page].unflatten(-1, (page, 2))
    scales[at, :, inside] = scale.to(torch.bfloat16).view(torch.uint8)
    back = scales[at, :, inside].contiguous().view(torch.bfloat16).float()
    return (_unpack(rows[at, :, inside]) * back).to(x.dtype)


def _plain_attend(s):
    case = s["case"]
    d, hk, page, n_max = case["dim"], case["kv_heads"], case["page"], case["new"]
    group = case["heads"] // hk
    table = s["table"].clamp(min=0).long()
    batch, width = table.shape
    blocks = s["cache"][table]  # [batch, width, head, block]
    half = page * d // 2

    def part(which):
        codes = _unpack(blocks[..., which * half:(which + 1) * half].reshape(batch, width, hk, page, d // 2))
        at = 2 * half + which * 2 * page
        scale = blocks[..., at:at + 2 * page].contiguous().view(torch.bfloat16).float()
        return (codes * scale[..., None]).permute(0, 2, 1, 3, 4).reshape(batch, hk, width * page, d)

    lens, cu = s["kv_lens"].long(), s["cu_q"].long()
    n = cu[1:] - cu[:-1]
    row = torch.arange(n_max, device="cuda")
    index = (cu[:-1, None] + row).clamp(max=s["rows"] - 1)  # [batch, new]
    q = s["q"][index].float().reshape(batch, n_max, hk, group, d).permute(0, 2, 3, 1, 4).reshape(batch, hk, group * n_max, d)
    scores = (q @ part(0).transpose(-1, -2)).reshape(batch, hk, group, n_max, width * page)
    scores *= s["scale"]
    key = torch.arange(width * page, device="cuda")
    seen = key < lens[:, None, None]  # [batch, 1, key]
    position = (lens - n)[:, None] + row
    if case["causal"]:
        seen = seen & (key <= position[..., None])
    if case["window"]:
        seen = seen & (key > position[..., None] - case["window"])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top.isfinite(), top, 0.0)
    scores -= top
    scores.exp_()
    total = scores.sum(-1, keepdim=True)
    out = (scores.reshape(batch, hk, group * n_max, -1) @ part(1)).reshape(batch, hk, group, n_max, d)
    out = out / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).squeeze(-1)
    valid = row < n[:, None]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, n_max, hk * group, d)[valid]
    return out.to(DTYPES[case["dtype"]]), lse.permute(0, 3, 1, 2).reshape(batch, n_max, hk * group)[valid]


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "attend":
        return _plain_attend(s)
    if case["op"] == "cache":
        return [_plain_store(s, s["k"], 0), _plain_store(s, s["v"], 1)]
    cos, sin = s["cos"][s["positions"]][:, None], s["sin"][s["positions"]][:, None]
    outs = {"q": _plain_rope(s, s["q"], s["wq"], cos, sin), "k": _plain_rope(s, s["k"], s["wk"], cos, sin)}
    if case["op"] == "train":
        outs["dq"], outs["dwq"] = _plain_rope_grad(s, s["q"], s["wq"], s["q_grad"], cos, sin)
        outs["dk"], outs["dwk"] = _plain_rope_grad(s, s["k"], s["wk"], s["k_grad"], cos, sin)
    return outs


# ---- the library's calls ------------------------------------------------------------


def _run_own(s, case):
    from bit_tensor_gemm_gb300 import lbgemm as L
    kind, stream, dim = {"bf16": L.BF16, "fp16": L.F16, "fp32": L.F32}[case["dtype"]], s["stream"], case["dim"]
    if case["op"] == "attend":
        L.lbgemm_kv4_attention(kind, case["batch"], s["rows"], case["new"], case["heads"], case["kv_heads"], dim, s["q"], s["q"].stride(0),
                               s["cu_q"], s["cache"], s["cache"].shape[0], case["page"], s["table"], s["table"].shape[1], s["kv_lens"],
                               case["context"], s["scale"], case["causal"], case["window"], s["out"], s["lse"], stream)
        return s["out"], s["lse"]
    if case["op"] == "cache":
        n, h, pages, page = case["tokens"], case["heads"], s["cache"].shape[0], case["page"]
        L.lbgemm_kv4_write(kind, n, h, dim, s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["slots"], s["cache"], pages, page, stream)
        L.lbgemm_kv4_read(kind, n, h, dim, s["slots"], s["cache"], pages, page, s["k_out"], h * dim, s["v_out"], h * dim, stream)
        return [s["k_out"], s["v_out"]]
    n, hq, hk = case["tokens"], case["heads"], case["kv_heads"]
    turn = (s["wq"], s["wk"], EPS, s["cos"], s["sin"], case["table"], s["positions"], case["rot"], case["interleaved"])
    L.lbgemm_qk_norm_rope(kind, n, hq, hk, dim, s["q"], s["q"].stride(0), s["k"], s["k"].stride(0), *turn,
                          s["q_out"], hq * dim, s["k_out"], hk * dim, stream)
    outs = {"q": s["q_out"], "k": s["k_out"]}
    if case["op"] == "train":
        L.lbgemm_qk_norm_rope_backward(kind, n, hq, hk, dim, s["q_grad"], hq * dim, s["k_grad"], hk * dim, s["q"], s["q"].stride(0),
                                       s["k"], s["k"].stride(0), *turn, s["dq"], hq * dim, s["dk"], hk * dim, s["dwq"], s["dwk"], stream)
        outs.update(dq=s["dq"], dk=s["dk"], dwq=s["dwq"], dwk=s["dwk"])
    return outs


# ---- the definitions in fp64 ----------------------------------------------------------


def exact(case, seed):
    w = work(case)
    if w["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "cache":
        outs = []
        for x in (s["k"].double(), s["v"].double()):
            scale = (x.abs().max(dim=-1, keepdim=True).values / 7).to(torch.bfloat16).double()
            outs.append(torch.clamp(torch.round(x / scale), -7, 7) * scale)
        return outs
    if case["op"] in ("rope", "train"):
        half = case["rot"] // 2
        turn = torch.complex(s["cos"].double(), s["sin"].double())[s["positions"]][:, None]

        def forward(x, weight):
            if weight is not None:
                x = weight * x / torch.sqrt((x ** 2).mean(dim=-1, keepdim=True) + EPS)
            head = x[..., :case["rot"]]
            if case["interleaved"]:
                z = torch.view_as_complex(head.reshape(*head.shape[:-1], half, 2).contiguous()) * turn
                head = torch.view_as_real(z).reshape(head.shape)
            else:
                z = torch.complex(head[..., :half], head[..., half:]) * turn
                head = torch.cat([z.real, z.imag], -1)
            return torch.cat([head, x[..., case["rot"]:]], -1)

        outs = {}
        for name in ("q", "k"):
            weight = s["w" + name]
            x = s[name].double().requires_grad_(case["op"] == "train")
            weight = weight.double().requires_grad_(case["op"] == "train") if weight is not None else None
            y = forward(x, weight)
            outs[name] = y.detach()
            if case["op"] == "train":
                got = torch.autograd.grad(y, [x] + ([weight] if weight is not None else []), s[name + "_grad"].double())
                outs["d" + name] = got[0]
                outs["dw" + name] = got[1] if weight is not None else None
        return outs
    d, hk, page = case["dim"], case["kv_heads"], case["page"]
    group = case["heads"] // hk
    out = torch.zeros((s["rows"], case["heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["rows"], case["heads"]), dtype=torch.float64, device="cuda")
    first = 0
    for b, (n, length) in enumerate(_lengths(case)):
        used = s["cache"][s["table"][b, :-(-length // page)].long()]
        values = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
        key = torch.arange(length, device="cuda")
        place = length - n + torch.arange(n, device="cuda")
        hidden = torch.zeros((n, length), dtype=torch.bool, device="cuda")
        if case["causal"]:
            hidden |= key[None] > place[:, None]
        if case["window"]:
            hidden |= key[None] <= place[:, None] - case["window"]
        for h in range(hk):
            k, v = (used[:, h, i * page * d // 2:(i + 1) * page * d // 2].reshape(-1, d // 2).long() for i in (0, 1))
            ks, vs = (used[:, h, page * d + 2 * i * page:page * d + 2 * (i + 1) * page].reshape(-1, 2).contiguous().view(torch.bfloat16)
                      for i in (0, 1))
            k, v = (torch.stack((values[c % 16], values[c // 16]), -1).reshape(-1, d)[:length] * z[:length].double()
                    for c, z in ((k, ks), (v, vs)))
            for j in range(h * group, (h + 1) * group):
                t = (s["q"][first:first + n, j].double() @ k.T) * s["scale"]
                t[hidden] = -math.inf
                lse[first:first + n, j] = torch.logsumexp(t, -1)
                out[first:first + n, j] = torch.softmax(t, -1) @ v
        first += n
    return out, lse
