"""Measured cases of the operators of a decoder block's feed-forward half with
weights in 4 bits.

Four operators, as a serving or training step uses them beside attention:

- ``linear``: 16-bit activations times 4-bit weights with group scales;
- ``route``: the top experts of every token and their weights;
- ``moe``: a mixture of experts over 4-bit weights, from the chosen experts to
  the summed output;
- ``norm`` / ``train``: the norms after and before a block with its gate and the
  residual stream's scales, alone or followed by the backward pass.

With ``own`` false ``run`` computes them by elementary torch operations in
fp32; with ``own`` true it makes the library's calls.  ``exact`` gives the
same outputs from the definitions in fp64.

4-bit weights [rows, k]: the weight (n, i) is code * scale * row_scale with
signed codes, one e4m3 scale for every `group` elements of a row (uint8 [rows,
k / group]) and one fp32 scale a row.  Eight codes along k make a little-endian
32-bit word: element 2j in bits 4j .. 4j + 3, element 2j + 1 in bits 16 + 4j ..
Experts are stacked: the up weights [experts, 2 inter, hidden] have the gate's
row i at 2i and the up projection's at 2i + 1, the down weights [experts,
hidden, inter].
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SIZES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6


def listed():
    return [
        # one new token of one sequence through a layer's widest projection: the weights' stream is all there is
        {"name": "w4_token", "op": "linear", "dtype": "bf16", "tokens": 1, "rows": 11008, "k": 4096, "group": 128},
        # a decoding step of a dozen sequences through the projection back, fp16
        {"name": "w4_step", "op": "linear", "dtype": "fp16", "tokens": 12, "rows": 4096, "k": 11008, "group": 64},
        # drafted tokens of nine sequences into a small vocabulary: odd rows, tokens, and a k that no tile divides
        {"name": "w4_drafts", "op": "linear", "dtype": "bf16", "tokens": 45, "rows": 5003, "k": 4000, "group": 32},
        # a long prompt through the same projection: bound by the matrix units
        {"name": "w4_prompt", "op": "linear", "dtype": "bf16", "tokens": 4096, "rows": 11008, "k": 4096, "group": 128},
        # the router of a decoding step, logits in fp32, an odd number of experts
        {"name": "route_step", "op": "route", "dtype": "fp32", "tokens": 33, "experts": 60, "top": 4, "renormalize": True, "masked": False},
        # the router of a long prompt, logits as a bf16 projection leaves them (many ties)
        {"name": "route_prompt", "op": "route", "dtype": "bf16", "tokens": 16384, "experts": 128, "top": 8, "renormalize": False,
         "masked": False},
        # one token through a layer of experts: as many experts' weights as it chose
        {"name": "moe_token", "op": "moe", "dtype": "bf16", "tokens": 1, "hidden": 2048, "inter": 1024, "experts": 64, "top": 6, "group": 128,
         "padded": 0},
        # a decoding step of 24 sequences: nearly all experts, two or three tokens each
        {"name": "moe_step", "op": "moe", "dtype": "bf16", "tokens": 24, "hidden": 2048, "inter": 1024, "experts": 64, "top": 6, "group": 64,
         "padded": 0},
        # prompts of 4096 tokens with some padding behind them
        {"name": "moe_prompt", "op": "moe", "dtype": "bf16", "tokens": 4096, "hidden": 2048, "inter": 1024, "experts": 64, "top": 6,
         "group": 128, "padded": 71},
        # a decoding step's norms and residual
        {"name": "norm_step", "op": "norm", "dtype": "bf16", "tokens": 16, "width": 4096, "post": True, "gate": "none", "next": True},
        # a training step of a block: the pass and its gradients, a gate for every channel
        {"name": "norm_train", "op": "train", "dtype": "bf16", "tokens": 8192, "width": 4096, "post": True, "gate": "channel", "next": True},
        # a small model in fp32 with a gate of every token's own, an odd number of tokens
        {"name": "norm_train_fp32", "op": "train", "dtype": "fp32", "tokens": 1021, "width": 1000, "post": True, "gate": "token", "next": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: _cost(op) for op in ("linear", "route", "moe", "norm")}
    while True:
        op = rng.choice(["linear", "linear", "route", "moe", "moe", "norm", "train"])
        two = rng.choice(["bf16", "bf16", "fp16"])
        if op == "linear":
            group = rng.choice([32, 64, 128])
            case = {"op": op, "dtype": two, "tokens": rng.choice([_log(rng, 1, 64), _log(rng, 1, 4096)]), "rows": _log(rng, 9, 32768),
                    "k": group * _log(rng, 1, 16384 // group), "group": group}
        elif op == "route":
            experts = _log(rng, 2, 512)
            case = {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "tokens": _log(rng, 1, 16384), "experts": experts,
                    "top": rng.randint(1, min(16, experts)), "renormalize": rng.random() < 0.5, "masked": rng.random() < 0.3}
        elif op == "moe":
            group, experts, tokens = rng.choice([32, 64, 128]), _log(rng, 1, 256), _log(rng, 1, 4096)
            case = {"op": op, "dtype": two, "tokens": tokens, "hidden": group * _log(rng, 2, 4096 // group),
                    "inter": group * _log(rng, 1, 4096 // group), "experts": experts, "top": rng.randint(1, min(8, experts)),
                    "group": group, "padded": rng.randrange(1 + tokens // 4) if rng.random() < 0.4 else 0}
        else:
            post = rng.random() < 0.7
            case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16", "fp32"]), "tokens": _log(rng, 1, 16384),
                    "width": 8 * _log(rng, 1, 1024), "post": post, "gate": rng.choice(["none", "channel", "token"]),
                    "next": rng.random() < 0.8 or not post}
        if op == "moe" and case["experts"] * case["hidden"] * case["inter"] > 1 << 28:
            continue
        w, limit = work(case), most["norm" if op == "train" else op]
        if w["bytes"] <= limit["bytes"] and w["flops"] <= limit["flops"]:
            return case


def _cost(op):
    works = [work(c) for c in listed() if c["op"] in ((op, "train") if op == "norm" else (op,))]
    return {k: max(w[k] for w in works) for k in ("bytes", "flops")}


def work(case):
    op, t = case["op"], case["tokens"]
    if op == "linear":
        n, k = case["rows"], case["k"]
        return {"bytes": n * k // 2 + n * k // case["group"] + 4 * n + 2 * t * (n + k), "flops": 2 * t * n * k}
    if op == "route":
        return {"bytes": t * (case["experts"] * SIZES[case["dtype"]] + 8 * case["top"]), "flops": 4 * t * case["experts"]}
    if op == "moe":
        h, i, e, top = case["hidden"], case["inter"], case["experts"], case["top"]
        real = t - case["padded"]
        active = e * (1 - (1 - top / e) ** real)  # experts that anyone chooses, were they all alike
        weights = 3 * h * i // 2 + 3 * h * i // case["group"] + 4 * (2 * i + h)
        return {"bytes": int(active * weights) + 4 * t * h + 8 * t * top, "flops": 6 * real * top * h * i}
    n = t * case["width"]
    gate = n if case["gate"] == "token" else 0
    reads, writes = 2 * n + gate, n * (2 if case["next"] else 1)
    if op == "train":  # and again: the inputs, the outputs' gradients in, the inputs' out
        reads, writes = 2 * reads + writes, writes + 2 * n + gate
    return {"bytes": (reads + writes) * SIZES[case["dtype"]], "flops": (10 if op == "norm" else 34) * n}


# ---- inputs ---------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, scale=1.0):
    return torch.randn(shape, generator=g, device="cuda").mul_(scale)


def _activations(g, tokens, width, dtype):
    """Hidden states: every channel with a size of its own, a few large."""
    return _normal(g, (tokens, width)).mul_(torch.exp(_normal(g, (width,), 0.4))).to(dtype)


def _quantise(w, group):
    """fp32 [rows, k] -> (packed codes, e4m3 scales as bytes, row scales)."""
    rows, k = w.shape
    row = w.abs().amax(1) * (1.0 / 3136.0)
    blocks = w.view(rows, k // group, group)
    scale = (blocks.abs().amax(2) * (1.0 / 7.0) / row[:, None]).to(torch.float8_e4m3fn)
    step = scale.float() * row[:, None]
    codes = torch.where(step[..., None] > 0, (blocks / step[..., None]).round().clamp(-7, 7), 0.0)
    c = (codes.to(torch.int32) & 15).reshape(rows, k // 8, 8)
    word = c[..., 0]
    for e in range(1, 8):
        word = word | (c[..., e] << (4 * (e // 2) + 16 * (e % 2)))
    return word.contiguous().view(torch.uint8).view(rows, k // 2), scale.view(torch.uint8), row


def _weights(g, rows, k, group):
    """Rows of different sizes, a few large elements in them, quantised in pieces."""
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((rows, k // group), dtype=torch.uint8, device="cuda")
    row = torch.empty(rows, device="cuda")
    piece = max(1, (1 << 26) // k)
    for a in range(0, rows, piece):
        b = min(rows, a + piece)
        w = _normal(g, (b - a, k), k ** -0.5).mul_(torch.exp(_normal(g, (b - a, 1), 0.3)))
        codes[a:b], scales[a:b], row[a:b] = _quantise(w, group)
    return codes, scales, row


def prepare(case, seed):
    g = _gen(seed)
    s = {"case": case, "stream": torch.cuda.current_stream().cuda_stream}
    op, t, dtype = case["op"], case["tokens"], DTYPES[case["dtype"]]
    if op == "linear":
        s["x"] = _activations(g, t, case["k"], dtype)
        s["w"] = _weights(g, case["rows"], case["k"], case["group"])
        s["y"] = torch.empty((t, case["rows"]), dtype=dtype, device="cuda")
        return s
    if op in ("route", "moe"):
        e, top = case["experts"], case["top"]
        logits = _normal(g, (t, e), 1.5).add_(_normal(g, (e,), 0.5))  # some experts are liked more
        if op == "route":
            if case["masked"]:  # experts that a token may not use, at times nearly all of them
                share = torch.rand((t, 1), generator=g, device="cuda") ** 0.25
                logits.masked_fill_(torch.rand((t, e), generator=g, device="cuda") < share, -math.inf)
            s["logits"] = logits.to(dtype)
            s["ids"] = torch.empty((t, top), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((t, top), device="cuda")
            return s
        values, ids = logits.topk(top, dim=1)
        s["ids"], s["weights"] = ids.to(torch.int32), values.softmax(1)
        if case["padded"]:
            s["ids"][t - case["padded"]:] = -1
        h, i = case["hidden"], case["inter"]
        s["x"] = _activations(g, t, h, dtype)
        s["up"], s["down"] = _weights(g, e * 2 * i, h, case["group"]), _weights(g, e * h, i, case["group"])
        s["y"] = torch.empty((t, h), dtype=dtype, device="cuda")
        return s
    n = case["width"]
    s["x"], s["y"] = _activations(g, t, n, dtype), _activations(g, t, n, dtype)
    s["post"], s["next"] = ((1 + 0.1 * _normal(g, (n,))).to(dtype) if case[name] else None for name in ("post", "next"))
    s["gate"] = None if case["gate"] == "none" else (0.5 + 0.2 * _normal(g, (t, n) if case["gate"] == "token" else (n,))).to(dtype)
    s["a"], s["b"] = 1.0, 0.75
    s["x_out"], s["n_out"] = torch.empty_like(s["x"]), torch.empty_like(s["x"]) if case["next"] else None
    if op == "train":
        s["x_grad"] = (0.1 * _normal(g, (t, n))).to(dtype)
        s["n_grad"] = (0.1 * _normal(g, (t, n))).to(dtype) if case["next"] else None
        s["dx"], s["dy"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        s["dgate"] = {"none": lambda: None, "token": lambda: torch.empty_like(s["x"]),
                      "channel": lambda: torch.empty(n, device="cuda")}[case["gate"]]()
        s["dpost"], s["dnext"] = (torch.empty(n, device="cuda") if case[name] else None for name in ("post", "next"))
    return s


# ---- the plain forms --------------------------------------------------------------


def _weight(w, group, rows=slice(None)):
    """Rows of 4-bit weights in fp32, without their row scales."""
    codes, scales, _ = w
    word = codes[rows].contiguous().view(torch.int32)
    parts = [((word >> (4 * (e // 2) + 16 * (e % 2))) & 15) for e in range(8)]
    values = ((torch.stack(parts, -1) ^ 8) - 8).float().flatten(1)
    scale = scales[rows].view(torch.float8_e4m3fn).float()
    return (values.view(values.shape[0], -1, group) * scale[..., None]).view(values.shape)


def _plain_moe(s, case):
    h, i, group = case["hidden"], case["inter"], case["group"]
    y = torch.zeros((case["tokens"], h), device="cuda")
    x = s["x"].float()
    for e in range(case["experts"]):
        token, pick = torch.where(s["ids"] == e)
        if token.numel() == 0:
            continue
        r = slice(e * 2 * i, (e + 1) * 2 * i)
        gu = (x[token] @ _weight(s["up"], group, r).T) * s["up"][2][r]
        act = gu[:, 0::2]
        act = act / (1 + torch.exp(-act)) * gu[:, 1::2]
        r = slice(e * h, (e + 1) * h)
        out = (act @ _weight(s["down"], group, r).T) * s["down"][2][r]
        y.index_add_(0, token, out * s["weights"][token, pick][:, None])
    return y.to(s["x"].dtype)


def _plain_norm(s, case):
    dtype = s["x"].dtype
    x, y = s["x"].float(), s["y"].float()
    one = torch.ones((), device="cuda")
    post, nxt, gate = (s[k].float() if s[k] is not None else one for k in ("post", "next", "gate"))
    r1 = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) if case["post"] else one
    yhat = y * r1
    z = yhat * post
    new = s["a"] * x + s["b"] * gate * z
    outs = {"x": new.to(dtype)}
    r2 = torch.rsqrt((new * new).mean(-1, keepdim=True) + EPS)
    xhat = new * r2
    if case["next"]:
        outs["n"] = (xhat * nxt).to(dtype)
    if case["op"] == "norm":
        return outs
    d = s["x_grad"].float()
    if case["next"]:
        dn = s["n_grad"].float()
        outs["dnext"] = (dn * xhat).sum(0)
        dn = dn * nxt
        d = d + r2 * (dn - xhat * (dn * xhat).mean(-1, keepdim=True))
    outs["dx"] = (s["a"] * d).to(dtype)
    d = s["b"] * d
    if case["gate"] != "none":
        dg = d * z
        outs["dgate"] = dg.to(dtype) if case["gate"] == "token" else dg.sum(0)
        d = d * gate
    if case["post"]:
        outs["dpost"] = (d * yhat).sum(0)
        d = d * post
        d = r1 * (d - yhat * (d * yhat).mean(-1, keepdim=True))
    outs["dy"] = d.to(dtype)
    return outs


def run(s):
    case = s["case"]
    if own:
        return _run_own(s, case)
    if case["op"] == "linear":
        return ((s["x"].float() @ _weight(s["w"], case["group"]).T) * s["w"][2]).to(s["x"].dtype)
    if case["op"] == "route":
        values, order = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True)
        top, ids = values[:, :case["top"]], order[:, :case["top"]]
        none = top == -math.inf
        first = torch.where(none[:, :1], 0.0, top[:, :1])
        p = torch.exp(top - first)
        total = p if case["renormalize"] else torch.exp(values - first)
        total = total.sum(1, keepdim=True)
        return torch.where(none, -1, ids).to(torch.int32), p / torch.where(total > 0, total, 1.0)
    if case["op"] == "moe":
        return _plain_moe(s, case)
    return _plain_norm(s, case)


# ---- the library's calls ------------------------------------------------------------


def _run_own(s, case):
    from bit_tensor_gemm_gb300 import lbgemm as L
    kind, stream, t = {"bf16": L.BF16, "fp16": L.F16, "fp32": L.F32}[case["dtype"]], s["stream"], case["tokens"]
    if case["op"] == "linear":
        L.lbgemm_w4_linear(kind, t, case["rows"], case["k"], case["group"], s["x"], case["k"], *s["w"], s["y"], case["rows"], stream)
        return s["y"]
    if case["op"] == "route":
        L.lbgemm_moe_route(kind, t, case["experts"], case["top"], s["logits"], case["experts"], case["renormalize"], s["ids"],
                           s["weights"], stream)
        return s["ids"], s["weights"]
    if case["op"] == "moe":
        h = case["hidden"]
        L.lbgemm_moe_w4(kind, t, h, case["inter"], case["experts"], case["top"], case["group"], s["x"], h, s["ids"], s["weights"],
                        *s["up"], *s["down"], s["y"], h, stream)
        return s["y"]
    n = case["width"]
    gate_stride = n if case["gate"] == "token" else 0
    given = (s["x"], n, s["y"], n, s["post"], s["gate"], gate_stride, s["a"], s["b"], s["next"], EPS)
    L.lbgemm_residual_norm(kind, t, n, *given, s["x_out"], n, s["n_out"], n, stream)
    outs = {"x": s["x_out"]}
    if case["next"]:
        outs["n"] = s["n_out"]
    if case["op"] == "train":
        L.lbgemm_residual_norm_backward(kind, t, n, s["x_grad"], n, s["n_grad"], n, *given, s["dx"], n, s["dy"], n, s["dgate"],
                                        gate_stride, s["dpost"], s["dnext"], stream)
        outs.update({"dnext": s["dnext"]} if case["next"] else {})
        outs["dx"] = s["dx"]
        outs.update({"dgate": s["dgate"]} if case["gate"] != "none" else {})
        outs.update({"dpost": s["dpost"]} if case["post"] else {})
        outs["dy"] = s["dy"]
    return outs


# ---- the definitions in fp64 ----------------------------------------------------------

VALUES = [0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1]


def _exact_weight(w, group, a, b):
    codes, scales, row = (z[a:b] for z in w)
    table = torch.tensor(VALUES, dtype=torch.float64, device="cuda")
    low, high = table[(codes % 16).long()], table[(codes // 16).long()]
    nibbles = torch.stack((low, high), -1).view(b - a, -1, 2, 4)  # [word][half of it][nibble]
    dense = nibbles.transpose(2, 3).reshape(b - a, -1)
    exponent, digits = (scales.long() >> 3) & 15, (scales & 7).double()
    size = torch.where(exponent > 0, (1 + digits / 8) * torch.exp2(exponent.double() - 7), digits * 2.0 ** -9)
    size = torch.where(scales >= 128, -size, size)
    return dense * size.repeat_interleave(group, 1) * row[:, None].double()


def exact(case, seed):
    if case["op"] in ("linear", "moe") and work(case)["flops"] > 2e12:
        return None
    s = prepare(case, seed)
    t = case["tokens"]
    if case["op"] == "linear":
        x, n = s["x"].double(), case["rows"]
        y = torch.empty((t, n), dtype=torch.float64, device="cuda")
        for a in range(0, n, 2048):
            b = min(n, a + 2048)
            y[:, a:b] = x @ _exact_weight(s["w"], case["group"], a, b).T
        return y
    if case["op"] == "route":
        left = s["logits"].double().clone()
        row = torch.arange(t, device="cuda")
        ids = torch.empty((t, case["top"]), dtype=torch.int32, device="cuda")
        chosen = torch.empty((t, case["top"]), dtype=torch.float64, device="cuda")
        place = torch.arange(case["experts"], device="cuda")
        for j in range(case["top"]):
            best = left.max(1).values
            at = torch.where(left == best[:, None], place, case["experts"]).min(1).values
            ids[:, j] = torch.where(best == -math.inf, -1, at)
            chosen[:, j] = best
            left[row, at] = -math.inf
        among = chosen if case["renormalize"] else s["logits"].double()
        weights = torch.exp(chosen - torch.logsumexp(among, 1, keepdim=True))
        return ids, torch.where(ids < 0, 0.0, weights)
    if case["op"] == "moe":
        h, i = case["hidden"], case["inter"]
        y = torch.zeros((t, h), dtype=torch.float64, device="cuda")
        for e in sorted(set(s["ids"].flatten().tolist()) - {-1}):
            weight = (s["weights"].double() * (s["ids"] == e)).sum(1)
            who = (s["ids"] == e).any(1).nonzero()[:, 0]
            both = (s["x"][who].double() @ _exact_weight(s["up"], case["group"], 2 * i * e, 2 * i * (e + 1)).T).view(-1, i, 2)
            inner = both[..., 0] * torch.sigmoid(both[..., 0]) * both[..., 1]
            y[who] += weight[who][:, None] * (inner @ _exact_weight(s["down"], case["group"], h * e, h * (e + 1)).T)
        return y

    train = case["op"] == "train"
    leaf = {k: s[k].double().requires_grad_(train) for k in ("x", "y", "post", "gate", "next") if s[k] is not None}

    def norm(v, w):
        return v / torch.sqrt((v ** 2).mean(1, keepdim=True) + EPS) * w

    z = norm(leaf["y"], leaf["post"]) if case["post"] else leaf["y"]
    new = s["a"] * leaf["x"] + s["b"] * (z * leaf["gate"] if "gate" in leaf else z)
    outs, loss = {"x": new.detach()}, 0
    if case["next"]:
        n = norm(new, leaf["next"])
        outs["n"] = n.detach()
    if train:
        loss = (new * s["x_grad"].double()).sum()
        if case["next"]:
            loss = loss + (n * s["n_grad"].double()).sum()
        got = dict(zip(leaf, torch.autograd.grad(loss, list(leaf.values()))))
        for name in ("next", "x", "gate", "post", "y"):
            if name in got:
                outs["d" + name] = got[name]
    return outs
