"""Cases of the prompt's step: products in microscaled 4-bit floating point and attention over whole prompts.

A prompt brings hundreds or thousands of tokens at once, before the decode and
verification steps.  These cases measure the library's operators for that:
quantizing to the microscaled format and reading it back (``quantize``),
products of many tokens or of a few with weights in that format
(``product``), and attention of packed sequences over their own 16-bit keys
and values (``prompt``).

``own`` selects what ``run`` computes with: the plain form below in
elementary torch operations, or the package's entry points.
"""

import math
import random

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # the activations of one decoded token of a 7B-shaped layer: the smallest call
        {"name": "quantize_one", "op": "quantize", "rows": 1, "cols": 4096, "wide": 4096, "dtype": F16},
        # a weight of a 13B-shaped layer, when the model is loaded
        {"name": "quantize_weight13b", "op": "quantize", "rows": 13824, "cols": 5120, "wide": 5120, "dtype": BF16},
        # the activations of a prompt, one half of a fused gate/up product
        {"name": "quantize_prompt7b", "op": "quantize", "rows": 4093, "cols": 11008, "wide": 22016, "dtype": F16},
        # one decoded token of a 7B-shaped projection: latency and the weight's bytes
        {"name": "product_one", "op": "product", "tokens": 1, "rows": 4096, "cols": 4096, "dtype": F16,
         "quantized": False, "out": F16},
        # 16 candidate tokens of a 13B-shaped up projection
        {"name": "product_verify13b", "op": "product", "tokens": 16, "rows": 13824, "cols": 5120, "dtype": BF16,
         "quantized": False, "out": BF16},
        # the last tokens of a few requests against an odd vocabulary, logits in fp32
        {"name": "product_vocab", "op": "product", "tokens": 37, "rows": 50257, "cols": 4096, "dtype": BF16,
         "quantized": True, "out": F32},
        # one short prompt, 7B-shaped gate projection
        {"name": "product_short7b", "op": "product", "tokens": 509, "rows": 11008, "cols": 4096, "dtype": F16,
         "quantized": False, "out": F16},
        # a long prompt, 13B-shaped up projection, activations quantized once for several products
        {"name": "product_prompt13b", "op": "product", "tokens": 8191, "rows": 13824, "cols": 5120, "dtype": BF16,
         "quantized": True, "out": BF16},
        # one short prompt: latency
        {"name": "prompt_short", "op": "prompt", "n": 1, "len": 61, "past": 0, "spread": False, "heads": 8, "share": 4,
         "dim": 128, "dtype": F16, "causal": True, "fused": True},
        # a batch of prompts of different lengths, grouped heads, sliced out of the fused q/k/v product
        {"name": "prompt_packed16", "op": "prompt", "n": 16, "len": 2047, "past": 0, "spread": True, "heads": 8,
         "share": 4, "dim": 128, "dtype": F16, "causal": True, "fused": True},
        # one long prompt of a 13B-shaped layer (40 heads of 128)
        {"name": "prompt_long13b", "op": "prompt", "n": 1, "len": 8191, "past": 0, "spread": False, "heads": 40,
         "share": 1, "dim": 128, "dtype": BF16, "causal": True, "fused": False},
        # the last token of one long context that is still held in 16 bits
        {"name": "prompt_token", "op": "prompt", "n": 1, "len": 1, "past": 65535, "spread": False, "heads": 8,
         "share": 4, "dim": 128, "dtype": BF16, "causal": True, "fused": False},
    ]


_MOST_PRODUCT = 8191 * 13824 * 5120 // 2
_MOST_PAIRS = 8191 * 8191 * 40 // 3


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quantize", "product", "product", "prompt", "prompt"))
    if op == "quantize":
        cols = 32 * _log_int(rng, 1, 432)
        return {"op": op, "rows": _log_int(rng, 1, 13824 * 5120 // cols // 2), "cols": cols,
                "wide": cols + 8 * rng.choice((0, 0, 1, cols // 8)), "dtype": rng.choice((F16, BF16))}
    if op == "product":
        tokens, rows, cols = _log_int(rng, 1, 8191), _log_int(rng, 16, 50257), 32 * _log_int(rng, 2, 432)
        while tokens * rows * cols > _MOST_PRODUCT:
            tokens = max(1, tokens // 2)
        dtype = rng.choice((F16, BF16))
        return {"op": op, "tokens": tokens, "rows": rows, "cols": cols, "dtype": dtype,
                "quantized": rng.random() < 0.5, "out": rng.choice((dtype, dtype, F32))}
    dim = rng.choice((64, 128, 128, 256))
    heads, share = rng.choice((1, 2, 4, 5, 8, 8, 16, 40)), rng.choice((1, 1, 2, 4, 5, 7, 8))
    n = _log_int(rng, 1, 32)
    length, past = _log_int(rng, 1, 8191), rng.choice((0, 0, 1, _log_int(rng, 1, 65535)))
    while n * heads * share * length * (length + past) * dim > _MOST_PAIRS * 128:
        length, past = max(1, length // 2), past // 2
    return {"op": op, "n": n, "len": length, "past": past, "spread": rng.random() < 0.7, "heads": heads,
            "share": share, "dim": dim, "dtype": rng.choice((F16, BF16)), "causal": rng.random() < 0.8,
            "fused": past == 0 and rng.random() < 0.5}


# ---------------------------------------------------------------------------
# sizes that follow from the case alone


def _lengths(c):
    """(query tokens, keys) of every sequence."""
    rng = random.Random("%d %d %d" % (c["n"], c["len"], c["past"]))
    q, k = [c["len"]], [c["len"] + c["past"]]
    for _ in range(c["n"] - 1):
        q.append(rng.randint(0, c["len"]) if c["spread"] else c["len"])
        k.append(q[-1] + (rng.randint(0, c["past"]) if c["spread"] else c["past"]))
    return q, k


def _mx_bytes(rows, cols):
    return rows * (cols // 2 + cols // 32)


def work(case):
    c, op = case, case["op"]
    if op == "quantize":
        values = c["rows"] * c["cols"]
        # values read, format written and read, values written
        return {"bytes": 4 * values + 2 * _mx_bytes(c["rows"], c["cols"]), "flops": 2 * values}
    if op == "product":
        t, n, k = c["tokens"], c["rows"], c["cols"]
        x = _mx_bytes(t, k) if c["quantized"] else 2 * t * k
        return {"bytes": x + _mx_bytes(n, k) + t * n * (4 if c["out"] == F32 else 2), "flops": 2 * t * n * k}
    q, k = _lengths(c)
    pairs = sum(m * l - (m * (m - 1) // 2 if c["causal"] else 0) for m, l in zip(q, k))
    rows = sum(q) * c["heads"] * c["share"]
    return {"bytes": 4 * rows * c["dim"] + 4 * rows + 4 * sum(k) * c["heads"] * c["dim"],
            "flops": 4 * pairs * c["heads"] * c["share"] * c["dim"]}


# ---------------------------------------------------------------------------
# the microscaled format


def _quantize(x):
    """(codes 0..15, scale bytes) of [rows, cols] values, a scale for 32 columns."""
    x = x.float().unflatten(1, (-1, 32))
    top = x.abs().amax(-1)
    e = (torch.frexp(top).exponent - 3).clamp(min=-127)
    e = torch.where(top > 0, e, -127)
    y = torch.ldexp(x.abs(), -e.unsqueeze(-1))
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6.0)
    code = torch.where(y < 2, 2 * y, torch.where(y < 4, y + 2, y / 2 + 4)).to(torch.uint8)
    return (code | (torch.signbit(x).to(torch.uint8) << 3)).flatten(1), (e + 127).to(torch.uint8)


def _pack(code, scale):
    """The format's two buffers: 16 rows x 128 columns of values lie together, and 16 rows x 512 columns of scales."""
    rows, cols = code.shape
    code = torch.nn.functional.pad(code, (0, -cols % 256, 0, -rows % 16))
    code = code.unflatten(0, (-1, 16)).unflatten(2, (-1, 4, 16, 2)).permute(0, 2, 3, 1, 4, 5)
    scale = torch.nn.functional.pad(scale, (0, -(cols // 32) % 16, 0, -rows % 16))
    scale = scale.unflatten(0, (-1, 16)).unflatten(2, (-1, 4, 4)).permute(0, 2, 4, 1, 3)
    return (code[..., 0] | (code[..., 1] << 4)).flatten(2), scale.flatten(2).contiguous()


def _unpack(vals, scales, rows, cols):
    """[rows, cols] values in fp32."""
    code = torch.stack((vals & 15, vals >> 4), -1).flatten(2).unflatten(2, (4, 16, 32)).permute(0, 3, 1, 2, 4)
    code = code.flatten(2).flatten(0, 1)[:rows, :cols].int()
    scale = scales.unflatten(2, (4, 16, 4)).permute(0, 3, 1, 4, 2).flatten(2).flatten(0, 1)[:rows, :cols // 32]
    size = code & 7
    y = torch.where(size < 4, 0.5 * size, torch.where(size < 6, size - 2.0, 2.0 * size - 8.0))
    y = torch.where(code > 7, -y, y).unflatten(1, (-1, 32))
    return torch.ldexp(y, (scale.int() - 127).unsqueeze(-1)).flatten(1)


# ---------------------------------------------------------------------------
# inputs


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return {"quantize": _prepare_quantize, "product": _prepare_product, "prompt": _prepare_prompt}[case["op"]](case, g)


def _activations(rows, cols, g):
    """Activations: some channels are much stronger than others."""
    return torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(
        0.7 * torch.randn(cols, generator=g, device="cuda"))


def _prepare_quantize(c, g):
    wide = _activations(c["rows"], c["wide"], g).to(getattr(torch, c["dtype"]))
    return {"op": "quantize", "x": wide[:, c["wide"] - c["cols"]:]}


def _prepare_product(c, g):
    w = _pack(*_quantize(0.02 * torch.randn(c["rows"], c["cols"], generator=g, device="cuda")))
    x = _activations(c["tokens"], c["cols"], g).to(getattr(torch, c["dtype"]))
    return {"op": "product", "x": _pack(*_quantize(x)) if c["quantized"] else x, "quantized": c["quantized"], "w": w,
            "tokens": c["tokens"], "rows": c["rows"], "cols": c["cols"], "out": getattr(torch, c["out"])}


def _starts(lengths):
    at = [0]
    for m in lengths:
        at.append(at[-1] + m)
    return torch.tensor(at, dtype=torch.int32).cuda()


def _prepare_prompt(c, g):
    q_len, k_len = _lengths(c)
    dtype, h, d = getattr(torch, c["dtype"]), c["heads"], c["dim"]
    many, tokens, keys = h * c["share"], sum(q_len), sum(k_len)
    if c["fused"]:  # slices of one q/k/v product
        qkv = torch.randn(tokens, (many + 2 * h) * d, generator=g, device="cuda").to(dtype)
        q, k, v = (x.unflatten(1, (-1, d)) for x in qkv.split((many * d, h * d, h * d), 1))
    else:
        q = torch.randn(tokens, many, d, generator=g, device="cuda").to(dtype)
        k, v = (torch.randn(keys, h, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k *= torch.exp(0.5 * torch.randn(h, d, generator=g, device="cuda")).to(dtype)  # keys have strong channels
    return {"op": "prompt", "q": q, "k": k, "v": v, "q_start": _starts(q_len), "k_start": _starts(k_len),
            "max_q": max(q_len), "max_k": max(k_len), "causal": c["causal"], "scale": d ** -0.5, "share": c["share"]}


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return {"quantize": _run_quantize, "product": _run_product, "prompt": _run_prompt}[state["op"]](state)


def _run_quantize(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        return i4s.mx_read(i4s.mx_quantize(s["x"]), dtype=s["x"].dtype)
    return _unpack(*_pack(*_quantize(s["x"])), *s["x"].shape).to(s["x"].dtype)


def _run_product(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        if "weight" not in s:  # the handles a program makes once, next to their buffers
            s["weight"] = i4s.MXTensor(s["rows"], s["cols"], *s["w"])
            if s["quantized"]:
                s["input"] = i4s.MXTensor(s["tokens"], s["cols"], *s["x"])
        return i4s.mx_product(s["input"] if s["quantized"] else s["x"], s["weight"], dtype=s["out"])
    x = _unpack(*(s["x"] if s["quantized"] else _pack(*_quantize(s["x"]))), s["tokens"], s["cols"])
    return (x @ _unpack(*s["w"], s["rows"], s["cols"]).t()).to(s["out"])


def _run_prompt(s):
    q, k, v = s["q"], s["k"], s["v"]
    if own:
        import int4_sparse_gemv_amd as i4s
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device="cuda")
        out = i4s.prompt_attention(q, k, v, s["q_start"], s["k_start"], max_q=s["max_q"], max_k=s["max_k"],
                                   causal=s["causal"], scale=s["scale"], lse=lse)
        return out, lse
    most, wide, share, heads = s["max_q"], s["max_k"], s["share"], k.shape[1]
    q_start, k_start = s["q_start"].long(), s["k_start"].long()
    q_len, k_len = q_start.diff(), k_start.diff()
    t, key = torch.arange(most, device="cuda"), torch.arange(wide, device="cuda")
    rows = (q_start[:-1, None] + t).clamp(max=q.shape[0] - 1)
    keys = (k_start[:-1, None] + key).clamp(max=k.shape[0] - 1)
    kk, vv = (x.float()[keys].movedim(1, 2) for x in (k, v))  # [n, heads, keys, dim]
    qq = q.float()[rows].unflatten(2, (heads, share)).movedim(1, 3).flatten(2, 3)  # [n, heads, share * most, dim]
    x = (qq @ kk.transpose(-1, -2)).unflatten(2, (share, most)) * s["scale"]
    seen = (key < k_len[:, None, None]).expand(-1, most, -1)
    if s["causal"]:
        seen = seen & (key <= (k_len - q_len)[:, None, None] + t[:, None])
    x = torch.where(seen[:, None, None], x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = torch.exp(x - m)
    l = x.sum(-1, keepdim=True)
    o = (x.flatten(2, 3) @ vv).unflatten(2, (share, most)) / torch.where(l > 0, l, 1)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0]
    mine = t < q_len[:, None]  # rows that a sequence has
    return (o.permute(0, 3, 1, 2, 4).flatten(2, 3)[mine].to(q.dtype), lse.permute(0, 3, 1, 2).flatten(2, 3)[mine])


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    with torch.no_grad():
        return {"quantize": _exact_quantize, "product": _exact_product, "prompt": _exact_prompt}[case["op"]](case, seed)


_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_rounded(x):
    """The values that the format holds for [rows, cols] values, from distances to every value of the grid."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    rows = max(1, (1 << 24) // x.shape[1])
    for at in range(0, x.shape[0], rows):
        y = x[at:at + rows].double().reshape(-1, 32)
        top = y.abs().max(1, keepdim=True).values
        unit = torch.where(top > 0, 2.0 ** (torch.floor(torch.log2(top)) - 2).clamp(min=-127), 2.0 ** -127)
        y = y / unit
        best, where = torch.full_like(y, math.inf), torch.zeros_like(y)
        for i in (0, 2, 4, 6, 1, 3, 5, 7):  # of two that are as near the even one stays
            far = (y.abs() - _GRID[i]).abs()
            where = torch.where(far < best, _GRID[i], where)
            best = torch.minimum(best, far)
        out[at:at + rows] = (torch.copysign(where, y) * unit).reshape(-1, x.shape[1])
    return out


def _exact_held(vals, scales, rows, cols):
    """The values at each place of the format's buffers."""
    row, col = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")
    lane = col % 128 // 32 * 16 + row % 16
    byte = vals[row // 16, col // 128, lane * 16 + col % 32 // 2]
    code = (byte >> (4 * (col % 2)).to(torch.uint8)) & 15
    unit = scales[row // 16, col // 512, lane * 4 + col % 512 // 128]
    grid = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device="cuda")
    return grid[code.long()] * 2.0 ** (unit.double() - 127)


def _exact_quantize(c, seed):
    return _exact_rounded(prepare(c, seed)["x"])


def _exact_product(c, seed):
    s = prepare(c, seed)
    x = _exact_held(*s["x"], c["tokens"], c["cols"]) if c["quantized"] else _exact_rounded(s["x"])
    parts = []
    step = max(1, (1 << 26) // c["cols"])
    for at in range(0, c["rows"], step - step % 16 if step > 16 else 16):
        n = min(step - step % 16 if step > 16 else 16, c["rows"] - at)
        w = _exact_held(s["w"][0][at // 16:], s["w"][1][at // 16:], n, c["cols"])
        parts.append(torch.mm(x, w.t().contiguous()))
    return torch.cat(parts, 1)


def _exact_prompt(c, seed):
    s = prepare(c, seed)
    q_start, k_start = s["q_start"].tolist(), s["k_start"].tolist()
    outs, lses = [], []
    for i in range(c["n"]):
        q = s["q"][q_start[i]:q_start[i + 1]].double()
        k, v = (s[x][k_start[i]:k_start[i + 1]].double() for x in ("k", "v"))
        n_q, n_k = q.shape[0], k.shape[0]
        o, e = torch.empty_like(q), torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
        hidden = torch.ones(n_q, n_k, dtype=torch.bool, device="cuda").triu(n_k - n_q + 1)
        for h in range(q.shape[1]):
            x = torch.mm(q[:, h].contiguous(), k[:, h // c["share"]].t().contiguous()) * s["scale"]
            if c["causal"]:
                x = x.masked_fill_(hidden, -math.inf)
            e[:, h] = torch.logsumexp(x, 1)
            o[:, h] = torch.mm(torch.exp(x.sub_(e[:, h, None])), v[:, h // c["share"]].contiguous())
        outs.append(o)
        lses.append(e)
    return torch.cat(outs), torch.cat(lses)
