"""Cases of the decode and verification step around the packed products.

Between two INT4 products a decoder step attends over its KV cache, and after
the last one it scores the tokens it verified.  These cases measure the
library's operators for that: block tables and slot maps from request lengths
(``extend``), writing tokens into the 4-bit paged cache and reading them back
(``append``), attention over that cache (``attend``) and the log
probabilities of given tokens (``score``).

``own`` selects what ``run`` computes with: the plain form below in
elementary torch operations, or the package's entry points.
"""

import math
import random

import torch

own = False

F16, BF16, F32 = "float16", "bfloat16", "float32"
_SLOT_ELEMENT = (0, 2, 4, 6, 1, 3, 5, 7)  # element held by nibble slot k of a K word
_SCALE_MAX = 9352.0                       # largest fp16 scale whose 7-fold is finite in fp16


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one decode step of a full batch of 16 requests: the smallest call
        {"name": "extend_decode16", "op": "extend", "n": 16, "page": 16, "width": 256, "held": 4000, "new": 1,
         "mix": "same", "pad": 0},
        # admission of a mixed batch: long prompts, short ones, requests that add nothing
        {"name": "extend_mixed512", "op": "extend", "n": 512, "page": 32, "width": 512, "held": 9000, "new": 700,
         "mix": "ragged", "pad": 1237},
        # 16 new tokens of a 7B-shaped layer (32 heads of 128)
        {"name": "append_decode16", "op": "append", "tokens": 16, "heads": 32, "dim": 128, "group": 64, "page": 16,
         "dtype": F16, "fused": True},
        # a long prompt of a 13B-shaped layer (40 heads of 128), sliced out of the fused q/k/v product
        {"name": "append_prompt13b", "op": "append", "tokens": 8191, "heads": 40, "dim": 128, "group": 64, "page": 64,
         "dtype": BF16, "fused": True},
        # one request, one token, a short context: latency
        {"name": "attend_one", "op": "attend", "n": 1, "len": 1023, "spread": False, "q": 1, "heads": 32, "share": 1,
         "dim": 128, "group": 64, "page": 16, "dtype": F16, "tree": False},
        # decode of 16 requests of different lengths, 7B shape
        {"name": "attend_decode16", "op": "attend", "n": 16, "len": 4095, "spread": True, "q": 1, "heads": 32,
         "share": 1, "dim": 128, "group": 64, "page": 16, "dtype": F16, "tree": False},
        # tree verification: 16 candidate tokens of one request, 13B shape
        {"name": "attend_verify13b", "op": "attend", "n": 1, "len": 2047, "spread": False, "q": 16, "heads": 40,
         "share": 1, "dim": 128, "group": 128, "page": 32, "dtype": F16, "tree": True},
        # one long context, grouped query heads
        {"name": "attend_long", "op": "attend", "n": 1, "len": 131071, "spread": False, "q": 1, "heads": 8, "share": 4,
         "dim": 128, "group": 64, "page": 64, "dtype": BF16, "tree": False},
        # a large serving batch, grouped query heads, a few candidate tokens each
        {"name": "attend_batch64", "op": "attend", "n": 64, "len": 16384, "spread": True, "q": 4, "heads": 8,
         "share": 8, "dim": 128, "group": 32, "page": 128, "dtype": BF16, "tree": False},
        # the scores of one decoded token
        {"name": "score_one", "op": "score", "rows": 1, "vocab": 32000, "top": 5, "dtype": F16},
        # the scores of a verification batch over a large vocabulary
        {"name": "score_verify16", "op": "score", "rows": 16, "vocab": 151643, "top": 20, "dtype": F32},
        # the scores of a long text, odd vocabulary
        {"name": "score_text", "op": "score", "rows": 4093, "vocab": 50257, "top": 8, "dtype": BF16},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("extend", "append", "attend", "attend", "score"))
    if op == "extend":
        n = _log_int(rng, 1, 1000)
        new = _log_int(rng, 1, 700)
        page = rng.choice((16, 32, 64, 128))
        held = _log_int(rng, 16, 9000)
        return {"op": op, "n": n, "page": page, "width": -(-(held + new) // page) + rng.randint(0, 9), "held": held,
                "new": new, "mix": rng.choice(("same", "ragged")), "pad": rng.choice((0, rng.randint(1, 2000)))}
    if op == "append":
        dim = rng.choice((64, 128, 128, 256))
        heads = rng.randint(1, 40)
        tokens = _log_int(rng, 1, max(2, 8191 * 40 * 128 // (heads * dim) // 4))
        return {"op": op, "tokens": tokens, "heads": heads, "dim": dim,
                "group": rng.choice([g for g in (32, 64, 128) if g <= dim]), "page": rng.choice((16, 32, 64, 128, 256)),
                "dtype": rng.choice((F16, BF16)), "fused": rng.random() < 0.5}
    if op == "attend":
        dim = rng.choice((64, 128, 128, 256))
        heads = rng.choice((1, 2, 4, 5, 8, 8, 16, 32, 40))
        share = rng.choice((1, 1, 2, 4, 5, 7, 8))
        n = _log_int(rng, 1, 64)
        longest = min(131072, 64 * 16384 * 8 * 128 // (n * heads * dim) // 2)
        return {"op": op, "n": n, "len": _log_int(rng, 20, longest), "spread": rng.random() < 0.7,
                "q": rng.choice((1, 1, 1, 2, 3, 5, 8, 16)), "heads": heads, "share": share, "dim": dim,
                "group": rng.choice([g for g in (32, 64, 128) if g <= dim]), "page": rng.choice((16, 32, 64, 128, 256)),
                "dtype": rng.choice((F16, BF16)), "tree": rng.random() < 0.4}
    rows = _log_int(rng, 1, 2000)
    return {"op": op, "rows": rows, "vocab": _log_int(rng, 1000, min(260000, 100_000_000 // rows)),
            "top": rng.choice((0, 1, 5, 10, 20, 32)), "dtype": rng.choice((F16, BF16, F32))}


# ---------------------------------------------------------------------------
# sizes that follow from the case alone


def _attend_lengths(c):
    """(tokens held with the new ones, new tokens) of every request."""
    rng = random.Random("%d %d %d" % (c["n"], c["len"], c["q"]))
    lens, q = [c["len"]], [min(c["q"], c["len"])]
    for _ in range(c["n"] - 1):
        lens.append(rng.randint(max(1, c["len"] // 8), c["len"]) if c["spread"] else c["len"])
        q.append(min(lens[-1], rng.randint(1, c["q"]) if c["spread"] else c["q"]))
    return lens, q


def _extend_lengths(c):
    rng = random.Random("%d %d %d" % (c["n"], c["held"], c["new"]))
    if c["mix"] == "same":
        return [rng.randint(0, c["held"]) for _ in range(c["n"])], [c["new"]] * c["n"]
    kinds = [rng.choice((0, 0, 1, 2, 3)) for _ in range(c["n"])]
    held = [0 if k == 3 else rng.randint(0, c["held"]) for k in kinds]
    new = [0 if k == 2 else (1 if k == 0 else rng.randint(1, c["new"])) for k in kinds]
    return held, new


def work(case):
    c, op = case, case["op"]
    if op == "extend":
        held, new = _extend_lengths(c)
        pages = sum(-(-(h + m) // c["page"]) - -(-h // c["page"]) for h, m in zip(held, new))
        # lengths read; lengths, starts, slots, positions written; new pages read and written
        return {"bytes": 16 * c["n"] + 8 * (sum(new) + c["pad"]) + 8 * pages, "flops": 0}
    if op == "append":
        values = 2 * c["tokens"] * c["heads"] * c["dim"]
        packed = values // 2 + 2 * values // c["group"]
        # values read, packed and written, then read and unpacked
        return {"bytes": 2 * values + 2 * packed + 2 * values, "flops": 2 * values}
    if op == "attend":
        lens, q = _attend_lengths(c)
        per_key = c["heads"] * (c["dim"] + 4 * c["dim"] // c["group"])
        rows = [m * c["heads"] * c["share"] for m in q]
        return {"bytes": sum(lens) * per_key + 4 * sum(rows) * c["dim"] + 4 * sum(rows),
                "flops": sum(4 * r * l * c["dim"] for r, l in zip(rows, lens))}
    size = 4 if c["dtype"] == F32 else 2
    return {"bytes": c["rows"] * (c["vocab"] * size + 16 + 8 * c["top"]), "flops": 6 * c["rows"] * c["vocab"]}


# ---------------------------------------------------------------------------
# the cache format


def _pack_k(q):
    """[..., D] whole numbers -7..7 -> [..., D/2] bytes of K rows."""
    d = q.shape[-1]
    u = (q + 8).to(torch.uint8).unflatten(-1, (d // 32, 4, 8))[..., list(_SLOT_ELEMENT)].transpose(-3, -2)
    return (u[..., 0::2] | (u[..., 1::2] << 4)).flatten(-3)


def _unpack_k(b):
    d = 2 * b.shape[-1]
    u = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (4, d // 32, 8)).transpose(-3, -2)
    return u[..., [_SLOT_ELEMENT.index(e) for e in range(8)]].flatten(-3).float() - 8


def _pack_v(q):
    """[..., D] whole numbers -7..7 -> [..., D/8, 4] bytes: the words of one token."""
    d = q.shape[-1]
    u = (q + 8).to(torch.uint8).unflatten(-1, (d // 64, 4, 16)).movedim(-1, -3)
    return (u[..., 0::2] | (u[..., 1::2] << 4)).flatten(-3).unflatten(-1, (d // 8, 4))


def _unpack_v(b):
    d = 8 * b.shape[-2]
    u = torch.stack((b & 15, b >> 4), -1).flatten(-3).unflatten(-1, (16, d // 64, 4)).movedim(-3, -1)
    return u.flatten(-3).float() - 8


def _quantize(x, group):
    """(whole numbers, fp16 scales) of [..., D] values."""
    x = x.float().unflatten(-1, (-1, group))
    s = (x.abs().amax(-1) / 7).clamp(max=_SCALE_MAX).half()
    f = s.float().unsqueeze(-1)
    q = torch.where(f > 0, torch.round(x / f), torch.zeros_like(x)).clamp(-7, 7)
    return q.flatten(-2), s


def _empty_cache(c, pages):
    h, p, d, g = c["heads"], c["page"], c["dim"], c["group"]
    byte = dict(dtype=torch.uint8, device="cuda")
    return {"page": p, "heads": h, "dim": d, "group": g,
            "k_vals": torch.full((pages, h, p * d // 2), 0x88, **byte),
            "v_vals": torch.full((pages, h, p * d // 2), 0x88, **byte),
            "k_scales": torch.zeros(pages, h, p * d // g, dtype=torch.float16, device="cuda"),
            "v_scales": torch.zeros(pages, h, p * d // g, dtype=torch.float16, device="cuda")}


def _views(cache):
    """The four buffers with an axis for everything: [pages, heads, P/4, ...]."""
    p, d, g = cache["page"], cache["dim"], cache["group"]
    return (cache["k_vals"].unflatten(-1, (p // 4, 4, d // 2)), cache["v_vals"].unflatten(-1, (p // 4, d // 8, 4, 4)),
            cache["k_scales"].unflatten(-1, (p // 4, d // g, 4)), cache["v_scales"].unflatten(-1, (p // 4, d // g, 4)))


# ---------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    return {"extend": _prepare_extend, "append": _prepare_append, "attend": _prepare_attend,
            "score": _prepare_score}[case["op"]](case, seed)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32).cuda()


def _prepare_extend(c, seed):
    g = _generator(seed)
    held, new = _extend_lengths(c)
    total = sum(-(-(h + m) // c["page"]) for h, m in zip(held, new))
    pages = torch.randperm(total + 64, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((c["n"], c["width"]), -1, dtype=torch.int32, device="cuda")
    old = torch.tensor([-(-h // c["page"]) for h in held]).cuda()
    inside = torch.arange(c["width"], device="cuda") < old[:, None]
    used = int(old.sum())
    table[inside] = pages[:used]
    return {"op": "extend", "page": c["page"], "table": table, "lens": _int32(held), "new": _int32(new),
            "free": pages[used:].clone(), "count": _int32([total + 64 - used]), "capacity": sum(new) + c["pad"]}


def _prepare_append(c, seed):
    g = _generator(seed)
    t, h, d = c["tokens"], c["heads"], c["dim"]
    dtype = getattr(torch, c["dtype"])
    if c["fused"]:  # k and v are slices of one q/k/v product
        qkv = torch.randn(t, 3 * h * d, generator=g, device="cuda").to(dtype)
        k, v = qkv[:, h * d:2 * h * d].unflatten(1, (h, d)), qkv[:, 2 * h * d:].unflatten(1, (h, d))
    else:
        k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k *= torch.exp(0.7 * torch.randn(h, d, generator=g, device="cuda")).to(dtype)  # keys have strong channels
    pages = -(-t // c["page"]) + 3
    order = torch.randperm(pages, generator=g, device="cuda")
    at = torch.arange(t, device="cuda") + 5  # the first page is partly held already
    slots = (order[at // c["page"]] * c["page"] + at % c["page"]).int()
    return {"op": "append", "cache": _empty_cache(c, pages), "k": k, "v": v, "slots": slots}


def _tree_masks(q, rng):
    """Ancestor bits of the candidates of every request: node t hangs off an earlier node."""
    masks = []
    for m in q:
        own_bits = []
        for t in range(m):
            up = rng.randrange(-1, t) if t else -1
            own_bits.append((own_bits[up] if up >= 0 else 0) | 1 << t)
        masks += own_bits
    return masks


def _prepare_attend(c, seed):
    g = _generator(seed)
    lens, q = _attend_lengths(c)
    p, h, d = c["page"], c["heads"], c["dim"]
    need = [-(-l // p) for l in lens]
    pages = sum(need) + 2
    cache = _empty_cache(c, pages)
    kv, vv, ks, vs = _views(cache)
    channel = torch.exp(0.5 * torch.randn(h, 1, 1, d, generator=g, device="cuda"))
    step = max(1, (1 << 26) // (h * p * d))
    for at in range(0, pages, step):
        m = min(step, pages - at)
        x, s = _quantize(torch.randn(m, h, p // 4, 4, d, generator=g, device="cuda") * channel, c["group"])
        kv[at:at + m], ks[at:at + m] = _pack_k(x), s.transpose(-1, -2)
        x, s = _quantize(torch.randn(m, h, p // 4, 4, d, generator=g, device="cuda"), c["group"])
        vv[at:at + m], vs[at:at + m] = _pack_v(x).transpose(-3, -2), s.transpose(-1, -2)
    order = torch.randperm(pages, generator=g, device="cuda", dtype=torch.int32)
    table = torch.full((c["n"], max(need)), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(max(need), device="cuda") < torch.tensor(need).cuda()[:, None]] = order[:sum(need)]
    starts = [0]
    for m in q:
        starts.append(starts[-1] + m)
    dtype = getattr(torch, c["dtype"])
    return {"op": "attend", "cache": cache, "table": table, "lens": _int32(lens), "starts": _int32(starts),
            "longest": max(lens), "most": max(q), "share": c["share"], "scale": d ** -0.5,
            "q": torch.randn(starts[-1], h * c["share"], d, generator=g, device="cuda").to(dtype),
            "masks": torch.tensor(_tree_masks(q, random.Random(seed))).cuda() if c["tree"] else None}


def _prepare_score(c, seed):
    g = _generator(seed)
    x = (3 * torch.randn(c["rows"], c["vocab"], generator=g, device="cuda")).to(getattr(torch, c["dtype"]))
    # the given tokens are likely ones: the best of 64 tried places
    tried = torch.randint(c["vocab"], (c["rows"], 64), generator=g, device="cuda")
    tokens = tried.gather(1, x.gather(1, tried).float().argmax(1, keepdim=True))[:, 0]
    return {"op": "score", "logits": x, "tokens": tokens, "top": c["top"]}


# ---------------------------------------------------------------------------
# one pass


def run(state):
    return {"extend": _extend, "append": _append, "attend": _attend, "score": _score}[state["op"]](state)


def _handle(state):
    """The cache handle a program makes once, next to its buffers."""
    if "handle" not in state:
        import int4_sparse_gemv_amd as i4s
        c = state["cache"]
        state["handle"] = i4s.KVCache(c["page"], c["heads"], c["dim"], c["group"], c["k_vals"], c["v_vals"],
                                      c["k_scales"], c["v_scales"])
    return state["handle"]


def _extend(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        r = i4s.kv_extend(s["table"], s["lens"], s["new"], s["free"], s["count"], s["page"], capacity=s["capacity"])
        return {"table": s["table"], "lens": r.lens, "starts": r.q_start, "slots": r.slots, "positions": r.positions,
                "count": r.free_count, "flags": r.flags}
    p, table, n, width = s["page"], s["table"], *s["table"].shape
    lens, new, count = s["lens"].long(), s["new"].long(), s["count"].long()
    old, tot = (lens + p - 1) // p, (lens + new + p - 1) // p
    starts = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    first = torch.nn.functional.pad((tot - old).cumsum(0), (1, 0))  # first new page of each request
    flags = ((lens < 0) | (new < 0)).any().int() + 2 * (tot > width).any().int()
    flags = flags + 4 * (first[-1] > count).int() + 8 * (starts[-1] > s["capacity"]).int()
    fine = flags == 0
    column = torch.arange(width, device="cuda")
    fresh = (column >= old[:, None]) & (column < tot[:, None]) & fine
    nth = (count - 1 - (first[:-1, None] + column - old[:, None])).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(fresh, s["free"][nth], table))
    t = torch.arange(s["capacity"], device="cuda")
    owner = torch.zeros(s["capacity"] + 1, dtype=torch.long, device="cuda")
    owner.index_add_(0, starts[1:-1].clamp(max=s["capacity"]), torch.ones(n - 1, dtype=torch.long, device="cuda"))
    owner = owner[:-1].cumsum(0)
    at = lens[owner] + t - starts[owner]
    inside = (t < starts[-1]) & fine
    slots = table[owner, (at // p).clamp(0, width - 1)].long() * p + at % p
    return {"table": table, "lens": torch.where(fine, lens + new, lens).int(),
            "starts": torch.where(fine, starts, 0).int(), "slots": torch.where(inside, slots, -1).int(),
            "positions": torch.where(inside, at, 0).int(), "count": torch.where(fine, count - first[-1], count).int(),
            "flags": flags.reshape(1).int()}


def _append(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        i4s.kv_append(_handle(s), s["k"], s["v"], s["slots"])
        return i4s.kv_read(_handle(s), s["slots"], dtype=s["k"].dtype)
    c = s["cache"]
    page, at = s["slots"].long() // c["page"], s["slots"].long() % c["page"]
    kv, vv, ks, vs = _views(c)
    x, f = _quantize(s["k"], c["group"])
    kv[page, :, at // 4, at % 4] = _pack_k(x)
    ks[page, :, at // 4, :, at % 4] = f
    x, f = _quantize(s["v"], c["group"])
    vv[page, :, at // 4, :, at % 4] = _pack_v(x)
    vs[page, :, at // 4, :, at % 4] = f
    out = []
    x = _unpack_k(kv[page, :, at // 4, at % 4]).unflatten(-1, (-1, c["group"]))
    out.append((x * ks[page, :, at // 4, :, at % 4].float()[..., None]).flatten(-2).to(s["k"].dtype))
    x = _unpack_v(vv[page, :, at // 4, :, at % 4]).unflatten(-1, (-1, c["group"]))
    out.append((x * vs[page, :, at // 4, :, at % 4].float()[..., None]).flatten(-2).to(s["v"].dtype))
    return tuple(out)


def _attend(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        lse = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
        out = i4s.kv_attention(_handle(s), s["q"], s["table"], s["lens"], q_start=s["starts"], max_q=s["most"],
                               max_len=s["longest"], scale=s["scale"], tree_mask=s["masks"], lse=lse)
        return out, lse
    c, n, most, share = s["cache"], s["table"].shape[0], s["most"], s["share"]
    wide = -(-s["longest"] // c["page"])
    pages = s["table"][:, :wide].long().clamp(min=0)
    kv, vv, ks, vs = (x[pages].movedim(2, 1) for x in _views(c))  # [n, heads, pages, P/4, ...]
    group = (-1, c["group"])
    k = _unpack_k(kv).unflatten(-1, group) * ks.transpose(-1, -2).float()[..., None]
    v = _unpack_v(vv.transpose(-3, -2)).unflatten(-1, group) * vs.transpose(-1, -2).float()[..., None]
    k, v = k.flatten(-2).flatten(2, 4), v.flatten(-2).flatten(2, 4)  # [n, heads, keys, dim]
    starts, lens = s["starts"].long(), s["lens"].long()
    q_len, total = starts[1:] - starts[:-1], s["q"].shape[0]
    t, key = torch.arange(most, device="cuda"), torch.arange(k.shape[2], device="cuda")
    row = (starts[:-1, None] + t).clamp(max=total - 1)
    q = s["q"].float()[row].unflatten(2, (c["heads"], share)).movedim(1, 2).flatten(2, 3)  # [n, heads, most*share, dim]
    x = (q @ k.transpose(-1, -2)).unflatten(2, (most, share)) * s["scale"]
    past = (lens - q_len)[:, None, None]
    if s["masks"] is None:
        seen = key <= past + t[:, None]
    else:
        bit = (key - past).clamp(0, 63)
        seen = (key < past) | ((s["masks"][row][:, :, None] >> bit & 1) > 0) & (key - past < 64)
    seen = (seen & (key < lens[:, None, None]))[:, None, :, None]
    x = torch.where(seen, x, -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=-1e30)
    e = torch.exp(x - m)
    l = e.sum(-1, keepdim=True)
    o = (e.flatten(2, 3) @ v).unflatten(2, (most, share)) / torch.where(l > 0, l, 1)
    lse = torch.where(l > 0, m + torch.log(l), -math.inf)[..., 0]
    owner = torch.zeros(total + 1, dtype=torch.long, device="cuda")
    owner.index_add_(0, starts[1:-1], torch.ones(n - 1, dtype=torch.long, device="cuda"))
    owner = owner[:-1].cumsum(0)
    at = torch.arange(total, device="cuda") - starts[owner]
    return o[owner, :, at].flatten(1, 2).to(s["q"].dtype), lse[owner, :, at].flatten(1, 2)


def _score(s):
    if own:
        import int4_sparse_gemv_amd as i4s
        r = i4s.token_logprobs(s["logits"], s["tokens"], top_k=s["top"])
        return [r.logprobs, r.entropy] + ([r.top_ids, r.top_logprobs] if s["top"] else [])
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    l = e.sum(1, keepdim=True)
    lse = m + torch.log(l)
    out = [x.gather(1, s["tokens"][:, None])[:, 0] - lse[:, 0],
           (torch.log(l) - ((x - m) * e).sum(1, keepdim=True) / l)[:, 0]]
    if s["top"]:
        # whole-number keys in the order of the values, the lower index first among equals
        bits = x.view(torch.int32).long()
        bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)
        ids = ((bits << 20) - torch.arange(x.shape[1], device="cuda")).topk(s["top"], 1).indices
        out += [ids.int(), x.gather(1, ids) - lse]
    return out


# ---------------------------------------------------------------------------
# the definitions in 64 bits


def exact(case, seed):
    with torch.no_grad():
        return {"extend": _exact_extend, "append": _exact_append, "attend": _exact_attend,
                "score": _exact_score}[case["op"]](case, seed)


def _exact_extend(c, seed):
    s = prepare(c, seed)
    p, table, free, count = c["page"], s["table"].tolist(), s["free"].tolist(), int(s["count"])
    held, new = s["lens"].tolist(), s["new"].tolist()
    starts, slots, positions = [0], [], []
    for row, have, more in zip(table, held, new):
        for pos in range(have, have + more):
            if pos % p == 0:
                count -= 1
                row[pos // p] = free[count]
            slots.append(row[pos // p] * p + pos % p)
            positions.append(pos)
        starts.append(len(slots))
    rest = s["capacity"] - len(slots)
    ints = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"table": ints(table), "lens": ints([a + b for a, b in zip(held, new)]), "starts": ints(starts),
            "slots": ints(slots + [-1] * rest), "positions": ints(positions + [0] * rest), "count": ints([count]),
            "flags": ints([0])}


def _exact_append(c, seed):
    s = prepare(c, seed)
    out = []
    for x in (s["k"], s["v"]):
        y = x.double().reshape(c["tokens"], c["heads"], c["dim"] // c["group"], c["group"])
        step = torch.minimum(y.abs().max(-1, keepdim=True).values / 7, torch.tensor(_SCALE_MAX, device="cuda").double())
        step = step.to(torch.float16).double()
        whole = torch.nan_to_num(torch.round(y / step), nan=0.0).clamp(-7, 7)
        out.append((whole * step).reshape(c["tokens"], c["heads"], c["dim"]))
    return tuple(out)


def _exact_attend(c, seed):
    s = prepare(c, seed)
    cache, p, d, g = s["cache"], c["page"], c["dim"], c["group"]
    dim = torch.arange(d, device="cuda")
    # byte and shift of every dimension of a token's K row, and of its V words, from the format's words
    j, a, e = dim // 32, dim % 32 // 8, dim % 8
    slot = e // 2 + 4 * (e % 2)
    k_byte, k_shift = 4 * (d // 32 * a + j) + slot // 2, 4 * (slot % 2)
    half, e = dim % 16 * (d // 64) + dim // 64, dim % 64 // 16
    v_word, v_byte, v_shift = half // 2, half % 2 * 2 + e // 2, 4 * (e % 2)
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    outs, lses = [], []
    for i, length in enumerate(lens):
        n_q = starts[i + 1] - starts[i]
        at = torch.arange(length, device="cuda")
        page, off = s["table"][i].long()[at // p], at % p
        q = s["q"][starts[i]:starts[i + 1]].double()
        bits = s["masks"][starts[i]:starts[i + 1]] if s["masks"] is not None else None
        past = length - n_q
        ahead = at - past
        if bits is None:
            seen = ahead[None] <= torch.arange(n_q, device="cuda")[:, None]
        else:
            seen = (ahead < 0)[None] | (torch.bitwise_right_shift(bits[:, None], ahead.clamp(min=0)[None]) % 2 == 1)
        seen = seen.repeat_interleave(c["share"], 0)
        o, e_sum = [], []
        for h in range(c["heads"]):
            k = (cache["k_vals"][:, h][page[:, None], off[:, None] * (d // 2) + k_byte] >> k_shift) % 16
            v = (cache["v_vals"][:, h][page[:, None], ((off // 4)[:, None] * (d // 8) + v_word) * 16
                                       + (off % 4)[:, None] * 4 + v_byte] >> v_shift) % 16
            place = ((off // 4)[:, None] * (d // g) + dim // g) * 4 + (off % 4)[:, None]
            k = (k.double() - 8) * cache["k_scales"][:, h][page[:, None], place].double()
            v = (v.double() - 8) * cache["v_scales"][:, h][page[:, None], place].double()
            rows = q[:, h * c["share"]:(h + 1) * c["share"]].reshape(-1, d)
            x = (torch.mm(rows, k.t().contiguous()) * s["scale"]).masked_fill(~seen, -math.inf)
            e_sum.append(torch.logsumexp(x, 1).view(n_q, c["share"]))
            o.append(torch.mm(torch.exp(x - torch.logsumexp(x, 1, keepdim=True)), v).view(n_q, c["share"], d))
        outs.append(torch.cat(o, 1))
        lses.append(torch.cat(e_sum, 1))
    return torch.cat(outs), torch.cat(lses)


def _exact_score(c, seed):
    s = prepare(c, seed)
    parts = []
    step = max(1, 50_000_000 // c["vocab"])
    for r in range(0, c["rows"], step):
        x = s["logits"][r:r + step].double()
        lp = x - torch.logsumexp(x, 1, keepdim=True)
        out = [lp.gather(1, s["tokens"][r:r + step, None])[:, 0], -(lp.exp() * lp).sum(1)]
        if c["top"]:
            ids = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :c["top"]]
            out += [ids.int(), lp.gather(1, ids)]
        parts.append(out)
    return [torch.cat(p) for p in zip(*parts)]
