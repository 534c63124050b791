"""Plain NumPy definitions of the serving operators, in float64 and exact
whole numbers.  Test infrastructure only; shares no code with the library.

Values travel as float64 arrays that hold exactly what fp16, bf16 or fp32
inputs hold.  The packed cache is addressed value by value from the format's
words, without the reshapes a kernel would use.
"""

from __future__ import annotations

import numpy as np

SCALE_MAX = 9352.0
SLOT_ELEMENT = (0, 2, 4, 6, 1, 3, 5, 7)


def quantize(x, group):
    """[..., D] -> (q in -7..7, fp16 scales [..., D/group]) as float64."""
    x = np.asarray(x, np.float64)
    y = np.where(np.isnan(x), 0.0, x).reshape(*x.shape[:-1], x.shape[-1] // group, group)
    with np.errstate(invalid="ignore", over="ignore"):
        amax = np.abs(y).max(-1)
        s = np.minimum(np.minimum(amax / 7.0, SCALE_MAX).astype(np.float16).astype(np.float64), SCALE_MAX)
        q = np.where(s[..., None] > 0, y / np.where(s > 0, s, 1.0)[..., None], 0.0)
    q = np.clip(np.rint(q), -7, 7)
    return q.reshape(x.shape), s


def k_place(dim, d):
    """(32-bit word, bit) of a channel in a token's K row of head_dim d."""
    j, r = divmod(dim, 32)
    a, e = divmod(r, 8)
    return (d // 32) * a + j, 4 * SLOT_ELEMENT.index(e)


def v_place(dim, d):
    """(word, bit) of a channel among a token's V words."""
    c, r = divmod(dim, 64)
    e, i = divmod(r, 16)
    half = i * (d // 64) + c
    return half // 2, 16 * (half % 2) + 4 * e


class Cache:
    """A packed cache in host memory, read and written value by value."""

    def __init__(self, pages, page_size, heads, dim, group):
        self.page_size, self.heads, self.dim, self.group, self.pages = page_size, heads, dim, group, pages
        n = page_size * dim
        self.k_vals = np.full((pages, heads, n // 2), 0x88, np.uint8)
        self.v_vals = self.k_vals.copy()
        self.k_scales = np.zeros((pages, heads, n // group), np.float16)
        self.v_scales = self.k_scales.copy()
        self.k_word, self.k_bit = np.array([k_place(x, dim) for x in range(dim)]).T
        self.v_word, self.v_bit = np.array([v_place(x, dim) for x in range(dim)]).T

    def _at(self, off):
        """Byte and shift of K and V, and the place of the scale, of every channel at offset off."""
        d = self.dim
        kb = off * (d // 2) + 4 * self.k_word + self.k_bit // 8
        vb = (off // 4) * 2 * d + (self.v_word * 4 + off % 4) * 4 + self.v_bit // 8
        sc = ((off // 4) * (d // self.group) + np.arange(d) // self.group) * 4 + off % 4
        return kb, self.k_bit % 8, vb, self.v_bit % 8, sc

    def write(self, slot, k, v):
        """Store [heads, D] keys and values at one slot; slots outside are skipped."""
        if not 0 <= slot < self.pages * self.page_size:
            return
        page, off = divmod(slot, self.page_size)
        kb, ks, vb, vs, sc = self._at(off)
        for x, vals, scales, b, sh in ((k, self.k_vals, self.k_scales, kb, ks), (v, self.v_vals, self.v_scales, vb, vs)):
            q, s = quantize(x, self.group)
            u = (q + 8).astype(np.uint8)
            for h in range(self.heads):
                for dim in range(self.dim):
                    old = int(vals[page, h, b[dim]]) & ~(15 << int(sh[dim])) & 255
                    vals[page, h, b[dim]] = old | int(u[h, dim]) << int(sh[dim])
                scales[page, h, sc] = np.repeat(s[h], self.group).astype(np.float16)

    def read(self, slots):
        """(k, v) float64 [tokens, heads, D]; a slot outside gives zeros."""
        slots = np.asarray(slots, np.int64)
        k = np.zeros((len(slots), self.heads, self.dim))
        v = np.zeros_like(k)
        for off in range(self.page_size):
            at = np.nonzero((slots >= 0) & (slots < self.pages * self.page_size) & (slots % self.page_size == off))[0]
            if not len(at):
                continue
            page = slots[at] // self.page_size
            kb, ks, vb, vs, sc = self._at(off)
            for out, vals, scales, b, sh in ((k, self.k_vals, self.k_scales, kb, ks),
                                             (v, self.v_vals, self.v_scales, vb, vs)):
                u = (vals[page][:, :, b] >> sh) & 15
                out[at] = (u.astype(np.float64) - 8) * scales[page][:, :, sc].astype(np.float64)
        return k, v

    def scale_of(self, slots):
        """K scales of every channel, float64 [tokens, heads, D]."""
        out = np.zeros((len(slots), self.heads, self.dim))
        for n, slot in enumerate(slots):
            page, off = divmod(int(slot), self.page_size)
            out[n] = self.k_scales[page][:, self._at(off)[4]]
        return out


def attention(q, k, v, ctx, scale, masks=None):
    """One sequence: q [n_q, q_heads, D], k and v [len, kv_heads, D].
    Returns (out, lse, weight of |v|: sum p |v|)."""
    n_q, heads, d = q.shape
    length, kv_heads = k.shape[0], k.shape[1]
    share = heads // kv_heads
    out, spread = np.zeros((n_q, heads, d)), np.zeros((n_q, heads, d))
    lse = np.full((n_q, heads), -np.inf)
    for t in range(n_q):
        seen = [j for j in range(length)
                if (j <= ctx + t if masks is None else
                    j < ctx or (j - ctx < 64 and (int(masks[t]) & (2**64 - 1)) >> (j - ctx) & 1))]
        if not seen:
            continue
        for h in range(heads):
            x = scale * (k[seen, h // share] @ q[t, h])
            m = x.max()
            e = np.exp(x - m)
            lse[t, h] = m + np.log(e.sum())
            p = e / e.sum()
            out[t, h] = p @ v[seen, h // share]
            spread[t, h] = p @ np.abs(v[seen, h // share])
    return out, lse, spread


def extend(table, lens, new, free, count, page_size, capacity):
    """The whole result of a kv_extend call, by walking over the tokens."""
    table, lens, new = np.array(table), [int(x) for x in lens], [int(x) for x in new]
    n, width = table.shape
    up = lambda x: -(-x // page_size)  # noqa: E731
    flags, good = 0, []
    for have, more in zip(lens, new):
        if have < 0 or more < 0 or have + more > 2**31 - 1:
            flags |= 1
        else:
            good.append((have, more))
            if up(have + more) > width:
                flags |= 2
    need = sum(up(a + b) - up(a) for a, b in good)
    if not 0 <= count <= len(free):
        flags |= 16
    if need > max(count, 0):
        flags |= 4
    if sum(b for _, b in good) > capacity:
        flags |= 8
    slots, positions, starts = [-1] * capacity, [0] * capacity, [0] * (n + 1)
    if flags:
        return dict(table=table, lens=lens, q_start=starts, slots=slots, positions=positions, free_count=count, flags=flags)
    at = 0
    for i, (have, more) in enumerate(good):
        starts[i] = at
        for pos in range(have, have + more):
            if pos % page_size == 0:
                count -= 1
                table[i, pos // page_size] = free[count]
            page = int(table[i, pos // page_size])
            slots[at] = page * page_size + pos % page_size if 0 <= page < 2**31 // page_size else -1
            positions[at] = pos
            at += 1
    starts[n] = at
    return dict(table=table, lens=[a + b for a, b in good], q_start=starts, slots=slots, positions=positions,
                free_count=count, flags=0)


def token_logprobs(x, tokens, k):
    """Rows of float64 logits -> (logprobs, entropy, top_ids, top_logprobs)."""
    rows, vocab = x.shape
    lp, ent = np.zeros(rows), np.zeros(rows)
    ids, top = np.zeros((rows, k), np.int64), np.zeros((rows, k))
    for r in range(rows):
        row = x[r]
        order = np.argsort(-np.where(np.isnan(row), np.inf, row), kind="stable")[:k]
        ids[r] = order
        t = int(tokens[r])
        valid = 0 <= t < vocab
        if np.isnan(row).any() or np.isposinf(row).any():
            lp[r] = ent[r] = np.nan
            top[r] = np.nan
            continue
        m = row.max()
        if np.isneginf(m):
            lp[r], ent[r], top[r] = (-np.inf if valid else np.nan), 0.0, -np.inf
            continue
        e = np.exp(row - m)
        logs = row - m - np.log(e.sum())
        lp[r] = logs[t] if valid else np.nan
        p = e / e.sum()
        some = p > 0
        ent[r] = -(p[some] * logs[some]).sum()
        top[r] = logs[order]
    return lp, ent, ids, top
