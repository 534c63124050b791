"""The serving operators on the GPU against their float64 definitions
(``oracle/serve_oracle.py``): block tables and slot maps, the 4-bit cache,
attention over it, token scores, and a step that runs them together.

Tolerances come from the arithmetic.  A value rounded to a type is off by at
most half a step, ``eps / 2`` of itself.  The probabilities of an attention
row are rounded once to fp16 after their multiplication with V's scale: at
most 2^-11 of each, so 2^-11 of sum p |v|.  Scores are fp32 sums of exact
products of q with 16 + u, from -24 sum q: at most D + D/G + 8 roundings, each
at most 2^-24 of what the sum of the absolute terms is, sum |q| (|k| + 24 s);
a score off by d moves every probability by at most a factor exp(2d).  Below
the normal range of fp16 a rounding is off by half the smallest step instead:
2^-25 for an fp16 output, and 2^-25 for a probability times its V scale.  Those
are scaled so that the largest scale's power of two lies at 2^6 at least when
the probability is that of the key that set the row's offset (a maximum when
it was set, so the sum that divides is at least its 1): 2^-31 of the largest
scale for every key, times a value of at most 7.  Where the values carry V's
scale instead (wide blocks of rows, bf16) each is rounded once to fp16 too: another
2^-11 of sum p |v|.
"""

import itertools

import numpy as np
import pytest

from oracle import serve_oracle as O

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F16, BF16, F32 = torch.float16, torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def i4s():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import int4_sparse_gemv_amd as I
    return I


def say(*a):
    print(*a, flush=True)


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


# ---------------------------------------------------------------------------
# block tables and slot maps


def extend_both(i4s, table, lens, new, free, count, page, capacity):
    want = O.extend(table, lens, new, free, count, page, capacity)
    dev = [torch.tensor(x, dtype=torch.int32).cuda() for x in (table, lens, new, free, [count])]
    keep = [x.clone() for x in dev]
    r = i4s.kv_extend(*dev, page, capacity)
    torch.cuda.synchronize()
    got = dict(table=dev[0], lens=r.lens, q_start=r.q_start, slots=r.slots, positions=r.positions, free_count=r.free_count,
               flags=r.flags)
    for key, t in got.items():
        np.testing.assert_array_equal(t.cpu().numpy().reshape(-1), np.asarray(want[key]).reshape(-1), err_msg=key)
    for a, b in zip(dev[1:], keep[1:]):
        assert torch.equal(a, b)
    return want


@pytest.mark.parametrize("n,page,width,most_new,pad", [
    (1, 16, 4, 1, 0), (1, 256, 3, 300, 5), (3, 16, 40, 97, 0), (64, 32, 30, 3, 1), (257, 16, 20, 1, 0),
    (1000, 64, 9, 33, 777), (4096, 16, 12, 5, 3)])
def test_extend(i4s, n, page, width, most_new, pad):
    say("extend", n, page, width, most_new, pad)
    rng = np.random.default_rng(n + page)
    lens = rng.integers(0, width * page - most_new + 1, n)
    lens[rng.random(n) < 0.2] = 0
    lens[rng.random(n) < 0.2] //= page
    new = rng.integers(0, most_new + 1, n)
    table = rng.integers(0, 10**6, (n, width))
    need = int((-(-(lens + new) // page) - -(-lens // page)).sum())
    free = rng.permutation(need + 7)
    for count in (need + 7, need):
        w = extend_both(i4s, table, lens, new, free, count, page, int(new.sum()) + pad)
        assert w["flags"] == 0


@pytest.mark.parametrize("what,flags", [("length", 1), ("new", 1), ("sum", 1), ("width", 2), ("pages", 4), ("slots", 8),
                                        ("count", 16), ("negative_count", 20), ("two", 6)])
def test_extend_changes_nothing_when_something_does_not_fit(i4s, what, flags):
    say("extend refusal", what)
    lens, new, free, count, cap = [3, 0, 30], [2, 17, 2], list(range(50, 60)), 10, 30
    if what == "length":
        lens[1] = -1
    elif what == "new":
        new[2] = -5
    elif what == "sum":
        lens[0], new[0] = 2**31 - 3, 9
    elif what == "width":
        new[1] = 65
        cap = 100
    elif what == "pages":
        count = 1
    elif what == "slots":
        cap = 20
    elif what == "count":
        count = 11
    elif what == "negative_count":
        count = -2
    else:
        new[1], count, cap = 65, 2, 100
    table = np.arange(12).reshape(3, 4)
    w = extend_both(i4s, table, lens, new, free, count, 16, cap)
    assert w["flags"] == flags


@pytest.mark.parametrize("page", [16, 256])
def test_extend_page_numbers_that_no_cache_has(i4s, page):
    # in the table and in the free list: none comes round to another page's slots
    say("extend bad page numbers", page)
    shift = page.bit_length() - 1
    most = (2**31 - 1) >> shift
    odd = [-1, -2**31, most + 1, 2**(32 - shift) % 2**31, most, 7, 2**31 - 1, -2**31 + 3]
    table = np.array(odd).reshape(-1, 1).repeat(2, 1)
    w = extend_both(i4s, table, [page - 3] * len(odd), [5] * len(odd), odd[::-1], len(odd), page, 5 * len(odd))
    assert w["flags"] == 0 and max(w["slots"]) == 2**31 - 1 and w["slots"].count(-1) == 5 * 6


def test_extend_nothing_to_do(i4s):
    say("extend empty")
    extend_both(i4s, np.zeros((2, 3), np.int64), [5, 0], [0, 0], [1], 1, 16, 0)
    extend_both(i4s, np.zeros((2, 3), np.int64), [5, 0], [0, 0], [1], 0, 16, 9)
    r = i4s.kv_extend(torch.zeros(0, 4, dtype=torch.int32).cuda(), *[torch.zeros(0, dtype=torch.int32).cuda()] * 3,
                      torch.zeros(1, dtype=torch.int32).cuda(), 16, 3)
    assert r.slots.tolist() == [-1] * 3 and r.q_start.tolist() == [0] and int(r.flags) == 0


# ---------------------------------------------------------------------------
# the cache


def device_cache(i4s, c):
    """The oracle's cache on the GPU."""
    return i4s.KVCache(c.page_size, c.heads, c.dim, c.group, *[torch.from_numpy(x.copy()).cuda() for x in (
        c.k_vals, c.v_vals, c.k_scales, c.v_scales)])


def assert_same_cache(got, want):
    for name in ("k_vals", "v_vals"):
        np.testing.assert_array_equal(getattr(got, name).cpu().numpy(), getattr(want, name), err_msg=name)
    for name in ("k_scales", "v_scales"):
        np.testing.assert_array_equal(getattr(got, name).cpu().numpy().view(np.uint16), getattr(want, name).view(np.uint16),
                                      err_msg=name)


@pytest.mark.parametrize("dim,group", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)])
@pytest.mark.parametrize("tokens,heads,page,dtype", [(1, 1, 16, F16), (7, 3, 16, BF16), (37, 2, 32, F16)])
def test_append_is_bit_exact_and_read_returns_it(i4s, dim, group, tokens, heads, page, dtype):
    say("append", dim, group, tokens, heads, page, dtype)
    g = torch.Generator().manual_seed(dim + group + tokens)
    pages = -(-tokens // page) + 2
    c = O.Cache(pages, page, heads, dim, group)
    d = device_cache(i4s, c)
    qkv = (torch.randn(tokens, 3, heads, dim, generator=g) * torch.exp(torch.randn(heads, dim, generator=g))).to(dtype)
    slots = torch.randperm(pages * page, generator=g)[:tokens].int()
    if tokens > 5:
        slots[2], slots[5] = -1, pages * page  # padding, and a slot past the cache
    k, v = qkv[:, 1], qkv[:, 2]  # strided tokens
    for t in range(tokens):
        c.write(int(slots[t]), f64(k[t]), f64(v[t]))
    dev = qkv.cuda()
    i4s.kv_append(d, dev[:, 1], dev[:, 2], slots.cuda())
    torch.cuda.synchronize()
    assert_same_cache(d, c)
    wk, wv = c.read(slots.numpy())
    for out in (F16, BF16, F32):
        gk, gv = i4s.kv_read(d, slots.cuda(), dtype=out)
        for got, want in ((gk, wk), (gv, wv)):
            assert got.dtype == out
            assert torch.equal(got.cpu(), torch.from_numpy(want).to(F32).to(out))  # 4-bit x fp16 is exact in fp32


def test_quantizer_over_every_maximum(i4s):
    """Every finite positive fp16 as a group's maximum, with values around the borders between two steps."""
    say("quantizer")
    rng = np.random.default_rng(4)
    top = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)
    for dtype in (F16, BF16):
        with np.errstate(over="ignore"):
            x = top[:, None] * np.concatenate([np.ones((len(top), 1)), (rng.integers(-7, 7, (len(top), 31)) + 0.5) / 7
                                               * (1 + rng.integers(-1, 2, (len(top), 31)) * 2.0**-10)], 1)
        t = torch.from_numpy(x).to(dtype)
        t[::3] *= 2.0**-9 if dtype == BF16 else 1  # bf16 reaches below fp16's range: scales that round to 0 or a step
        t = torch.cat([t, t[:1].expand(-len(t) % 2, -1)]).reshape(-1, 1, 64)
        n = len(t)
        d = i4s.kv_cache(-(-n // 256), 256, 1, 64, 32)
        slots = torch.arange(n, dtype=torch.int32).cuda()
        i4s.kv_append(d, t.cuda(), t.cuda(), slots)
        k, v = i4s.kv_read(d, slots, dtype=F32)
        q, s = O.quantize(f64(t), 32)
        np.testing.assert_array_equal(f64(k), q * s.repeat(32, -1))
        np.testing.assert_array_equal(f64(v), q * s.repeat(32, -1))


def test_append_special_values(i4s):
    say("append special values")
    tiny = float(torch.finfo(F16).smallest_normal)
    rows = [[0.0] * 32, [-0.0] * 32, [1.0] + [0.0] * 31, [float("inf"), -float("inf"), 1.0, -70000.0] + [2.0] * 28,
            [float("nan")] * 32, [float("nan"), 3.0, -7.0] + [0.4] * 29, [1e-30] * 32, [2.0**-24 * 10, -2.0**-24 * 10] * 16,
            [1e30, -1e30, 65504.0, 9352.0 * 7] + [-1e5] * 28, [3.5 / 7, 7.0, -2.5, 0.5] + [1.5] * 28, [tiny] * 31 + [-tiny],
            [x / 2 for x in range(-16, 16)]]
    x = torch.tensor(rows).reshape(6, 1, 64)
    for dtype in (F16, BF16):
        c = O.Cache(1, 16, 1, 64, 32)
        d = device_cache(i4s, c)
        y = x.to(dtype)
        for t in range(6):
            c.write(t, f64(y[t]), f64(y[5 - t]))
        i4s.kv_append(d, y.cuda(), y.flip(0).cuda(), torch.arange(6, dtype=torch.int32).cuda())
        torch.cuda.synchronize()
        assert_same_cache(d, c)
        k, v = i4s.kv_read(d, torch.arange(6, dtype=torch.int32).cuda())
        assert torch.isfinite(k).all() and torch.isfinite(v).all()


def test_append_and_read_nothing(i4s):
    d = i4s.kv_cache(2, 16, 3, 64)
    before = d.k_vals.clone()
    none = torch.zeros(0, dtype=torch.int32).cuda()
    i4s.kv_append(d, *[torch.zeros(0, 3, 64, dtype=F16).cuda()] * 2, none)
    k, v = i4s.kv_read(d, none)
    assert k.shape == v.shape == (0, 3, 64) and torch.equal(d.k_vals, before)
    k, v = i4s.kv_read(d, torch.tensor([-1, 31, 32, 2**31 - 1], dtype=torch.int32).cuda(), dtype=F32)
    assert not k.any() and not v.any()


# ---------------------------------------------------------------------------
# attention


def filled(i4s, rng, pages, page, heads, dim, group, channel=0.5):
    """A cache with every slot held, its oracle twin, made without the library."""
    c = O.Cache(pages, page, heads, dim, group)
    n = pages * page
    strong = np.exp(channel * rng.standard_normal((heads, dim)))
    q = rng.integers(-7, 8, (2, pages, heads, page, dim))
    k_bytes = np.zeros((pages, heads, page, dim // 2), np.uint8)
    for x in range(dim):
        k_bytes[..., 4 * c.k_word[x] + c.k_bit[x] // 8] |= ((q[0][..., x] + 8) << (c.k_bit[x] % 8)).astype(np.uint8)
    c.k_vals[:] = k_bytes.reshape(pages, heads, -1)
    v_bytes = np.zeros((pages, heads, page // 4, 4, dim // 8, 4), np.uint8)
    for x in range(dim):
        v_bytes[..., c.v_word[x], c.v_bit[x] // 8] |= ((q[1][..., x] + 8) << (c.v_bit[x] % 8)).astype(np.uint8).reshape(
            pages, heads, page // 4, 4)
    c.v_vals[:] = v_bytes.transpose(0, 1, 2, 4, 3, 5).reshape(pages, heads, -1)
    ng = dim // group
    s = np.exp(0.3 * rng.standard_normal((2, pages, heads, page // 4, ng, 4))) / 4
    s[0] *= strong.reshape(heads, ng, group).mean(-1)[None, :, None, :, None]
    c.k_scales[:] = s[0].reshape(pages, heads, -1).astype(np.float16)
    c.v_scales[:] = s[1].reshape(pages, heads, -1).astype(np.float16)
    return c, device_cache(i4s, c)


def check_attention(i4s, rng, c, d, lens, q_lens, share, dtype, tree=False, scale=None, max_len=0, garbage=True, q_scale=1.0):
    page, heads, dim = c.page_size, c.heads, c.dim
    width = max(1, max(-(-l // page) for l in lens))
    order = rng.permutation(c.pages)
    # a page number behind a sequence's last page may be anything
    table = rng.integers(-2**31, 2**31, (len(lens), width)) if garbage else np.zeros((len(lens), width), np.int64)
    at = 0
    for i, l in enumerate(lens):
        n = -(-l // page)
        table[i, :n] = order[at:at + n]
        at += n
    total = sum(q_lens)
    starts = np.concatenate([[0], np.cumsum(q_lens)])
    q = torch.from_numpy(q_scale * rng.standard_normal((total, heads * share, dim))).to(dtype)
    masks = None
    if tree:
        masks = np.concatenate([[sum(1 << int(b) for b in np.nonzero(rng.random(t + 1) < 0.5)[0]) for t in range(n)]
                                for n in q_lens]).astype(np.uint64).view(np.int64)
    scale = dim**-0.5 if scale is None else scale
    extra = 3  # rows behind the last sequence
    out = torch.full((total + extra, heads * share, dim), 7.0, dtype=dtype).cuda()
    lse = torch.full((total + extra, heads * share), 7.0).cuda()
    q_dev = torch.cat([q, torch.full((extra, heads * share, dim), float("nan"), dtype=dtype)]).cuda()
    mask_dev = torch.from_numpy(np.concatenate([masks, np.zeros(extra, np.int64)])).cuda() if tree else None
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32).cuda()  # noqa: E731
    args = dict(q_start=i32(starts), max_q=max(max(q_lens), 1), max_len=max_len, scale=scale, tree_mask=mask_dev)
    i4s.kv_attention(d, q_dev, i32(table), i32(lens), out=out, lse=lse, **args)
    torch.cuda.synchronize()
    assert (out[total:] == 7).all() and (lse[total:] == 7).all(), "rows behind the last sequence"
    first = out.clone()
    i4s.kv_attention(d, q_dev, i32(table), i32(lens), out=out, lse=lse, **args)
    assert torch.equal(first, out), "two calls differ"
    got, got_lse = f64(out[:total]), f64(lse[:total])
    rows = max(max(q_lens), 1) * share
    wide = dtype == BF16 and (2 if rows > 16 and dim // c.group >= 4 else 1) * (dim // c.group) >= 8
    for i, (l, n_q) in enumerate(zip(lens, q_lens)):
        slots = [int(table[i, j // page]) * page + j % page for j in range(l)]
        k, v = c.read(slots)
        a, b = starts[i], starts[i + 1]
        qi = f64(q[a:b])
        want, want_lse, spread = O.attention(qi, k, v, l - n_q, scale, masks[a:b] if tree else None)
        s = c.scale_of(slots) if l else np.zeros((0, heads, dim))
        terms = np.zeros((n_q, heads * share))
        for h in range(heads * share if l else 0):
            terms[:, h] = (np.abs(qi[:, h]) @ (np.abs(k[:, h // share]) + 24 * s[:, h // share]).T).max(1)
        d_score = scale * terms * (dim + dim // c.group + 8) * 2.0**-24
        weight = np.expm1(2 * d_score) + (2 if wide else 1) * 2.0**-11 + (l + 64) * 2.0**-24
        v_top = 0.0 if not l else float(c.v_scales[table[i, :-(-l // page)]].max())
        tol = half_step(dtype) * np.abs(want) + 1.01 * weight[..., None] * spread + l * 7 * 2.0**-31 * v_top
        tol += 2.0**-25 if dtype == F16 else 2.0**-134
        bad = np.abs(got[a:b] - want) > tol
        assert not bad.any(), (i, np.argwhere(bad)[:3], np.abs(got[a:b] - want)[bad][:3], tol[bad][:3])
        empty = np.isneginf(want_lse)
        assert np.array_equal(empty, np.isneginf(got_lse[a:b]))
        with np.errstate(invalid="ignore"):
            off = np.abs(got_lse[a:b] - want_lse) > d_score + (l + 64) * 2.0**-24 + 2.0**-22 * np.abs(want_lse)
        assert not (off & ~empty).any()
    return got


SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128), (256, 32), (256, 64), (256, 128)]


@pytest.mark.parametrize("dim,group", SHAPES)
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_attention_shapes(i4s, dim, group, dtype):
    """Every channel count, group and query type, with one and several blocks of rows."""
    for share, q_lens in ((1, [1, 1, 1]), (3, [7, 1, 4]), (5, [9, 13, 2])):
        say("attention shapes", dim, group, dtype, share, q_lens)
        rng = np.random.default_rng(dim + group + share)
        c, d = filled(i4s, rng, 40, 16, 2, dim, group)
        check_attention(i4s, rng, c, d, [161, 33, 250], q_lens, share, dtype)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attention_lengths(i4s, page):
    """Lengths around a tile, a step of 32 keys, a page; zero and one."""
    for lens in ([0, 1, 2, 15], [16, 17, 31, 32], [33, 64, 65, page], [page + 1, page - 1, 255, 128]):
        say("attention lengths", page, lens)
        rng = np.random.default_rng(page + sum(lens))
        c, d = filled(i4s, rng, sum(-(-l // page) for l in lens) + 1, page, 1, 64, 64)
        check_attention(i4s, rng, c, d, lens, [1] * 4, 2, F16)
        check_attention(i4s, rng, c, d, lens, [3, 2, 0, 5], 2, BF16)  # more queries than keys: rows that see nothing


@pytest.mark.parametrize("q_lens,share,heads", [([16], 1, 2), ([1, 16, 5], 4, 1), ([64], 1, 1), ([33, 2], 8, 1), ([64, 1], 2, 2)])
def test_attention_tree(i4s, q_lens, share, heads):
    say("attention tree", q_lens, share, heads)
    rng = np.random.default_rng(sum(q_lens) + share)
    lens = [n + int(rng.integers(0, 90)) for n in q_lens]
    lens[0] = q_lens[0]  # no keys before the candidates: masks that leave a row empty
    c, d = filled(i4s, rng, sum(-(-l // 16) for l in lens) + 1, 16, heads, 128, 64)
    check_attention(i4s, rng, c, d, lens, q_lens, share, F16, tree=True)


@pytest.mark.parametrize("dim,heads,share,lens,q_lens", [
    (128, 2, 1, [2500], [1]), (64, 1, 4, [4097], [2]), (128, 1, 8, [1500, 7, 700], [1, 1, 1]), (256, 1, 1, [1025], [3]),
    (128, 1, 1, [3000, 1], [20, 1])])
def test_attention_splits(i4s, dim, heads, share, lens, q_lens):
    """Few rows over many keys: the keys are split and joined."""
    say("attention splits", dim, heads, share, lens)
    rng = np.random.default_rng(sum(lens))
    c, d = filled(i4s, rng, sum(-(-l // 32) for l in lens) + 1, 32, heads, dim, 64)
    check_attention(i4s, rng, c, d, lens, q_lens, share, F16)
    # a largest length that is too small costs time, not correctness
    check_attention(i4s, rng, c, d, lens, q_lens, share, BF16, max_len=40)


@pytest.mark.parametrize("q_scale,scale", [(30.0, None), (1.0, 3.0), (0.01, None), (1000.0, 1e-3)])
def test_attention_peaked_and_flat(i4s, q_scale, scale):
    say("attention peaked", q_scale, scale)
    rng = np.random.default_rng(5)
    c, d = filled(i4s, rng, 30, 16, 2, 128, 64, channel=1.5)
    c.v_scales[:, :, ::7] = 2.0**-20  # a wide range of V scales
    c.v_scales[:, 1] = 0
    c.v_scales[3:6] = 4000.0
    d = device_cache(i4s, c)
    check_attention(i4s, rng, c, d, [401], [4], 2, F16, q_scale=q_scale, scale=scale)


def test_attention_small_values_keep_their_bits(i4s):
    """V scales far below fp16's normal range, and one strong key among many weak ones."""
    say("attention small values")
    rng = np.random.default_rng(6)
    c, d = filled(i4s, rng, 70, 16, 1, 64, 64)
    c.v_scales[:] = 2.0**-24 * rng.integers(1, 5, c.v_scales.shape)
    c.k_scales[:] = (c.k_scales.astype(np.float32) / 50).astype(np.float16)
    c.k_scales[5] *= 100
    d = device_cache(i4s, c)
    # outputs near 1e-7 are subnormal in fp16: compare in bf16, which is not
    check_attention(i4s, rng, c, d, [1100], [1], 1, BF16, q_scale=2.0)


def test_attention_ignores_what_lies_behind_the_length(i4s):
    """Scales of NaN and infinity, and any nibbles, behind the last key and in the pages of others."""
    say("attention garbage")
    rng = np.random.default_rng(8)
    c, d = filled(i4s, rng, 4, 32, 2, 128, 32)
    for length in (1, 17, 33, 45):
        for bad in (np.nan, np.inf):
            d2 = device_cache(i4s, c)
            off = length % 32
            for name in ("k_scales", "v_scales"):
                s = getattr(d2, name).view(4, 2, 8, 4, 4)
                at = torch.arange(32, device="cuda").view(8, 1, 4).expand(8, 4, 4)
                last = (length - 1) // 32
                s[last][:, at >= (off if off else 32)] = bad
                s[last + 1:] = bad
            t = torch.arange(4, dtype=torch.int32).view(1, 4).cuda()
            q = torch.from_numpy(rng.standard_normal((1, 4, 128))).to(F16).cuda()
            l = torch.tensor([length], dtype=torch.int32).cuda()
            assert torch.equal(i4s.kv_attention(d2, q, t, l), i4s.kv_attention(d, q, t, l))


def test_attention_nan_query_stays_in_its_row(i4s):
    say("attention nan query")
    rng = np.random.default_rng(9)
    c, d = filled(i4s, rng, 8, 16, 1, 64, 32)
    q = torch.from_numpy(rng.standard_normal((3, 2, 64))).to(F16).cuda()
    t, l = torch.arange(8, dtype=torch.int32).view(1, 8).cuda(), torch.tensor([100], dtype=torch.int32).cuda()
    starts = torch.tensor([0, 3], dtype=torch.int32).cuda()
    want = i4s.kv_attention(d, q, t, l, q_start=starts)
    q2 = q.clone()
    q2[1, 0, 5] = float("nan")
    got = i4s.kv_attention(d, q2, t, l, q_start=starts)
    assert got[1, 0].isnan().all()
    keep = torch.ones(3, 2, dtype=torch.bool)
    keep[1, 0] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])


def test_attention_strided_query_and_bad_numbers(i4s):
    """q as a slice of a wider product; lengths, starts and pages outside their ranges stay inside the buffers."""
    say("attention strided")
    rng = np.random.default_rng(10)
    c, d = filled(i4s, rng, 6, 16, 2, 64, 64)
    wide = torch.from_numpy(rng.standard_normal((4, 8, 64))).to(BF16).cuda()
    t = torch.tensor([[0, 1, 2], [3, 4, 5], [1, 3, 5], [2, 2, 2]], dtype=torch.int32).cuda()
    l = torch.tensor([40, 48, 5, 17], dtype=torch.int32).cuda()
    a = i4s.kv_attention(d, wide[:, 2:6], t, l)
    assert torch.equal(a, i4s.kv_attention(d, wide[:, 2:6].contiguous(), t, l))
    # a page number outside is read from the nearest page inside; a length beyond the table counts as its end
    t2, l2 = t.clone(), l.clone()
    t2[0, 0], t2[1, 2], l2[1], l2[2] = -7, 2**31 - 1, 2**31 - 1, -4
    b = i4s.kv_attention(d, wide[:, 2:6], t2, l2)
    assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]]) and not b[2].any()
    starts = torch.tensor([-5, 1, 2, 3, 2**31 - 1], dtype=torch.int32).cuda()
    assert torch.equal(i4s.kv_attention(d, wide[:, 2:6], t, l, q_start=starts, max_q=1), a)


def test_attention_long_offsets(i4s):
    """Pages whose byte offsets pass 2^32."""
    say("attention long offsets")
    if torch.cuda.get_device_properties(0).total_memory < 64 << 30:
        pytest.skip("needs 64 GB")
    pages = (5 << 30) // (256 * 32 * 64)
    d = i4s.kv_cache(pages, 256, 32, 128, 128)
    slots = torch.tensor([(pages - 1) * 256 + i for i in range(40)] + [256 * (pages // 2)], dtype=torch.int32).cuda()
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(41, 32, 128, generator=g).to(F16) for _ in range(2))
    i4s.kv_append(d, k.cuda(), v.cuda(), slots)
    rk, rv = i4s.kv_read(d, slots, dtype=F32)
    (qk, sk), (qv, sv) = O.quantize(f64(k), 128), O.quantize(f64(v), 128)
    np.testing.assert_array_equal(f64(rk), qk * sk.repeat(128, -1))
    np.testing.assert_array_equal(f64(rv), qv * sv.repeat(128, -1))
    q = torch.randn(1, 32, 128, generator=g).to(F16)
    out = i4s.kv_attention(d, q.cuda(), torch.tensor([[pages - 1]], dtype=torch.int32).cuda(),
                           torch.tensor([40], dtype=torch.int32).cuda())
    want, _, spread = O.attention(f64(q), f64(rk)[:40], f64(rv)[:40], 39, 128**-0.5)
    assert (np.abs(f64(out) - want) <= half_step(F16) * np.abs(want) + 2.0**-10 * spread).all()


# ---------------------------------------------------------------------------
# scores


def check_logprobs(i4s, x, tokens, k):
    """x: torch [rows, vocab] on the CPU.  exp and log are good to 2^-22 of their value; a sum of n terms in
    partial sums of at most 64 + n / 8192 + 16 additions each has that many roundings."""
    n = x.shape[1]
    r = i4s.token_logprobs(x.cuda(), tokens.cuda(), top_k=k)
    torch.cuda.synchronize()
    lp, ent, ids, top = O.token_logprobs(f64(x), tokens.numpy(), k)
    rel = (n / 256 + 96) * 2.0**-24 + 2.0**-21
    np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
    spread = np.nanmax(np.where(np.isfinite(f64(x)), np.abs(f64(x)), 0), axis=1, initial=1.0)
    for name, got, want, s in (("logprobs", r.logprobs, lp, spread), ("entropy", r.entropy, ent, spread),
                               ("top_logprobs", r.top_logprobs, top, spread[:, None])):
        got = f64(got)
        assert got.shape == want.shape
        np.testing.assert_array_equal(np.isnan(got), np.isnan(want), err_msg=name)
        np.testing.assert_array_equal(np.isinf(got), np.isinf(want), err_msg=name)
        fine = np.isfinite(want)
        tol = rel * (2 + np.abs(np.where(fine, want, 0)) + np.log(n)) + 2.0**-23 * s * np.ones_like(want)
        assert (np.abs(np.where(fine, got, 0) - np.where(fine, want, 0)) <= tol).all(), name


@pytest.mark.parametrize("dtype", [F16, BF16, F32])
@pytest.mark.parametrize("rows,vocab,k", [(1, 1, 1), (1, 1, 0), (2, 7, 7), (3, 33, 32), (5, 1000, 1), (1, 8192, 20), (2, 8193, 32),
                                          (3, 32000, 5), (16, 50257, 20), (1, 131071, 32), (4, 151643, 0), (900, 257, 3),
                                          (800, 9000, 32)])
def test_logprobs(i4s, dtype, rows, vocab, k):
    say("logprobs", dtype, rows, vocab, k)
    g = torch.Generator().manual_seed(rows * 7 + vocab)
    x = (3 * torch.randn(rows, vocab, generator=g)).to(dtype)
    check_logprobs(i4s, x, torch.randint(vocab, (rows,), generator=g), k)


@pytest.mark.parametrize("vocab", [40, 8200, 70001])
def test_logprobs_ties_and_masks(i4s, vocab):
    """Equal values everywhere, masked vocabularies, empty rows, infinities and NaN, tokens outside."""
    say("logprobs ties", vocab)
    inf, nan = float("inf"), float("nan")
    g = torch.Generator().manual_seed(vocab)
    x = torch.zeros(17, vocab)
    x[1] = -inf                                                    # nothing left
    x[2] = -inf
    x[2, torch.randperm(vocab, generator=g)[:5]] = torch.tensor([1.0, 2.0, 2.0, 2.0, -3.0])  # a few tokens left
    x[3] = torch.randint(0, 3, (vocab,), generator=g).float()      # few different values
    x[4] = torch.arange(vocab).float().clamp(max=2000)             # rising: the best lie together
    x[5] = -torch.arange(vocab).float().clamp(max=2000)
    x[6, vocab // 2] = inf
    x[7, vocab // 3] = nan
    x[8, ::2] = -0.0                                               # -0 equals 0
    x[9] = -inf
    x[9, vocab - 1] = 4.0                                          # one token left
    x[10] = 60000.0
    x[10, 3] = -60000.0
    x[11] = torch.randn(vocab, generator=g)
    x[12, :33] = 5.0
    x[13, -33:] = 5.0
    tokens = torch.tensor([vocab - 1, 0, 1, 2, 3, 4, 5, 6, 7, vocab - 1, 3, -1, vocab, 2**40, 5, 6, 7])
    for dtype in (F16, BF16, F32):
        y = x.to(dtype)
        y[14] = torch.finfo(dtype).min                             # masked with the type's lowest value, all
        y[15] = torch.finfo(dtype).min
        y[15, 6:9] = torch.tensor([1.0, 3.0, 1.0]).to(dtype)       # or all but three
        y[16, ::3] = torch.finfo(dtype).max
        for k in (0, 1, 8, 32):
            check_logprobs(i4s, y, tokens, k)


def test_logprobs_rows_at_any_address(i4s):
    """Rows that start at every offset inside 16 bytes, strided rows, many rows (not split)."""
    say("logprobs addresses")
    g = torch.Generator().manual_seed(2)
    for dtype, rows in ((F16, 3), (F32, 3), (BF16, 800)):
        base = (2 * torch.randn(rows, 9001, generator=g)).to(dtype)
        dev = base.cuda()
        for off in range(0, 9 if rows < 9 else 3):
            x, t = dev[:, off:off + 8990], torch.full((rows,), 8989 - off)
            r = i4s.token_logprobs(x, t.cuda(), top_k=4)
            w = i4s.token_logprobs(x.contiguous(), t.cuda(), top_k=4)
            assert torch.equal(r.top_ids, w.top_ids)
            lp, ent, ids, top = O.token_logprobs(f64(x.cpu())[:5], t.numpy()[:5], 4)
            np.testing.assert_array_equal(r.top_ids.cpu().numpy()[:5], ids)
            np.testing.assert_allclose(f64(r.logprobs)[:5], lp, rtol=2e-6)
            np.testing.assert_allclose(f64(r.entropy)[:5], ent, rtol=2e-6)


def test_logprobs_no_rows(i4s):
    r = i4s.token_logprobs(torch.zeros(0, 9).cuda(), torch.zeros(0, dtype=torch.int64).cuda(), top_k=2)
    assert r.logprobs.shape == (0,) and r.top_ids.shape == (0, 2)


# ---------------------------------------------------------------------------
# together


class Server:
    """Requests of a small decoder layer: everything a step needs stays on the GPU."""

    def __init__(self, i4s, requests=3, page=16, heads=2, share=2, dim=64, vocab=500):
        self.i, self.page, self.heads, self.share, self.dim, self.vocab, self.n = i4s, page, heads, share, dim, vocab, requests
        self.cache = i4s.kv_cache(64, page, heads, dim, 32)
        self.table = torch.full((requests, 12), -1, dtype=torch.int32).cuda()
        self.lens = torch.zeros(requests, dtype=torch.int32).cuda()
        self.free = torch.randperm(64, generator=torch.Generator().manual_seed(1)).int().cuda()
        self.count = torch.tensor([64], dtype=torch.int32).cuda()

    def step(self, qkv, new, capacity, max_q, mask=None, logits=None, tokens=None):
        i4s, h, s, d = self.i, self.heads, self.share, self.dim
        r = i4s.kv_extend(self.table, self.lens, new, self.free, self.count, self.page, capacity)
        q = qkv[:, :h * s * d].unflatten(1, (h * s, d))
        k = qkv[:, h * s * d:h * (s + 1) * d].unflatten(1, (h, d))
        v = qkv[:, h * (s + 1) * d:].unflatten(1, (h, d))
        i4s.kv_append(self.cache, k, v, r.slots)
        out = torch.zeros(capacity, h * s, d, dtype=qkv.dtype, device="cuda")
        i4s.kv_attention(self.cache, q, self.table, r.lens, q_start=r.q_start, max_q=max_q, tree_mask=mask, out=out)
        scores = i4s.token_logprobs(logits, tokens, top_k=4) if logits is not None else None
        return r, out, scores

    def inputs(self, capacity, seed):
        g = torch.Generator().manual_seed(seed)
        qkv = torch.randn(capacity, self.heads * (self.share + 2) * self.dim, generator=g).to(F16).cuda()
        logits = (2 * torch.randn(capacity, self.vocab, generator=g)).to(F16).cuda()
        return qkv, logits, torch.randint(self.vocab, (capacity,), generator=g).cuda()


def test_step_together(i4s):
    """Prompts, decode steps and a tree step of three requests, against the oracle run over the same tokens."""
    say("together")
    srv = Server(i4s)
    h, s, d = srv.heads, srv.share, srv.dim
    c = O.Cache(64, 16, h, d, 32)
    held = [[], [], []]  # the slots of every request
    for n, (new, capacity) in enumerate((([5, 0, 37], 50), ([1, 1, 1], 3), ([0, 4, 1], 8), ([3, 3, 3], 9))):
        tree = n == 3
        qkv, logits, tokens = srv.inputs(capacity, n)
        mask = torch.tensor([1, 3, 5] * 3).cuda() if tree else None
        r, out, scores = srv.step(qkv, torch.tensor(new, dtype=torch.int32).cuda(), capacity, max(new), mask, logits, tokens)
        torch.cuda.synchronize()
        assert int(r.flags) == 0
        slots, at, x = r.slots.tolist(), 0, f64(qkv)
        for i, m in enumerate(new):
            for t in range(at, at + m):
                held[i].append(slots[t])
                c.write(slots[t], x[t, h * s * d:h * (s + 1) * d].reshape(h, d), x[t, h * (s + 1) * d:].reshape(h, d))
            k, v = c.read(held[i])
            q = x[at:at + m, :h * s * d].reshape(m, h * s, d)
            want, _, spread = O.attention(q, k, v, len(held[i]) - m, d**-0.5, [1, 3, 5] if tree else None)
            assert (np.abs(f64(out[at:at + m]) - want) <= half_step(F16) * np.abs(want) + 2.0**-10 * spread).all()
            at += m
        assert slots[at:] == [-1] * (capacity - at) and not out[at:].any()
        lp, ent, ids, top = O.token_logprobs(f64(logits), tokens.cpu().numpy(), 4)
        np.testing.assert_array_equal(scores.top_ids.cpu().numpy(), ids)
        np.testing.assert_allclose(f64(scores.logprobs), lp, rtol=2e-6)
        srv.lens, srv.count = r.lens, r.free_count
        assert_same_cache(srv.cache, c)
    assert len(set(itertools.chain(*held))) == sum(map(len, held))


def test_captured_step_replays(i4s):
    """A decode step in a graph, replayed with eager work and other lengths in between, against the eager call."""
    say("captured")
    srv = Server(i4s)
    r, _, _ = srv.step(srv.inputs(60, 0)[0], torch.tensor([20, 3, 30], dtype=torch.int32).cuda(), 60, 30)
    lens, count = r.lens.clone(), r.free_count.clone()
    srv.lens, srv.count = lens, count
    new = torch.ones(3, dtype=torch.int32).cuda()
    qkv, logits, tokens = srv.inputs(3, 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        srv.step(qkv, new, 3, 1, None, logits, tokens)  # warm up; writes what the next call writes again
    torch.cuda.current_stream().wait_stream(stream)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, out, scores = srv.step(qkv, new, 3, 1, None, logits, tokens)
    eager = Server(i4s)
    for seed in (6, 7, 8, 9):
        for mine, theirs in zip((qkv, logits, tokens), srv.inputs(3, seed)):
            mine.copy_(theirs)
        eager.cache.k_vals.copy_(srv.cache.k_vals), eager.cache.v_vals.copy_(srv.cache.v_vals)
        eager.cache.k_scales.copy_(srv.cache.k_scales), eager.cache.v_scales.copy_(srv.cache.v_scales)
        eager.table, eager.lens, eager.count, eager.free = srv.table.clone(), lens.clone(), count.clone(), srv.free
        graph.replay()
        torch.cuda.synchronize()
        er, eout, escores = eager.step(qkv, new, 3, 1, None, logits, tokens)
        assert torch.equal(out, eout) and all(torch.equal(a, b) for a, b in zip(r, er))
        assert all(torch.equal(a, b) for a, b in zip(scores, escores))
        assert torch.equal(srv.table, eager.table) and torch.equal(srv.cache.v_vals, eager.cache.v_vals)
        lens.copy_(r.lens), count.copy_(r.free_count)
        torch.randn(100, device="cuda").sum()


def test_verification_step_of_a_packed_layer(i4s):
    """The step that ``bench.py --verify-step`` times, on a small layer: packed products, slots, 4-bit cache, tree
    attention, scores; attention and scores against the oracle on the step's own inputs."""
    say("verification step")
    import bench
    s = bench.VerifyStep(i4s, 7, 77, seed=3, hidden=256, heads=4, mlp=512, vocab=640)
    before = (s.lens.clone(), s.count.clone())
    a, y, r = s.run()
    torch.cuda.synchronize()
    q, k, v = s.project()
    step = s.extend()
    assert int(step.flags) == 0 and step.lens.tolist() == [84] and torch.equal(s.lens, before[0])
    slots = [int(s.table[0, p // 16]) * 16 + p % 16 for p in range(84)]
    assert step.slots.tolist() == slots[77:] and step.positions.tolist() == list(range(77, 84))
    keys, values = i4s.kv_read(s.cache, torch.tensor(slots, dtype=torch.int32).cuda(), dtype=F32)
    for got, x in ((keys, k), (values, v)):
        n, f = O.quantize(f64(x).reshape(7, 4, 64), 64)
        np.testing.assert_array_equal(f64(got)[77:], n * f.repeat(64, -1))
    masks = [1, 0b11, 0b101, 0b1011, 0b10011, 0b100101, 0b1000101]
    assert s.mask.tolist() == masks
    want, _, spread = O.attention(f64(q).reshape(7, 4, 64), f64(keys), f64(values), 77, 64**-0.5, masks)
    assert (np.abs(f64(a).reshape(7, 4, 64) - want) <= half_step(F16) * np.abs(want) + 2.0**-10 * spread).all()
    logits = i4s.run(s.head, y)
    lp, ent, ids, top = O.token_logprobs(f64(logits), s.given.cpu().numpy(), 8)
    np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ids)
    # sums of 640 terms, a handful of roundings each
    np.testing.assert_allclose(f64(r.logprobs), lp, rtol=2.0**-20)
    np.testing.assert_allclose(f64(r.entropy), ent, rtol=2.0**-19)


def test_two_streams_at_once(i4s):
    """Split calls on two streams at the same time, each with a workspace of its own."""
    say("two streams")
    rng = np.random.default_rng(12)
    c, d = filled(i4s, rng, 130, 16, 1, 128, 64)
    t = torch.arange(130, dtype=torch.int32).view(1, 130).cuda()
    l = torch.tensor([2075], dtype=torch.int32).cuda()
    qs = [torch.from_numpy(rng.standard_normal((1, 4, 128))).to(F16).cuda() for _ in range(2)]
    xs = [torch.from_numpy(rng.standard_normal((2, 60000))).to(F16).cuda() for _ in range(2)]
    tok = torch.tensor([3, 4]).cuda()
    want = [(i4s.kv_attention(d, q, t, l), i4s.token_logprobs(x, tok, 5)) for q, x in zip(qs, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s, q, x, g in zip(streams, qs, xs, got):
            with torch.cuda.stream(s):
                g.append((i4s.kv_attention(d, q, t, l), i4s.token_logprobs(x, tok, 5)))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for out, r in g:
            assert torch.equal(out, w[0]) and all(torch.equal(a, b) for a, b in zip(r, w[1]))


def test_python_refusals(i4s):
    d = i4s.kv_cache(4, 16, 2, 64, 32)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32).cuda()  # noqa: E731
    q = torch.zeros(1, 2, 64, dtype=F16).cuda()
    t, l = i32(1, 2), i32(1)
    for call in (lambda: i4s.kv_attention(d, q.float(), t, l), lambda: i4s.kv_attention(d, q[..., :32], t, l),
                 lambda: i4s.kv_attention(d, q.cpu(), t, l), lambda: i4s.kv_attention(d, q, t.long(), l),
                 lambda: i4s.kv_attention(d, q, t[:, ::2], i32(2)), lambda: i4s.kv_attention(d, q, t, l, tree_mask=i32(1)),
                 lambda: i4s.kv_attention(d, q, t, l, lse=torch.zeros(2).cuda()),
                 lambda: i4s.kv_attention(d, q, t, l, out=torch.zeros(1, 2, 64).cuda()),
                 lambda: i4s.kv_append(d, q, q.bfloat16(), l), lambda: i4s.kv_append(d, q[:, :1], q[:, :1], l),
                 lambda: i4s.kv_append(d, q, q, i32(2)), lambda: i4s.kv_append(d, q.transpose(1, 2), q.transpose(1, 2), l),
                 lambda: i4s.kv_read(d, l.long()), lambda: i4s.kv_read(d, l, dtype=torch.int32),
                 lambda: i4s.kv_extend(t, i32(2), l, l, l, 16, 1), lambda: i4s.kv_extend(t.cpu(), l, l, l, l, 16, 1),
                 lambda: i4s.token_logprobs(torch.zeros(2, 5), i32(2)), lambda: i4s.token_logprobs(torch.zeros(2, 5).cuda(), i32(2)),
                 lambda: i4s.token_logprobs(torch.zeros(5, 2).cuda().t(), torch.zeros(2, dtype=torch.int64).cuda()),
                 lambda: i4s.KVCache(16, 2, 64, 32, d.k_vals, d.v_vals, d.k_scales, d.v_scales[:2])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: i4s.kv_cache(4, 17, 2, 64), lambda: i4s.kv_cache(4, 16, 2, 80), lambda: i4s.kv_cache(4, 16, 2, 64, 128),
                 lambda: i4s.kv_attention(d, torch.zeros(1, 3, 64, dtype=F16).cuda(), t, l),
                 lambda: i4s.kv_attention(d, q, t, l, scale=0.0), lambda: i4s.kv_attention(d, q, t, l, scale=float("nan")),
                 lambda: i4s.kv_attention(d, q, t, l, out=q), lambda: i4s.kv_attention(d, q, t, l, max_q=2),
                 lambda: i4s.kv_extend(t, i32(1), i32(1), i32(1), i32(1), 20, 1),
                 lambda: i4s.token_logprobs(torch.zeros(1, 5).cuda(), torch.zeros(1, dtype=torch.int64).cuda(), top_k=6)):
        with pytest.raises(i4s.I4SError):
            call()
