// Host layer of the serving operators of libi4s (include/i4s_serve.h):
// argument checks, the launch shape of every call, and status reporting.
// Every check runs before anything is enqueued; nothing here allocates.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "i4s_serve.h"
#include "i4s_serve_internal.h"

using i4s::aligned;
using i4s::check_device;
using i4s::device_error;
using i4s::fail;
using i4s::overlap;

namespace {

// blocks along one axis of a grid: threads are counted in 32 bits, up to 512 a block
constexpr int64_t kMaxBlocks = 0x7FFFFF;

struct Span {
  const void *p;
  uint64_t n;
  const char *name;
};

// No output may share a byte with an input or with another output.
template <int NO, int NI>
i4s_status check_spans(const Span (&out)[NO], const Span (&in)[NI]) {
  for (int i = 0; i < NO; ++i) {
    if (!out[i].p || !out[i].n) continue;
    for (int j = i + 1; j < NO; ++j)
      if (out[j].p && out[j].n && overlap(out[i].p, out[i].n, out[j].p, out[j].n))
        return fail(I4S_ERR_INVALID_ARGUMENT, "%s and %s overlap", out[i].name, out[j].name);
    for (const Span &r : in)
      if (r.p && r.n && overlap(out[i].p, out[i].n, r.p, r.n))
        return fail(I4S_ERR_INVALID_ARGUMENT, "%s overlaps %s", out[i].name, r.name);
  }
  return I4S_OK;
}

i4s_status check_page_size(int32_t page_size) {
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "page_size=%d must be 16, 32, 64, 128 or 256", page_size);
  return I4S_OK;
}

i4s_status check_cache_shape(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                             int32_t group_size) {
  const i4s_status st = check_page_size(page_size);
  if (st != I4S_OK) return st;
  if (num_pages < 1 || (int64_t)num_pages * page_size > 0x7FFFFFFFll)
    return fail(I4S_ERR_INVALID_ARGUMENT, "num_pages=%d must be >= 1 and num_pages * page_size below 2^31", num_pages);
  if (kv_heads < 1 || kv_heads > 1024)
    return fail(I4S_ERR_INVALID_ARGUMENT, "kv_heads=%d must be in [1, 1024]", kv_heads);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(I4S_ERR_INVALID_ARGUMENT, "head_dim=%d must be 64, 128 or 256", head_dim);
  if ((group_size != 32 && group_size != 64 && group_size != 128) || group_size > head_dim)
    return fail(I4S_ERR_INVALID_ARGUMENT, "group_size=%d must be 32, 64 or 128 and at most head_dim=%d", group_size,
                head_dim);
  return I4S_OK;
}

void cache_sizes(const i4s_kv_cache &c, i4s_kv_sizes *out) {
  const uint64_t values = (uint64_t)c.num_pages * c.page_size * c.kv_heads * c.head_dim;
  out->vals = values / 2;
  out->scales = 2 * (values / c.group_size);
}

i4s_status check_cache(const i4s_kv_cache *c, bool buffers) {
  if (!c) return fail(I4S_ERR_INVALID_ARGUMENT, "cache is NULL");
  const i4s_status st = check_cache_shape(c->num_pages, c->page_size, c->kv_heads, c->head_dim, c->group_size);
  if (st != I4S_OK) return st;
  if (c->reserved) return fail(I4S_ERR_INVALID_ARGUMENT, "reserved=%d must be 0", c->reserved);
  if (!buffers) return I4S_OK;
  if (!c->k_vals || !aligned(c->k_vals, 16) || !c->v_vals || !aligned(c->v_vals, 16) || !c->k_scales ||
      !aligned(c->k_scales, 16) || !c->v_scales || !aligned(c->v_scales, 16))
    return fail(I4S_ERR_INVALID_ARGUMENT, "a buffer of the cache is NULL or not 16-byte aligned");
  return I4S_OK;
}

// Strides of [tokens][heads][D] values whose channels are adjacent.
i4s_status check_strides(int64_t token, int64_t head, const char *name) {
  constexpr int64_t kMost = int64_t(1) << 40;
  if (token < 0 || head < 0 || token % 8 || head % 8 || token > kMost || head > kMost)
    return fail(I4S_ERR_INVALID_ARGUMENT, "strides of %s (%lld, %lld) must be multiples of 8 elements, 0 to 2^40", name,
                (long long)token, (long long)head);
  return I4S_OK;
}

// A block takes 2048 / D tokens of a head: fewer than kMaxBlocks + 1 blocks.
i4s_status check_tokens(const i4s_kv_cache &c, int32_t tokens) {
  if (tokens < 0 || c.kv_heads * ((int64_t)tokens * c.head_dim + 2048) >= (kMaxBlocks + 1) * 2048)
    return fail(I4S_ERR_INVALID_ARGUMENT,
                "tokens=%d must be 0 or more, and kv_heads * (head_dim * tokens + 2048) below 2^34", tokens);
  return I4S_OK;
}

uint64_t extent(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
  return tokens < 1 ? 0 : 2ull * ((tokens - 1) * token + (heads - 1) * head + dim);
}

i4s_status check_attention(const i4s_attention_args *a) {
  if (!a) return fail(I4S_ERR_INVALID_ARGUMENT, "args is NULL");
  i4s_status st = check_cache(a->cache, false);
  if (st != I4S_OK) return st;
  const i4s_kv_cache &c = *a->cache;
  if (a->dtype != I4S_F16 && a->dtype != I4S_BF16)
    return fail(I4S_ERR_INVALID_ARGUMENT, "dtype=%d must be I4S_F16 or I4S_BF16", a->dtype);
  if (a->q_heads < 1 || a->q_heads > 65536 || a->q_heads % c.kv_heads)
    return fail(I4S_ERR_INVALID_ARGUMENT, "q_heads=%d must be a multiple of kv_heads=%d, at most 65536", a->q_heads,
                c.kv_heads);
  if (a->num_tokens < 0 || a->num_seqs < 0 || a->num_seqs > 65535)
    return fail(I4S_ERR_INVALID_ARGUMENT, "num_tokens=%d and num_seqs=%d must be 0 or more, num_seqs at most 65535",
                a->num_tokens, a->num_seqs);
  if (a->table_width < 1 || (int64_t)a->table_width * c.page_size > (1 << 30))
    return fail(I4S_ERR_INVALID_ARGUMENT, "table_width=%d must be >= 1 and table_width * page_size at most 2^30",
                a->table_width);
  if (a->max_q < 1 || a->max_q > 1 << 20)
    return fail(I4S_ERR_INVALID_ARGUMENT, "max_q=%d must be in [1, 2^20]", a->max_q);
  if (!a->q_start && (a->num_tokens != a->num_seqs || a->max_q != 1))
    return fail(I4S_ERR_INVALID_ARGUMENT, "without q_start num_tokens=%d must be num_seqs=%d and max_q=%d must be 1",
                a->num_tokens, a->num_seqs, a->max_q);
  if (a->max_len < 0) return fail(I4S_ERR_INVALID_ARGUMENT, "max_len=%d must be 0 or more", a->max_len);
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
    return fail(I4S_ERR_INVALID_ARGUMENT, "scale=%g must be positive and finite", (double)a->scale);
  if (a->tree_mask && a->max_q > I4S_MAX_TREE)
    return fail(I4S_ERR_INVALID_ARGUMENT, "a tree mask needs max_q=%d at most %d", a->max_q, I4S_MAX_TREE);
  if ((int64_t)a->max_q * a->q_heads > kMaxBlocks)
    return fail(I4S_ERR_INVALID_ARGUMENT, "max_q=%d times q_heads=%d must be below 2^23", a->max_q, a->q_heads);
  return I4S_OK;
}

int dtype_size(int32_t dtype) { return dtype == I4S_F32 ? 4 : 2; }

i4s_status check_logprobs(int32_t dtype, int32_t rows, int32_t vocab, int32_t top_k) {
  if (dtype != I4S_F16 && dtype != I4S_BF16 && dtype != I4S_F32)
    return fail(I4S_ERR_INVALID_ARGUMENT, "dtype=%d must be I4S_F16, I4S_BF16 or I4S_F32", dtype);
  if (rows < 0 || rows > kMaxBlocks) return fail(I4S_ERR_INVALID_ARGUMENT, "rows=%d must be in [0, 2^23)", rows);
  if (vocab < 1 || vocab > I4S_MAX_VOCAB)
    return fail(I4S_ERR_INVALID_ARGUMENT, "vocab=%d must be in [1, %d]", vocab, I4S_MAX_VOCAB);
  if (top_k < 0 || top_k > I4S_MAX_TOP_K || top_k > vocab)
    return fail(I4S_ERR_INVALID_ARGUMENT, "top_k=%d must be in [0, %d] and at most vocab=%d", top_k, I4S_MAX_TOP_K, vocab);
  return I4S_OK;
}

}  // namespace

namespace i4s {

AttentionPlan attention_plan(const i4s_attention_args &a) {
  const i4s_kv_cache &c = *a.cache;
  AttentionPlan p{};
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / c.kv_heads);
  // 16 rows a block, or 32 where four groups make a key dear by itself (its
  // scales) and the registers hold it.  Us, 32 / 16 rows a block, fp16 unless said
  // otherwise: D = 128, G = 32, 512 x up to 16384 keys, 32 rows: 237 / 364, bf16 199
  // / 362; but D = 256, 64 x 4000, 32 rows, G = 32: 48 / 45, bf16 44 / 40, G = 64: 45
  // / 40, bf16 41 / 40; D = 64, G = 32, 256 x 4000, 40 rows: 95 / 56; D = 128, G = 64,
  // 32 x 2000, 128 rows: 27 / 21, though 512 x 4000, 32 rows: 93 / 111.
  p.row_tiles = rows > 16 && c.head_dim <= 128 && c.head_dim / c.group_size >= 4 ? 2 : 1;
  p.row_blocks = (int)((rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles));
  // eight waves a block where their registers fit a compute unit: twice the
  // keys before a second launch has to join pieces
  p.waves = p.row_tiles == 1 && c.head_dim <= 128 ? 8 : 4;
  const int64_t capacity = (int64_t)a.table_width * c.page_size;
  const int64_t len = a.max_len > 0 && a.max_len < capacity ? a.max_len : capacity;
  // The keys in pieces.  Measured in graphs, us, one query token of fp16, D =
  // 128, unless said otherwise (units = sequences x KV heads x row blocks):
  //   about one block for each of the 256 compute units: 8 units x 131071
  //     keys in 32 / 64 / 16 pieces 35 / 33 / 54; 64 x 8000 (8 rows) in 4 / 8 / 2:
  //     22.4 / 22.3 / 31.4; 40 x 2047 (16 rows) in 4 / 8 / 1: 13.5 / 14.8 / 18.8;
  //     160 x 4000 (16 rows) in 1 / 4 / 8: 33 / 33 / 35;
  //   with as many units as that one piece (512 x 4095, in 1 / 2 / 4: 59 / 58 /
  //     63), but none longer than 4096 keys while that gives no more than about
  //     2048 blocks (and partial results of 35 MB), so that sequences of
  //     different lengths fill the chip to the end (512 x up to 16384, 32 rows,
  //     in 4 / 2 / 1: 197 / 209 / 224);
  //   a step or four of every wave are not worth a second launch (32 x 1023:
  //     11.9 in one launch, 12.1 in two, and that costs the host 3).
  // The pieces follow max_len, or the table's width where that is 0: a length far
  // below it uses few of them (8 x 16384 keys, 4 rows: 14 with the length, 31
  // with a table for 131072 tokens; 512 x up to 4095: 42 / 42).
  const int64_t units = (int64_t)p.row_blocks * c.kv_heads * (a.num_seqs > 0 ? a.num_seqs : 1);
  const int64_t step = kStepKeys * p.waves;
  const int64_t even = clamp_to<int64_t>((len + 4095) / 4096, 1, 2048 / units + 1);
  const int64_t want = len <= 4 * step ? 1 : clamp_to<int64_t>(256 / units, even, kMaxSplits);
  const int64_t per = clamp_to<int64_t>((len + want * step - 1) / (want * step), 1, (1 << 30) / step);
  p.chunk = (int)(per * step);
  p.splits = (int)clamp_to<int64_t>((len + p.chunk - 1) / p.chunk, 1, kMaxSplits);
  if (p.splits > 1)
    p.workspace_bytes = (uint64_t)p.splits * a.num_tokens * a.q_heads * (c.head_dim + 4) * sizeof(float);
  return p;
}

LogprobsPlan logprobs_plan(int32_t dtype, int32_t rows, int32_t vocab, int32_t top_k) {
  LogprobsPlan p{};
  // Pieces for about two blocks a compute unit, where that pays a second
  // launch.  Measured in graphs, us, in one / several pieces: 1 x 150000 fp16
  // 25 / 13 (10), 16 x 151643 fp32 35 / 17.5 (10), 64 x 50257 bf16 20 / 17
  // (7), 200 x 151643 37 / 32 (2); but 16 x 32000 11 / 13 (2), 200 x 32000 15
  // / 19 (2), 600 x 50257 31 / 35 (2).
  const int all = (vocab + 128 / dtype_size(dtype) - 1 + kSegment - 1) / kSegment;  // rows begin inside a line
  const int want = rows < 1 || rows > 256 || vocab <= 32768 ? 1 : clamp_to(512 / rows, 1, 16);
  p.segments = clamp_to((all + want - 1) / want, 1, kMaxSegments);
  p.splits = (all + p.segments - 1) / p.segments;
  if (p.splits > 1)
    p.workspace_bytes = (uint64_t)rows * p.splits * (4 * sizeof(float) + top_k * sizeof(uint64_t));
  return p;
}

}  // namespace i4s

extern "C" {

i4s_status i4s_kv_cache_sizes(int32_t num_pages, int32_t page_size, int32_t kv_heads, int32_t head_dim,
                              int32_t group_size, i4s_kv_sizes *out) {
  if (!out) return fail(I4S_ERR_INVALID_ARGUMENT, "out is NULL");
  const i4s_status st = check_cache_shape(num_pages, page_size, kv_heads, head_dim, group_size);
  if (st != I4S_OK) return st;
  i4s_kv_cache c{};
  c.num_pages = num_pages, c.page_size = page_size, c.kv_heads = kv_heads;
  c.head_dim = head_dim, c.group_size = group_size;
  cache_sizes(c, out);
  return I4S_OK;
}

i4s_status i4s_kv_extend(int32_t *table, int32_t n, int32_t width, int32_t page_size, const int32_t *lens,
                         const int32_t *new_lens, const int32_t *free_pages, int32_t free_entries,
                         const int32_t *free_count, int32_t capacity, int32_t *lens_out, int32_t *q_start,
                         int32_t *slots, int32_t *positions, int32_t *free_count_out, int32_t *flags, void *stream) {
  i4s_status st = check_page_size(page_size);
  if (st != I4S_OK) return st;
  if (n < 0 || n > I4S_KV_MAX_REQUESTS)
    return fail(I4S_ERR_INVALID_ARGUMENT, "n=%d must be in [0, %d]", n, I4S_KV_MAX_REQUESTS);
  if (width < 1) return fail(I4S_ERR_INVALID_ARGUMENT, "width=%d must be >= 1", width);
  if (capacity < 0 || free_entries < 0)
    return fail(I4S_ERR_INVALID_ARGUMENT, "capacity=%d and free_entries=%d must be 0 or more", capacity, free_entries);
  const Span out[] = {{table, 4ull * n * width, "table"},
                      {lens_out, 4ull * n, "lens_out"},
                      {q_start, 4ull * (n + 1), "q_start"},
                      {slots, 4ull * capacity, "slots"},
                      {positions, 4ull * capacity, "positions"},
                      {free_count_out, 4, "free_count_out"},
                      {flags, 4, "flags"}};
  const Span in[] = {{lens, 4ull * n, "lens"},
                     {new_lens, 4ull * n, "new_lens"},
                     {free_pages, 4ull * free_entries, "free_pages"},
                     {free_count, 4, "free_count"}};
  for (const Span &s : out)
    if (s.n && (!s.p || !aligned(s.p, 4))) return fail(I4S_ERR_INVALID_ARGUMENT, "%s is NULL or not 4-byte aligned", s.name);
  for (const Span &s : in)
    if (s.n && (!s.p || !aligned(s.p, 4))) return fail(I4S_ERR_INVALID_ARGUMENT, "%s is NULL or not 4-byte aligned", s.name);
  st = check_spans(out, in);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  i4s::ExtendArgs a{table, n, width, i4s::page_shift(page_size), lens, new_lens, free_pages, free_entries, free_count,
                    capacity, lens_out, q_start, slots, positions, free_count_out, flags};
  const hipError_t e = i4s::launch_kv_extend(a, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "kv_extend launch");
}

i4s_status i4s_kv_append(const i4s_kv_cache *cache, const void *k, const void *v, int32_t dtype, int64_t k_token_stride,
                         int64_t k_head_stride, int64_t v_token_stride, int64_t v_head_stride, const int32_t *slots,
                         int32_t tokens, void *stream) {
  i4s_status st = check_cache(cache, true);
  if (st != I4S_OK) return st;
  if (dtype != I4S_F16 && dtype != I4S_BF16)
    return fail(I4S_ERR_INVALID_ARGUMENT, "dtype=%d must be I4S_F16 or I4S_BF16", dtype);
  st = check_tokens(*cache, tokens);
  if (st != I4S_OK) return st;
  st = check_strides(k_token_stride, k_head_stride, "k");
  if (st != I4S_OK) return st;
  st = check_strides(v_token_stride, v_head_stride, "v");
  if (st != I4S_OK) return st;
  if (tokens == 0) return I4S_OK;
  if (!k || !aligned(k, 16) || !v || !aligned(v, 16))
    return fail(I4S_ERR_INVALID_ARGUMENT, "k or v is NULL or not 16-byte aligned");
  if (!slots || !aligned(slots, 4)) return fail(I4S_ERR_INVALID_ARGUMENT, "slots is NULL or not 4-byte aligned");
  i4s_kv_sizes sz;
  cache_sizes(*cache, &sz);
  const Span out[] = {{cache->k_vals, sz.vals, "k_vals"},
                      {cache->v_vals, sz.vals, "v_vals"},
                      {cache->k_scales, sz.scales, "k_scales"},
                      {cache->v_scales, sz.scales, "v_scales"}};
  const Span in[] = {{k, extent(tokens, k_token_stride, cache->kv_heads, k_head_stride, cache->head_dim), "k"},
                     {v, extent(tokens, v_token_stride, cache->kv_heads, v_head_stride, cache->head_dim), "v"},
                     {slots, 4ull * tokens, "slots"}};
  st = check_spans(out, in);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  const i4s::AppendArgs a{*cache, k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, tokens};
  const hipError_t e = i4s::launch_kv_append(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "kv_append launch");
}

i4s_status i4s_kv_read(const i4s_kv_cache *cache, const int32_t *slots, int32_t tokens, int32_t dtype, void *k_out,
                       void *v_out, void *stream) {
  i4s_status st = check_cache(cache, true);
  if (st != I4S_OK) return st;
  if (dtype != I4S_F16 && dtype != I4S_BF16 && dtype != I4S_F32)
    return fail(I4S_ERR_INVALID_ARGUMENT, "dtype=%d must be I4S_F16, I4S_BF16 or I4S_F32", dtype);
  st = check_tokens(*cache, tokens);
  if (st != I4S_OK) return st;
  if (tokens == 0) return I4S_OK;
  if (!k_out || !aligned(k_out, 16) || !v_out || !aligned(v_out, 16))
    return fail(I4S_ERR_INVALID_ARGUMENT, "k_out or v_out is NULL or not 16-byte aligned");
  if (!slots || !aligned(slots, 4)) return fail(I4S_ERR_INVALID_ARGUMENT, "slots is NULL or not 4-byte aligned");
  i4s_kv_sizes sz;
  cache_sizes(*cache, &sz);
  const uint64_t bytes = (uint64_t)tokens * cache->kv_heads * cache->head_dim * dtype_size(dtype);
  const Span out[] = {{k_out, bytes, "k_out"}, {v_out, bytes, "v_out"}};
  const Span in[] = {{cache->k_vals, sz.vals, "k_vals"},
                     {cache->v_vals, sz.vals, "v_vals"},
                     {cache->k_scales, sz.scales, "k_scales"},
                     {cache->v_scales, sz.scales, "v_scales"},
                     {slots, 4ull * tokens, "slots"}};
  st = check_spans(out, in);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  const i4s::ReadArgs a{*cache, slots, tokens, k_out, v_out};
  const hipError_t e = i4s::launch_kv_read(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "kv_read launch");
}

i4s_status i4s_attention_workspace_size(const i4s_attention_args *a, uint64_t *bytes) {
  if (!bytes) return fail(I4S_ERR_INVALID_ARGUMENT, "bytes is NULL");
  const i4s_status st = check_attention(a);
  if (st != I4S_OK) return st;
  *bytes = a->num_tokens && a->num_seqs ? i4s::attention_plan(*a).workspace_bytes : 0;
  return I4S_OK;
}

i4s_status i4s_attention(const i4s_attention_args *a, void *stream) {
  i4s_status st = check_attention(a);
  if (st != I4S_OK) return st;
  const i4s_kv_cache &c = *a->cache;
  st = check_cache(&c, true);
  if (st != I4S_OK) return st;
  st = check_strides(a->q_token_stride, a->q_head_stride, "q");
  if (st != I4S_OK) return st;
  if (a->num_tokens == 0 || a->num_seqs == 0) return I4S_OK;
  if (!a->q || !aligned(a->q, 16) || !a->out || !aligned(a->out, 16))
    return fail(I4S_ERR_INVALID_ARGUMENT, "q or out is NULL or not 16-byte aligned");
  if (!a->table || !aligned(a->table, 4) || !a->lens || !aligned(a->lens, 4))
    return fail(I4S_ERR_INVALID_ARGUMENT, "table or lens is NULL or not 4-byte aligned");
  if (!aligned(a->q_start, 4) || !aligned(a->lse, 4) || !aligned(a->tree_mask, 8))
    return fail(I4S_ERR_INVALID_ARGUMENT, "q_start, lse or tree_mask is misaligned (need 4/4/8 bytes)");
  const i4s::AttentionPlan p = i4s::attention_plan(*a);
  if (p.workspace_bytes) {
    if (!a->workspace || !aligned(a->workspace, 16))
      return fail(I4S_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (a->workspace_bytes < p.workspace_bytes)
      return fail(I4S_ERR_WORKSPACE_TOO_SMALL, "workspace has %llu bytes, %llu needed",
                  (unsigned long long)a->workspace_bytes, (unsigned long long)p.workspace_bytes);
  }
  i4s_kv_sizes sz;
  cache_sizes(c, &sz);
  const uint64_t rows = (uint64_t)a->num_tokens * a->q_heads;
  const Span out[] = {{a->out, 2 * rows * c.head_dim, "out"},
                      {a->lse, 4 * rows, "lse"},
                      {a->workspace, p.workspace_bytes, "workspace"}};
  const Span in[] = {{a->q, extent(a->num_tokens, a->q_token_stride, a->q_heads, a->q_head_stride, c.head_dim), "q"},
                     {c.k_vals, sz.vals, "k_vals"},
                     {c.v_vals, sz.vals, "v_vals"},
                     {c.k_scales, sz.scales, "k_scales"},
                     {c.v_scales, sz.scales, "v_scales"},
                     {a->table, 4ull * a->num_seqs * a->table_width, "table"},
                     {a->lens, 4ull * a->num_seqs, "lens"},
                     {a->q_start, 4ull * (a->num_seqs + 1), "q_start"},
                     {a->tree_mask, 8ull * a->num_tokens, "tree_mask"}};
  st = check_spans(out, in);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;

  i4s::AttentionKernelArgs k{};
  k.k_vals = c.k_vals, k.v_vals = c.v_vals, k.k_scales = c.k_scales, k.v_scales = c.v_scales;
  k.num_pages = c.num_pages, k.shift = i4s::page_shift(c.page_size), k.kv_heads = c.kv_heads;
  k.share = a->q_heads / c.kv_heads;
  k.q = a->q, k.q_token = a->q_token_stride, k.q_head = a->q_head_stride;
  k.num_tokens = a->num_tokens, k.num_seqs = a->num_seqs;
  k.table = a->table, k.width = a->table_width, k.lens = a->lens, k.q_start = a->q_start;
  k.max_q = a->max_q, k.row_blocks = p.row_blocks, k.splits = p.splits, k.chunk = p.chunk;
  const double scale_log2 = (double)a->scale * 1.4426950408889634;
  k.scale_log2 = (float)std::fmin(scale_log2, FLT_MAX);
  k.slack = (float)std::fmin(i4s::kAttentionSlack / scale_log2, FLT_MAX);
  k.tree = a->tree_mask, k.out = a->out, k.lse = a->lse;
  k.part_o = static_cast<float *>(a->workspace);
  k.part_ml = p.workspace_bytes ? k.part_o + (uint64_t)p.splits * rows * c.head_dim : nullptr;
  const hipError_t e = i4s::launch_attention(k, p, c.head_dim, c.group_size, a->dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "attention launch");
}

i4s_status i4s_token_logprobs_workspace_size(int32_t dtype, int32_t rows, int32_t vocab, int32_t top_k, uint64_t *bytes) {
  if (!bytes) return fail(I4S_ERR_INVALID_ARGUMENT, "bytes is NULL");
  const i4s_status st = check_logprobs(dtype, rows, vocab, top_k);
  if (st != I4S_OK) return st;
  *bytes = i4s::logprobs_plan(dtype, rows, vocab, top_k).workspace_bytes;
  return I4S_OK;
}

i4s_status i4s_token_logprobs(const void *logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t stride,
                              const int64_t *tokens, int32_t top_k, float *logprobs, float *entropy, int32_t *top_ids,
                              float *top_logprobs, void *workspace, uint64_t workspace_bytes, void *stream) {
  i4s_status st = check_logprobs(dtype, rows, vocab, top_k);
  if (st != I4S_OK) return st;
  if (stride < vocab || stride > int64_t(1) << 40)
    return fail(I4S_ERR_INVALID_ARGUMENT, "stride=%lld must be at least vocab=%d, at most 2^40", (long long)stride, vocab);
  if (rows == 0) return I4S_OK;
  if (!logits || !aligned(logits, dtype_size(dtype)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "logits is NULL or not aligned to its element");
  if (!tokens || !aligned(tokens, 8)) return fail(I4S_ERR_INVALID_ARGUMENT, "tokens is NULL or not 8-byte aligned");
  if (!logprobs || !aligned(logprobs, 4) || !entropy || !aligned(entropy, 4))
    return fail(I4S_ERR_INVALID_ARGUMENT, "logprobs or entropy is NULL or not 4-byte aligned");
  if (top_k && (!top_ids || !aligned(top_ids, 4) || !top_logprobs || !aligned(top_logprobs, 4)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "top_ids or top_logprobs is NULL or not 4-byte aligned");
  const i4s::LogprobsPlan p = i4s::logprobs_plan(dtype, rows, vocab, top_k);
  if (p.workspace_bytes) {
    if (!workspace || !aligned(workspace, 16))
      return fail(I4S_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (workspace_bytes < p.workspace_bytes)
      return fail(I4S_ERR_WORKSPACE_TOO_SMALL, "workspace has %llu bytes, %llu needed", (unsigned long long)workspace_bytes,
                  (unsigned long long)p.workspace_bytes);
  }
  const Span out[] = {{logprobs, 4ull * rows, "logprobs"},
                      {entropy, 4ull * rows, "entropy"},
                      {top_ids, 4ull * rows * top_k, "top_ids"},
                      {top_logprobs, 4ull * rows * top_k, "top_logprobs"},
                      {workspace, p.workspace_bytes, "workspace"}};
  const Span in[] = {{logits, ((uint64_t)(rows - 1) * stride + vocab) * dtype_size(dtype), "logits"},
                     {tokens, 8ull * rows, "tokens"}};
  st = check_spans(out, in);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  i4s::LogprobsArgs a{};
  a.logits = logits, a.rows = rows, a.vocab = vocab, a.stride = stride, a.tokens = tokens, a.top_k = top_k;
  a.logprobs = logprobs, a.entropy = entropy, a.top_ids = top_ids, a.top_logprobs = top_logprobs;
  a.part_keys = static_cast<uint64_t *>(workspace);
  a.part_stats = reinterpret_cast<float *>(a.part_keys + (uint64_t)rows * p.splits * top_k);
  const hipError_t e = i4s::launch_token_logprobs(a, p, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "token_logprobs launch");
}

}  // extern "C"
