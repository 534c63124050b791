// Host layer of the prompt's operators of libi4s (include/i4s_prompt.h):
// argument checks, the launch shape of every call, and status reporting.
// Every check runs before anything is enqueued; nothing here allocates.

#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "i4s_prompt.h"
#include "i4s_prompt_internal.h"

using i4s::aligned;
using i4s::check_device;
using i4s::check_spans;
using i4s::device_error;
using i4s::dtype_size;
using i4s::fail;
using i4s::kMaxBlocks;
using i4s::Span;

namespace {

constexpr int32_t kMxMaxRows = 1 << 24, kMxMaxCols = 1 << 20;
constexpr int64_t kMaxStride = int64_t(1) << 40, kMaxTokenStride = 1 << 23;

i4s_status check_mx_shape(int32_t rows, int32_t cols) {
  if (rows < 0 || rows > kMxMaxRows) return fail(I4S_ERR_INVALID_ARGUMENT, "rows=%d must be in [0, 2^24]", rows);
  if (cols < 32 || cols > kMxMaxCols || cols % 32)
    return fail(I4S_ERR_INVALID_ARGUMENT, "cols=%d must be a multiple of 32 in [32, 2^20]", cols);
  // a block of 64 threads takes 16 rows x 512 columns
  if ((int64_t)i4s::mx_row_tiles(rows) * i4s::mx_groups(cols) > 4 * kMaxBlocks)
    return fail(I4S_ERR_INVALID_ARGUMENT, "rows=%d times cols=%d must be below 2^38", rows, cols);
  return I4S_OK;
}

i4s_status check_mx(const i4s_mx *m, const char *name, bool buffers) {
  if (!m) return fail(I4S_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  const i4s_status st = check_mx_shape(m->rows, m->cols);
  if (st != I4S_OK) return st;
  if (buffers && m->rows && (!m->vals || !aligned(m->vals, 16) || !m->scales || !aligned(m->scales, 16)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "a buffer of %s is NULL or not 16-byte aligned", name);
  return I4S_OK;
}

i4s_status check_half(int32_t dtype, const char *name) {
  if (dtype != I4S_F16 && dtype != I4S_BF16)
    return fail(I4S_ERR_INVALID_ARGUMENT, "%s=%d must be I4S_F16 or I4S_BF16", name, dtype);
  return I4S_OK;
}

i4s_status check_any(int32_t dtype, const char *name) {
  if (dtype != I4S_F16 && dtype != I4S_BF16 && dtype != I4S_F32)
    return fail(I4S_ERR_INVALID_ARGUMENT, "%s=%d must be I4S_F16, I4S_BF16 or I4S_F32", name, dtype);
  return I4S_OK;
}

i4s_status check_row_stride(int64_t stride, int32_t cols, const char *name) {
  if (stride < cols || stride % 8 || stride > kMaxStride)
    return fail(I4S_ERR_INVALID_ARGUMENT, "%s=%lld must be a multiple of 8, at least cols=%d and at most 2^40", name,
                (long long)stride, cols);
  return I4S_OK;
}

Span vals_of(const i4s_mx &m, const char *name) { return {m.vals, i4s::mx_vals_bytes(m.rows, m.cols), name}; }
Span scales_of(const i4s_mx &m, const char *name) { return {m.scales, i4s::mx_scales_bytes(m.rows, m.cols), name}; }

// What the size of the workspace follows from: of x only whether it is given.
i4s_status check_product(const i4s_mx_product_args *a) {
  if (!a) return fail(I4S_ERR_INVALID_ARGUMENT, "args is NULL");
  i4s_status st = check_mx(a->w, "w", false);
  if (st != I4S_OK) return st;
  st = check_mx_shape(a->tokens, a->w->cols);
  if (st != I4S_OK) return st;
  // Blocks of a grid.  Those of less than 128 x 128 outputs are taken only while they are
  // few (mx_product_plan), or for up to 64 tokens: two weight tiles each, up to 2^19.
  if (((int64_t)a->tokens + 127) / 128 * (((int64_t)a->w->rows + 127) / 128) > kMaxBlocks)
    return fail(I4S_ERR_INVALID_ARGUMENT, "tokens=%d times w's rows=%d must be below 2^37", a->tokens, a->w->rows);
  if (a->reserved) return fail(I4S_ERR_INVALID_ARGUMENT, "reserved=%d must be 0", a->reserved);
  return I4S_OK;
}

i4s_status check_prompt(const i4s_prompt_args *a) {
  if (!a) return fail(I4S_ERR_INVALID_ARGUMENT, "args is NULL");
  const i4s_status st = check_half(a->dtype, "dtype");
  if (st != I4S_OK) return st;
  if (a->head_dim != 64 && a->head_dim != 128 && a->head_dim != 256)
    return fail(I4S_ERR_INVALID_ARGUMENT, "head_dim=%d must be 64, 128 or 256", a->head_dim);
  if (a->kv_heads < 1 || a->kv_heads > 1024)
    return fail(I4S_ERR_INVALID_ARGUMENT, "kv_heads=%d must be in [1, 1024]", a->kv_heads);
  if (a->q_heads < 1 || a->q_heads > 65536 || a->q_heads % a->kv_heads)
    return fail(I4S_ERR_INVALID_ARGUMENT, "q_heads=%d must be a multiple of kv_heads=%d, at most 65536", a->q_heads,
                a->kv_heads);
  if (a->num_tokens < 0 || a->num_keys < 0 || a->num_tokens > 1 << 30 || a->num_keys > 1 << 30)
    return fail(I4S_ERR_INVALID_ARGUMENT, "num_tokens=%d and num_keys=%d must be in [0, 2^30]", a->num_tokens, a->num_keys);
  if (a->num_seqs < 0 || a->num_seqs > 65535)
    return fail(I4S_ERR_INVALID_ARGUMENT, "num_seqs=%d must be in [0, 65535]", a->num_seqs);
  if (a->max_q < 1 || a->max_q > 1 << 24)
    return fail(I4S_ERR_INVALID_ARGUMENT, "max_q=%d must be in [1, 2^24]", a->max_q);
  if (a->max_k < 0) return fail(I4S_ERR_INVALID_ARGUMENT, "max_k=%d must be 0 or more", a->max_k);
  if (a->causal != 0 && a->causal != 1) return fail(I4S_ERR_INVALID_ARGUMENT, "causal=%d must be 0 or 1", a->causal);
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
    return fail(I4S_ERR_INVALID_ARGUMENT, "scale=%g must be positive and finite", (double)a->scale);
  if (a->reserved) return fail(I4S_ERR_INVALID_ARGUMENT, "reserved=%d must be 0", a->reserved);
  const int64_t rows = (int64_t)a->max_q * (a->q_heads / a->kv_heads);
  const int64_t blocks = (rows + 127) / 128 * a->kv_heads * (a->num_seqs > 0 ? a->num_seqs : 1);
  if (blocks > kMaxBlocks)
    return fail(I4S_ERR_INVALID_ARGUMENT, "max_q=%d, q_heads=%d and num_seqs=%d make %lld blocks of 128 rows; at most 2^23 - 1",
                a->max_q, a->q_heads, a->num_seqs, (long long)blocks);
  return I4S_OK;
}

i4s_status check_strides(int64_t token, int64_t head, const char *name) {
  if (token < 0 || head < 0 || token % 8 || head % 8 || token > kMaxTokenStride || head > kMaxStride)
    return fail(I4S_ERR_INVALID_ARGUMENT,
                "strides of %s (%lld, %lld) must be multiples of 8 elements, 0 to 2^23 between tokens, to 2^40 between heads",
                name, (long long)token, (long long)head);
  return I4S_OK;
}

uint64_t extent(int64_t tokens, int64_t token, int64_t heads, int64_t head, int64_t dim) {
  return tokens < 1 ? 0 : 2ull * ((tokens - 1) * token + (heads - 1) * head + dim);
}

}  // namespace

namespace i4s {

MxProductPlan mx_product_plan(int32_t tokens, int32_t rows, int32_t cols, bool x_given) {
  MxProductPlan p{};
  // 16-bit tokens: quantized by every block of the product while they are few,
  // else by a launch of its own.  Us in graphs, on the way / before: 13824 x 5120, 8
  // tokens 9.3 / 11.5, 12: 11.1 / 11.5, 16: 12.6 / 11.5; 4096 x 4096, 8: 4.9 / 6.3, 16: 6.7 /
  // 6.4; 22016 x 4096, 8: 12.4 / 13.1, 16: 16.1 / 13.4; 4096 x 11008, 8: 9.3 / 9.2, 16: 14.9 /
  // 9.5.
  p.quantize = !x_given && (tokens > 16 || (int64_t)tokens * cols >= 1 << 16);
  p.token_tiles = (tokens + 15) / 16;
  // Blocks of eight waves and 1, 2 or (where each quantizes the tokens) 4 weight
  // tiles, about one or two for each of the 256 compute units; beyond, and for
  // more than 16 tokens sooner, four waves and 2.  Waves decide the order of the
  // sums and so must not depend on how the tokens are given.
  // Us, 16 quantized tokens, tiles x waves 1x8 / 2x8 / 2x4: 4096 x 4096 3.7 / 4.1 / 4.3;
  // 5120 x 13824 11.9 / 10.6 / 10.8; 13824 x 5120 10.5 / 9.8 / 9.7, 64 tokens 21.4 / 17.8
  // / 13.5; 50257 x 4096, 48 tokens 45 / 42 / 30.  8 tokens quantized on the way, four at
  // a time, 2x8 / 4x8 / 2x4: 13824 x 5120 14.5 / 10.9 / 12.8; 50257 x 4096 32 / 31 / 26.
  const int32_t tiles = mx_row_tiles(rows);
  p.row_tiles = tiles <= 256 ? 1 : 2;
  p.waves = tiles <= (p.token_tiles == 1 ? 1024 : 512) ? 8 : 4;
  if (!x_given && !p.quantize && tiles > 512 && p.waves == 8) p.row_tiles = 4;
  // Few tokens' blocks (more than 64 tokens: several of them, 2x4) while they are few
  // enough to be on the chip together.  Us, few / 64 x 128 outputs: 4096 x 4096, 128 tokens
  // 6.5 / 9.5, 256 (512 blocks) 8.6 / 10.4, 320 (640) 11.1 / 10.7; 5120 x 13824, 256 (640) 28 / 30,
  // 320 (800) 34 / 30; 11008 x 4096, 80 (688) 13.0 / 11.5; 2048 x 2048, 512 (512) 5.9 / 6.5, 768
  // (768) 8.3 / 6.7.  11008 x 4096, 64 tokens 11 / 13 (128 x 128).
  p.few = p.token_tiles <= 4 || ((int64_t)tiles + 1) / 2 * ((p.token_tiles + 3) / 4) <= 640;
  if (p.token_tiles > 4) p.row_tiles = 2, p.waves = 4;
  // 64 x 128 outputs while there is a compute unit for each block.  Us, 64 x 128 / 128 x
  // 128: 4096 x 4096, 512 tokens 11.3 / 13.4; 11008 x 4096, 128 (172 blocks) 12.0 / 14.2, 192
  // (344) 15.2 / 14.0; 13824 x 5120, 128 (216) 15.7 / 18.2, 160 (432) 18.8 / 17.4.
  // 256 x 256 outputs, one block a compute unit, where they fill more than three
  // quarters of whole rounds of them; else 128 x 128, two blocks.  Us, 256 / 128:
  // 4096^3 37 / 41 (256 blocks); 9000 x 13824 x 5120 348 / 402 (7.6 rounds of 8); 3000 x
  // 13824 x 5120 114 / 125 (2.5 of 3); 5000 x 5120 x 5120 74 / 80 (400 blocks); 6000 x
  // 4096 x 4096 61 / 59 (384); 4096 x 5120 x 13824 162 / 148 (320); 2048 x 4096 x 4096
  // 34 / 23 (half of one).
  const int64_t small = ((int64_t)tokens + 127) / 128 * (((int64_t)rows + 63) / 64);
  const int64_t large = ((int64_t)tokens + 255) / 256 * (((int64_t)rows + 255) / 256);
  p.tile = small <= 256 ? 64 : 4 * large > 3 * ((large + 255) / 256 * 256) ? 256 : 128;
  if (p.quantize) {
    p.x_vals = mx_vals_bytes(tokens, cols);
    p.x_scales = mx_scales_bytes(tokens, cols);
  }
  p.workspace_bytes = p.x_vals + p.x_scales;
  return p;
}

PromptPlan prompt_plan(const i4s_prompt_args &a) {
  PromptPlan p{};
  const int64_t rows = (int64_t)a.max_q * (a.q_heads / a.kv_heads);
  const int64_t pairs = (int64_t)a.kv_heads * (a.num_seqs > 0 ? a.num_seqs : 1), large = (rows + 255) / 256;
  // Blocks of 32 rows where those are all; of 256 (head dimension 128) for long keys,
  // where their ends weigh little, and some rounds of the 256 compute units; else 128.
  // Us, 256 / 128: 8191 tokens x 40 heads 661 / 679, x 16 (512 blocks of 256) 265 / 289;
  // 16384 x 16 991 / 1036; 6144 x 40 394 / 427; 4096 x 64 297 / 304, x 40 196 / 192; 16 x up
  // to 2047 tokens, 8 x 4 heads 345 / 321, x up to 1023 146 / 114; head dimension 64, 4096
  // x 40 131 / 114.
  const int64_t len = a.max_k > 0 && a.max_k < a.num_keys ? a.max_k : a.num_keys;
  p.rows = rows <= kPromptRows ? kPromptRows
           : a.head_dim == 128 && len >= 6144 && pairs * large >= 448 ? 8 * kPromptRows : 4 * kPromptRows;
  p.row_blocks = (int32_t)((rows + p.rows - 1) / p.rows);
  const int64_t units = p.row_blocks * pairs;
  // Pairs of sequence and KV head that run together: as many as keep their keys in
  // the L2s, but enough that long rows of one are done next to short ones of others.
  // Us, for 8 / 160 / 320 blocks of an XCD and all: 16 x up to 2047 tokens, 8 x 4 heads
  // 321 / 321 / 325 / 421; 8191 tokens, 40 heads 730 / 667 / 667 / 668; 16 x 1024 tokens,
  // 40 heads 299 / 286 / 301 / 316.
  p.group = 8 * ((160 + p.row_blocks - 1) / p.row_blocks);
  // The keys in pieces for about two blocks of 128 rows a compute unit, or one of
  // 32, but none shorter than 512 keys: partial results are fp32 and need a second
  // launch.  Us, for half as many / these / twice as many: 65536 keys, 8 x 4 rows 63 /
  // 49 / 52; 128 tokens behind 32639, 8 x 4 heads 100 / 93 / 104; 4 x 16 behind 8176
  // 41 / 40 / 51.  512 tokens, 40 heads in one piece / two of 256 keys 19 / 43; 1024
  // tokens, 8 heads in one / of 512 / 256 26 / 30 / 26; 2048 tokens in one / these, 8
  // heads 47 / 49, 16 heads (256 blocks, two pieces) 48 / 82: not worth it there.
  const int64_t want = clamp_to<int64_t>((p.rows == kPromptRows ? 256 : 512) / units, 1, len > 512 ? (len + 511) / 512 : 1);
  const int64_t per = clamp_to<int64_t>((len + want * kPromptKeys - 1) / (want * kPromptKeys), 1, (1 << 30) / kPromptKeys);
  p.chunk = (int32_t)(per * kPromptKeys);
  p.splits = (int32_t)clamp_to<int64_t>((len + p.chunk - 1) / p.chunk, 1, kMaxPromptSplits);
  if (p.splits > 1)
    p.workspace_bytes = (uint64_t)p.splits * a.num_tokens * a.q_heads * (a.head_dim + 2) * sizeof(float);
  return p;
}

}  // namespace i4s

extern "C" {

i4s_status i4s_mx_sizes(int32_t rows, int32_t cols, i4s_mx_buffers *out) {
  if (!out) return fail(I4S_ERR_INVALID_ARGUMENT, "out is NULL");
  const i4s_status st = check_mx_shape(rows, cols);
  if (st != I4S_OK) return st;
  out->vals = i4s::mx_vals_bytes(rows, cols);
  out->scales = i4s::mx_scales_bytes(rows, cols);
  return I4S_OK;
}

i4s_status i4s_mx_quantize(const void *x, int32_t dtype, int64_t stride, const i4s_mx *out, void *stream) {
  i4s_status st = check_mx(out, "out", true);
  if (st != I4S_OK) return st;
  st = check_half(dtype, "dtype");
  if (st != I4S_OK) return st;
  st = check_row_stride(stride, out->cols, "stride");
  if (st != I4S_OK) return st;
  if (out->rows == 0) return I4S_OK;
  if (!x || !aligned(x, 16)) return fail(I4S_ERR_INVALID_ARGUMENT, "x is NULL or not 16-byte aligned");
  const Span outs[] = {vals_of(*out, "vals"), scales_of(*out, "scales")};
  const Span ins[] = {{x, 2ull * ((out->rows - 1) * (uint64_t)stride + out->cols), "x"}};
  st = check_spans(outs, ins);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  const i4s::MxQuantizeArgs a{x, stride, out->rows, out->cols, out->vals, out->scales};
  const hipError_t e = i4s::launch_mx_quantize(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "mx_quantize launch");
}

i4s_status i4s_mx_read(const i4s_mx *m, int32_t dtype, void *out, void *stream) {
  i4s_status st = check_mx(m, "m", true);
  if (st != I4S_OK) return st;
  st = check_any(dtype, "dtype");
  if (st != I4S_OK) return st;
  if (m->rows == 0) return I4S_OK;
  if (!out || !aligned(out, 16)) return fail(I4S_ERR_INVALID_ARGUMENT, "out is NULL or not 16-byte aligned");
  const Span outs[] = {{out, (uint64_t)m->rows * m->cols * dtype_size(dtype), "out"}};
  const Span ins[] = {vals_of(*m, "vals"), scales_of(*m, "scales")};
  st = check_spans(outs, ins);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;
  const i4s::MxReadArgs a{m->vals, m->scales, m->rows, m->cols, out};
  const hipError_t e = i4s::launch_mx_read(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "mx_read launch");
}

i4s_status i4s_mx_product_workspace_size(const i4s_mx_product_args *a, uint64_t *bytes) {
  if (!bytes) return fail(I4S_ERR_INVALID_ARGUMENT, "bytes is NULL");
  const i4s_status st = check_product(a);
  if (st != I4S_OK) return st;
  *bytes = a->tokens && a->w->rows ? i4s::mx_product_plan(a->tokens, a->w->rows, a->w->cols, a->x != nullptr).workspace_bytes : 0;
  return I4S_OK;
}

i4s_status i4s_mx_product(const i4s_mx_product_args *a, void *stream) {
  i4s_status st = check_product(a);
  if (st != I4S_OK) return st;
  const i4s_mx &w = *a->w;
  st = check_mx(&w, "w", true);
  if (st != I4S_OK) return st;
  st = check_any(a->y_dtype, "y_dtype");
  if (st != I4S_OK) return st;
  const int size = dtype_size(a->y_dtype);
  if (a->y_stride < w.rows || a->y_stride > kMaxStride)
    return fail(I4S_ERR_INVALID_ARGUMENT, "y_stride=%lld must be at least w's rows=%d, at most 2^40", (long long)a->y_stride,
                w.rows);
  if (a->x) {
    st = check_mx(a->x, "x", true);
    if (st != I4S_OK) return st;
    if (a->x->rows != a->tokens || a->x->cols != w.cols)
      return fail(I4S_ERR_INVALID_ARGUMENT, "x is [%d][%d], tokens=%d and w's cols=%d", a->x->rows, a->x->cols, a->tokens,
                  w.cols);
  } else {
    st = check_half(a->x_dtype, "x_dtype");
    if (st != I4S_OK) return st;
    st = check_row_stride(a->x_stride, w.cols, "x_stride");
    if (st != I4S_OK) return st;
  }
  if (a->tokens == 0 || w.rows == 0) return I4S_OK;
  if (!a->x && (!a->x_values || !aligned(a->x_values, 16)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "x_values is NULL or not 16-byte aligned");
  if (!a->y || !aligned(a->y, size)) return fail(I4S_ERR_INVALID_ARGUMENT, "y is NULL or not aligned to its element");
  const i4s::MxProductPlan p = i4s::mx_product_plan(a->tokens, w.rows, w.cols, a->x != nullptr);
  if (p.workspace_bytes) {
    if (!a->workspace || !aligned(a->workspace, 16))
      return fail(I4S_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (a->workspace_bytes < p.workspace_bytes)
      return fail(I4S_ERR_WORKSPACE_TOO_SMALL, "workspace has %llu bytes, %llu needed",
                  (unsigned long long)a->workspace_bytes, (unsigned long long)p.workspace_bytes);
  }
  const Span outs[] = {{a->y, ((uint64_t)(a->tokens - 1) * a->y_stride + w.rows) * size, "y"},
                       {a->workspace, p.workspace_bytes, "workspace"}};
  const i4s_mx none{};
  const Span ins[] = {vals_of(w, "w's vals"), scales_of(w, "w's scales"),
                      a->x ? vals_of(*a->x, "x's vals") : Span{none.vals, 0, "x"},
                      a->x ? scales_of(*a->x, "x's scales")
                           : Span{a->x_values, 2ull * ((a->tokens - 1) * (uint64_t)a->x_stride + w.cols), "x_values"}};
  st = check_spans(outs, ins);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;

  i4s::MxProductKernelArgs k{};
  k.w_vals = w.vals, k.w_scales = w.scales, k.rows = w.rows, k.cols = w.cols;
  k.tokens = a->tokens, k.y = a->y, k.y_stride = a->y_stride;
  uint8_t *ws = static_cast<uint8_t *>(a->workspace);
  if (a->x) {
    k.x_vals = a->x->vals, k.x_scales = a->x->scales;
  } else if (p.quantize) {
    const i4s::MxQuantizeArgs q{a->x_values, a->x_stride, a->tokens, w.cols, ws, ws + p.x_vals};
    const hipError_t e = i4s::launch_mx_quantize(q, a->x_dtype, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return device_error(e, "mx_quantize launch");
    k.x_vals = ws, k.x_scales = ws + p.x_vals;
  } else {
    k.x = a->x_values, k.x_stride = a->x_stride, k.x_dtype = a->x_dtype;
  }
  const hipError_t e = i4s::launch_mx_product(k, p, a->y_dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "mx_product launch");
}

i4s_status i4s_prompt_attention_workspace_size(const i4s_prompt_args *a, uint64_t *bytes) {
  if (!bytes) return fail(I4S_ERR_INVALID_ARGUMENT, "bytes is NULL");
  const i4s_status st = check_prompt(a);
  if (st != I4S_OK) return st;
  *bytes = a->num_tokens && a->num_seqs ? i4s::prompt_plan(*a).workspace_bytes : 0;
  return I4S_OK;
}

i4s_status i4s_prompt_attention(const i4s_prompt_args *a, void *stream) {
  i4s_status st = check_prompt(a);
  if (st != I4S_OK) return st;
  st = check_strides(a->q_token_stride, a->q_head_stride, "q");
  if (st != I4S_OK) return st;
  st = check_strides(a->k_token_stride, a->k_head_stride, "k");
  if (st != I4S_OK) return st;
  st = check_strides(a->v_token_stride, a->v_head_stride, "v");
  if (st != I4S_OK) return st;
  if (a->num_tokens == 0 || a->num_seqs == 0) return I4S_OK;
  if (!a->q || !aligned(a->q, 16) || !a->out || !aligned(a->out, 16))
    return fail(I4S_ERR_INVALID_ARGUMENT, "q or out is NULL or not 16-byte aligned");
  if (a->num_keys && (!a->k || !aligned(a->k, 16) || !a->v || !aligned(a->v, 16)))
    return fail(I4S_ERR_INVALID_ARGUMENT, "k or v is NULL or not 16-byte aligned");
  if (!a->q_start != !a->k_start || (!a->q_start && a->num_seqs != 1))
    return fail(I4S_ERR_INVALID_ARGUMENT, "q_start or k_start is NULL; both may be for num_seqs=1, not %d", a->num_seqs);
  if (!aligned(a->q_start, 4) || !aligned(a->k_start, 4) || !aligned(a->lse, 4))
    return fail(I4S_ERR_INVALID_ARGUMENT, "q_start, k_start or lse is not 4-byte aligned");
  const i4s::PromptPlan p = i4s::prompt_plan(*a);
  if (p.workspace_bytes) {
    if (!a->workspace || !aligned(a->workspace, 16))
      return fail(I4S_ERR_INVALID_ARGUMENT, "workspace is NULL or not 16-byte aligned");
    if (a->workspace_bytes < p.workspace_bytes)
      return fail(I4S_ERR_WORKSPACE_TOO_SMALL, "workspace has %llu bytes, %llu needed",
                  (unsigned long long)a->workspace_bytes, (unsigned long long)p.workspace_bytes);
  }
  const uint64_t rows = (uint64_t)a->num_tokens * a->q_heads;
  const Span outs[] = {{a->out, 2 * rows * a->head_dim, "out"},
                       {a->lse, 4 * rows, "lse"},
                       {a->workspace, p.workspace_bytes, "workspace"}};
  const Span ins[] = {
      {a->q, extent(a->num_tokens, a->q_token_stride, a->q_heads, a->q_head_stride, a->head_dim), "q"},
      {a->k, extent(a->num_keys, a->k_token_stride, a->kv_heads, a->k_head_stride, a->head_dim), "k"},
      {a->v, extent(a->num_keys, a->v_token_stride, a->kv_heads, a->v_head_stride, a->head_dim), "v"},
      {a->q_start, a->q_start ? 4ull * (a->num_seqs + 1) : 0, "q_start"},
      {a->k_start, a->k_start ? 4ull * (a->num_seqs + 1) : 0, "k_start"}};
  st = check_spans(outs, ins);
  if (st != I4S_OK) return st;
  st = check_device();
  if (st != I4S_OK) return st;

  i4s::PromptKernelArgs k{};
  k.q = a->q, k.k = a->k, k.v = a->v;
  k.q_token = a->q_token_stride, k.q_head = a->q_head_stride;
  k.k_token = a->k_token_stride, k.k_head = a->k_head_stride;
  k.v_token = a->v_token_stride, k.v_head = a->v_head_stride;
  k.kv_heads = a->kv_heads, k.share = a->q_heads / a->kv_heads;
  k.num_tokens = a->num_tokens, k.num_keys = a->num_keys, k.num_seqs = a->num_seqs;
  k.max_q = a->max_q, k.causal = a->causal;
  k.row_blocks = p.row_blocks, k.group = p.group, k.splits = p.splits, k.chunk = p.chunk;
  k.scale_log2 = (float)std::fmin((double)a->scale * 1.4426950408889634, FLT_MAX);
  k.q_start = a->q_start, k.k_start = a->k_start, k.out = a->out, k.lse = a->lse;
  k.part_o = static_cast<float *>(a->workspace);
  k.part_ml = p.workspace_bytes ? k.part_o + (uint64_t)p.splits * rows * a->head_dim : nullptr;
  const hipError_t e = i4s::launch_prompt_attention(k, p, a->head_dim, a->dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? I4S_OK : device_error(e, "prompt_attention launch");
}

}  // extern "C"
