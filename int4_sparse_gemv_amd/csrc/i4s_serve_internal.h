// Internal declarations of the serving operators of libi4s (KV cache,
// attention, token scores), shared by their host layer (i4s_serve_api.cpp)
// and their kernels.  Not part of the public ABI.
#pragma once

#include "i4s_internal.h"
#include "i4s_serve.h"

namespace i4s {

// A length or slot from device memory, moved into [lo, hi].
template <typename T>
__host__ __device__ inline T clamp_to(T v, T lo, T hi) {
  return v < lo ? lo : (v > hi ? hi : v);
}

// log2 of a page size (16 .. 256).
inline int page_shift(int32_t page_size) { return __builtin_ctz((unsigned)page_size); }

// ---------------------------------------------------------------------------
// block tables and slot maps, cache writes and reads (i4s_kv.hip)

struct ExtendArgs {
  int32_t *table;
  int32_t n, width, shift;
  const int32_t *lens, *new_lens, *free_pages;
  int32_t free_entries;
  const int32_t *free_count;
  int32_t capacity;
  int32_t *lens_out, *q_start, *slots, *positions, *free_count_out, *flags;
};
hipError_t launch_kv_extend(const ExtendArgs &a, hipStream_t stream);

struct AppendArgs {
  i4s_kv_cache cache;
  const void *k, *v;
  int64_t k_token, k_head, v_token, v_head;  // strides in elements
  const int32_t *slots;
  int32_t tokens;
};
hipError_t launch_kv_append(const AppendArgs &a, int32_t dtype, hipStream_t stream);

struct ReadArgs {
  i4s_kv_cache cache;
  const int32_t *slots;
  int32_t tokens;
  void *k, *v;
};
hipError_t launch_kv_read(const ReadArgs &a, int32_t dtype, hipStream_t stream);

// ---------------------------------------------------------------------------
// attention (i4s_attention.hip)

// Launch shape of an attention call: 16 * row_tiles query rows (tokens x
// query heads of one KV head) per block, row_blocks such blocks per sequence
// and KV head, the keys in `splits` pieces of `chunk` keys (the last takes
// what is left), `waves` waves per block.
struct AttentionPlan {
  int row_tiles, row_blocks, splits, chunk, waves;
  uint64_t workspace_bytes;
};
AttentionPlan attention_plan(const i4s_attention_args &a);

constexpr int kMaxSplits = 4096;

// How far (log2) a row's largest probability may pass 1 before its reference follows.
constexpr int kAttentionSlack = 8;

// Keys of one step of a wave.
constexpr int kStepKeys = 32;

struct AttentionKernelArgs {
  const uint8_t *k_vals, *v_vals;
  const uint16_t *k_scales, *v_scales;
  int32_t num_pages, shift, kv_heads, share;
  const void *q;
  int64_t q_token, q_head;
  int32_t num_tokens, num_seqs;
  const int32_t *table;
  int32_t width;
  const int32_t *lens, *q_start;
  int32_t max_q, row_blocks, splits, chunk;
  float scale_log2;  // scale * log2(e)
  float slack;       // kAttentionSlack in units of scores
  const int64_t *tree;
  void *out;
  float *lse;
  float *part_o;     // [splits][num_tokens * q_heads][D]
  float *part_ml;    // [splits][num_tokens * q_heads][2]: reference, sum
};
hipError_t launch_attention(const AttentionKernelArgs &a, const AttentionPlan &p, int32_t head_dim,
                            int32_t group_size, int32_t dtype, hipStream_t stream);

// ---------------------------------------------------------------------------
// token scores (i4s_logprobs.hip)

// Launch shape of a call: blocks of 256 threads, each over a piece of
// `segments` segments (32 values a thread) of a row, `splits` pieces a row (1:
// one launch).
constexpr int kMaxLogprobsSplits = 64;  // the lanes of a wave join them
constexpr int kSegment = 256 * 32;
constexpr int kMaxSegments = 32;        // 1 KB of LDS each
struct LogprobsPlan {
  int splits, segments;
  uint64_t workspace_bytes;
};
LogprobsPlan logprobs_plan(int32_t dtype, int32_t rows, int32_t vocab, int32_t top_k);

struct LogprobsArgs {
  const void *logits;
  int32_t rows, vocab;
  int64_t stride;
  const int64_t *tokens;
  int32_t top_k;
  float *logprobs, *entropy;
  int32_t *top_ids;
  float *top_logprobs;
  float *part_stats;    // [rows][splits][4]: max, reference, sum, weighted sum
  uint64_t *part_keys;  // [rows][splits][top_k]
};
hipError_t launch_token_logprobs(const LogprobsArgs &a, const LogprobsPlan &p, int32_t dtype, hipStream_t stream);

}  // namespace i4s
