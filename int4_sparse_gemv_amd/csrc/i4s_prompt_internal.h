// Internal declarations of the prompt's operators of libi4s (microscaled
// format, products, attention of whole prompts), shared by their host layer
// (i4s_prompt_api.cpp) and their kernels.  Not part of the public ABI.
#pragma once

#include "i4s_prompt.h"
#include "i4s_serve_internal.h"

namespace i4s {

// ---------------------------------------------------------------------------
// the microscaled format (i4s_mx.hip)

constexpr int kMxRows = 16;            // rows of a tile
constexpr int kMxStep = 128;           // columns of a tile: one matrix instruction
constexpr int kMxTileBytes = 1024;     // values of a tile
constexpr int kMxGroup = 512;          // columns whose scales lie together
constexpr int kMxGroupBytes = 256;     // scales of 16 rows x 512 columns
constexpr uint32_t kMxNaN = 255;       // scale byte of a block that is not finite

__host__ __device__ inline int32_t mx_row_tiles(int32_t rows) { return (rows + kMxRows - 1) / kMxRows; }
__host__ __device__ inline int32_t mx_steps(int32_t cols) { return 2 * ((cols + 255) / 256); }
__host__ __device__ inline int32_t mx_groups(int32_t cols) { return (cols + kMxGroup - 1) / kMxGroup; }
inline uint64_t mx_vals_bytes(int32_t rows, int32_t cols) {
  return (uint64_t)mx_row_tiles(rows) * mx_steps(cols) * kMxTileBytes;
}
inline uint64_t mx_scales_bytes(int32_t rows, int32_t cols) {
  return (uint64_t)mx_row_tiles(rows) * mx_groups(cols) * kMxGroupBytes;
}

struct MxQuantizeArgs {
  const void *x;
  int64_t stride;
  int32_t rows, cols;
  uint8_t *vals, *scales;
};
hipError_t launch_mx_quantize(const MxQuantizeArgs &a, int32_t dtype, hipStream_t stream);

struct MxReadArgs {
  const uint8_t *vals, *scales;
  int32_t rows, cols;
  void *out;
};
hipError_t launch_mx_read(const MxReadArgs &a, int32_t dtype, hipStream_t stream);

// ---------------------------------------------------------------------------
// products (i4s_mx_product.hip)

// How a product runs.  `quantize`: the 16-bit tokens are quantized into the
// workspace first (otherwise the kernel does it on the way).  Few: blocks of
// `waves` waves that split the columns of `row_tiles` weight tiles and up to
// four token tiles.  Else blocks of `tile` x `tile` outputs, or 64 x 128.  The order of the
// sums follows `few` and `waves`, which do not depend on how the tokens are given.
struct MxProductPlan {
  bool quantize, few;
  int32_t token_tiles;       // 16-token tiles
  int32_t row_tiles, waves;  // few: (1, 8), (2, 8), (2, 4), or (4, 8) for 16-bit tokens
  int32_t tile;              // 64, 128 or 256
  uint64_t x_vals, x_scales;  // workspace bytes of the quantized tokens
  uint64_t workspace_bytes;
};
MxProductPlan mx_product_plan(int32_t tokens, int32_t rows, int32_t cols, bool x_given);

struct MxProductKernelArgs {
  const uint8_t *w_vals, *w_scales;
  int32_t rows, cols;
  const uint8_t *x_vals, *x_scales;
  const void *x;          // 16-bit tokens, or null
  int64_t x_stride;
  int32_t x_dtype;
  int32_t tokens;
  void *y;
  int64_t y_stride;
};
hipError_t launch_mx_product(const MxProductKernelArgs &a, const MxProductPlan &p, int32_t y_dtype, hipStream_t stream);

// ---------------------------------------------------------------------------
// attention of whole prompts (i4s_prompt_attention.hip)

// Launch shape: blocks of 128 or 256 query rows (tokens x query heads of one KV
// head), or of up to 32 that a sequence and KV head has in all, row_blocks such
// blocks a sequence and KV head, the keys in `splits` pieces of `chunk` keys (the
// last takes what is left).
struct PromptPlan {
  int32_t rows;  // of a block
  int32_t row_blocks;
  int32_t group;  // pairs of sequence and KV head that run together
  int32_t splits, chunk;
  uint64_t workspace_bytes;
};
PromptPlan prompt_plan(const i4s_prompt_args &a);

constexpr int kPromptRows = 32;  // query rows of a wave
constexpr int kMaxPromptSplits = 512;
constexpr int kPromptKeys = 64;  // pieces of the keys are multiples of it

struct PromptKernelArgs {
  const void *q, *k, *v;
  int64_t q_token, q_head, k_token, k_head, v_token, v_head;  // strides in elements
  int32_t kv_heads, share;
  int32_t num_tokens, num_keys, num_seqs, max_q, causal;
  int32_t row_blocks, group, splits, chunk;
  float scale_log2;
  const int32_t *q_start, *k_start;  // null: one sequence
  void *out;
  float *lse;
  float *part_o;   // [splits][num_tokens * q_heads][D]
  float *part_ml;  // [splits][num_tokens * q_heads][2]: the reference (a q . k, at most
                   // 8 / scale_log2 below the largest), the sum
};
hipError_t launch_prompt_attention(const PromptKernelArgs &a, const PromptPlan &p, int32_t head_dim, int32_t dtype,
                                   hipStream_t stream);

}  // namespace i4s
