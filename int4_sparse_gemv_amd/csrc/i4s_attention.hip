// Attention of a few query tokens per sequence over the 4-bit paged KV cache
// (format: include/i4s_serve.h), for gfx950.
//
// A block takes the query rows (tokens x query heads) of one sequence that
// read one KV head, up to 16 * RT of them, and a piece of the keys; its waves
// take steps of 32 keys in turn, each with a softmax of its own (running
// maximum and sum), and join at the end.  Pieces join in a second launch.
//
// Everything is computed transposed, so that no value moves between lanes on
// the way: lane l = i + 16a of a wave.
//   S^T = K Q^T: v_mfma_f32_16x16x32 with 16 keys as rows, 16 query rows as
//     columns and 32 channels.  A lane loads key i's words of the channels
//     32j + 8a .. +7, j = 0..D/32-1: neighbours in the format, so that one
//     wide load per lane covers 16 keys without a gap.  The tile comes out
//     with query row i and keys 4a .. 4a+3 in lane l.
//   O^T = V^T P^T: v_mfma_f32_16x16x32 with 16 channels as rows, 16 query
//     rows as columns and 32 keys.  Its B operand wants query row i and 8
//     keys in lane l: take the keys 4a .. 4a+3 of two tiles, and P is in
//     place as S came out.  Its A operand wants channel i (of 16) and the
//     same 8 keys: the format keeps the words of channel i for 4 neighbouring
//     tokens together, and a v_perm_b32 of two tokens' words puts their
//     halves into one dword, whose nibbles then widen to pairs (token, next
//     token) of one channel.
// 4-bit values are widened with bit operations: for K the nibble goes into
// the mantissa of 16.0 (16 + u, exact in fp16 and bf16), and the offset 24 =
// 16 + 8 leaves with the sum: the products start from -24 * sum(q) of the
// group's channels, in fp32, so that a score's rounding error follows sum |q|
// (|k| + 24 s), s K's scale, not the score.  The sum over groups starts from minus
// the row's reference (a score near the row's running maximum): exponents are
// differences of scores, taken before they are scaled, and stay small however far
// from 0 the scores lie.
//
// Scales: K's multiply the fp32 sums of a group's channels; V's multiply the
// probabilities, in fp32, and the products go to the matrix instruction as two
// bf16 terms, the value rounded and what that left, rounded: 2^-16 of it, at any
// size, since bf16 has fp32's exponents.  (One fp16 term made a third more error
// than an fp16 output's own rounding, and lost whole bits of values that lay far
// below the largest product of probability and scale, in any group.)  V's
// nibbles become 16 + u for even tokens and -(31 - u) for odd ones, exact in bf16
// too: the value + 24 and - 23, two offsets that mostly cancel; what they add
// is summed beside (`extra`, v_dot2) and leaves at the end.
// Up to 8 rows fill half of the 16 columns only: there the other half takes the
// second terms of the same rows (PAIR), at no cost in matrix instructions.  Us,
// one term in fp16 / two in turn / two side by side: 16 x up to 4095 keys, 32
// heads 40.3 / 46.9 / 41.9, 131071 keys, 8 heads x 4 rows 34.8 / 39.9 / 36.0.
//
// Where the probabilities are many (row tiles x groups >= 8) V's scales go to
// V's values instead.  For fp16 outputs probabilities and scaled values are
// two fp16 terms each (a 4-bit value times a scale is exact in two, and the
// product of the two second terms, 2^-22, is left out); for bf16 outputs, whose
// own rounding is eight times as coarse, one each: 2^-11 of either.  Us, 512 x up
// to 16384 keys, 32 rows, G = 32: 197 with one term each, 240 with two, 287 with
// V's scales of four groups on the probabilities.  The probability of the key that
// set a row's reference is 2^7 at least and the smallest step of fp16 2^-31 of that:
// whatever else a wave sees, a key's value loses at most half of it.
//
// Bound by: memory's latency and the vector units together while few query rows
// share a key (a key of one head is D + 4D/G bytes; a plain read of such sizes
// reaches 6.7 TB/s, a copy 4.8): 512 x up to 4095 keys, one row, D = 128, G = 64: 170
// MB in 41 us, 4.2 TB/s, vector instructions in 47 % of the cycles; 8 x 131071
// keys, 4 rows: 143 MB in 31 us, 4.6 TB/s, and 4.0 us for the join of its 32
// pieces.  With 32 rows a key neither is full: 512 x up to 16384 keys, G = 32, bf16:
// 675 MB in 193 us, 3.5 TB/s, vector units 49 %, matrix units 15 %, two waves a SIMD
// (what the registers leave).  Short contexts: 6 us for any (launch, page numbers,
// queries, joining the waves) and 1.5 us for each step of a wave, 256 keys: 32 x
// 1 / 256 / 512 / 1023 keys 6.2 / 7.8 / 9.4 / 12.  Many query tokens: each block
// of 16 rows reads and widens every key, also those that its rows do not see: 2048
// causal tokens of 40 heads 0.3 ms, 8191 4.0 ms, 172 TFLOP/s of what counts.

#include <float.h>

#include <type_traits>

#include "i4s_gemv_common.h"
#include "i4s_serve_internal.h"

namespace i4s {
namespace {

typedef _Float16 hf8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef uint32_t w4_t __attribute__((ext_vector_type(4)));
typedef uint32_t w2_t __attribute__((ext_vector_type(2)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

// fp16 and bf16 query types: the matrix instruction, and how nibble p (and
// p + 4, 16 bits on) of a word becomes 16 + u.
struct F16 {
  typedef hf8_t vec;
  static constexpr uint32_t kMask = 0x03C003C0u, kSixteen = 0x4C004C00u;
  static constexpr int kShift = 6;  // left shift of nibble 0
  static constexpr bool kCoarse = false;
  static __device__ f4_t mfma(vec a, vec b, f4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0); }
  static __device__ float to_float(uint32_t bits) { return fp16_bits_to_float(bits); }
  static __device__ uint32_t from_float(float f) { return float_to_fp16_bits(f); }
};
struct BF16 {
  typedef bf8_t vec;
  static constexpr uint32_t kMask = 0x00780078u, kSixteen = 0x41804180u;
  static constexpr int kShift = 3;
  static constexpr bool kCoarse = true;  // its rounding, next to fp16's
  static __device__ f4_t mfma(vec a, vec b, f4_t c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }
  static __device__ float to_float(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
  static __device__ uint32_t from_float(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};

constexpr float kOffset = 24.0f;   // 16 of the widening + 8 of the nibble
// A row's reference is a score near its running maximum: its first key's step
// sets it, and it follows the maximum only when that has grown by more than
// kAttentionSlack (log2): with 16 rows or more a wave some row's maximum grows in most
// steps, and every change scales all of O.
// Below every reference: where rows without keys join others.
constexpr float kLowest = -FLT_MAX;

// (a & m) | c.  In one v_and_or_b32 if the constants are in registers (the
// instruction takes no literal): masks and magic numbers are made once, hidden
// from the optimizer.  The instruction itself is left to the compiler: it does
// not see which registers inline asm writes when it places the waits that a
// VALU write to a matrix instruction's registers needs.
__device__ inline uint32_t mask_or(uint32_t a, uint32_t m, uint32_t c) { return (a & m) | c; }
__device__ inline uint32_t in_sgpr(uint32_t v) {
  asm("" : "+s"(v));
  return v;
}
__device__ inline uint32_t in_vgpr(uint32_t v) {
  asm("" : "+v"(v));
  return v;
}

// Masks and magic numbers of the widening.
struct Constants {
  uint32_t k_mask, k_sixteen, v_mask, v_pair, v_low, v_high, v_magic;
};

// Nibbles p and p + 4 of w, p = 0..3, as exact bf16 pairs (16 + u, -(31 - u)):
// the values + 24 and - 23 (one v_bitop3_b32 each after the shift).
__device__ inline void widen_v(uint32_t w, const Constants &k, uint32_t q[4]) {
  q[0] = (w << 3 & k.v_mask) ^ k.v_pair;
  q[1] = (w >> 1 & k.v_mask) ^ k.v_pair;
  q[2] = (w >> 5 & k.v_mask) ^ k.v_pair;
  q[3] = (w >> 9 & k.v_mask) ^ k.v_pair;
}
constexpr uint32_t kPairBias = 0xC1B841C0u;  // (24, -23) in bf16

__device__ inline float dot2(bf2_t a, uint32_t b, float c) {
  return __builtin_amdgcn_fdot2_f32_bf16(a, __builtin_bit_cast(bf2_t, b), c, false);
}

// Nibbles p and p + 4 of w, p = 0..3, as exact fp16 pairs u - 8: the nibble
// goes into the mantissa of 1024 at its place 0..3 or 4..7.
__device__ inline void widen_v(uint32_t w, const Constants &k, h2_t q[4]) {
  const uint32_t t = w >> 8;
  const h2_t bias = {(_Float16)-1032.0f, (_Float16)-1032.0f};
  const h2_t sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
  const h2_t bias16 = {(_Float16)-72.0f, (_Float16)-72.0f};
  q[0] = as_h2(mask_or(w, k.v_low, k.v_magic)) + bias;
  q[2] = as_h2(mask_or(t, k.v_low, k.v_magic)) + bias;
  q[1] = __builtin_elementwise_fma(as_h2(mask_or(w, k.v_high, k.v_magic)), sixteenth, bias16);
  q[3] = __builtin_elementwise_fma(as_h2(mask_or(t, k.v_high, k.v_magic)), sixteenth, bias16);
}

// The eight channels of a K word as 16 + u.
template <typename T>
__device__ inline typename T::vec widen_k(uint32_t w, const Constants &k) {
  w4_t r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const int s = T::kShift - 4 * p;
    r[p] = mask_or(s >= 0 ? w << (s & 31) : w >> (-s & 31), k.k_mask, k.k_sixteen);
  }
  return __builtin_bit_cast(typename T::vec, r);
}

// Maximum and sum over the four lanes i, i + 16, i + 32, i + 48.  (The bits of
// a vector's element are copied out before they are taken for a float:
// __builtin_bit_cast of the element itself reads element 0.)
struct Two {
  float a, b;
};
__device__ inline Two halves_of(float v) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t a = s[0], b = s[1];
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
__device__ inline Two quarters_of(float v) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane16_swap(x, x, false, false);
  const uint32_t a = s[0], b = s[1];
  return {__builtin_bit_cast(float, a), __builtin_bit_cast(float, b)};
}
// v_maximum(3)_f32: unlike fmaxf it passes a NaN on, so its operands need no
// quieting first.
__device__ inline float maximum(float a, float b) { return __builtin_elementwise_maximum(a, b); }
__device__ inline float max4(float v) {
  const Two h = halves_of(v), q = quarters_of(maximum(h.a, h.b));
  return maximum(q.a, q.b);
}
__device__ inline float sum4(float v) {
  const Two h = halves_of(v), q = quarters_of(h.a + h.b);
  return q.a + q.b;
}

// Natural logarithm of a row's sum of exponentials, from its reference and the sum
// relative to that; -inf for a row without keys.
__device__ inline float lse_of(float reference, float sum, float scale_log2) {
  return sum == 0.0f ? -INFINITY : fmaf(reference, scale_log2, __builtin_amdgcn_logf(sum)) * 0.6931471805599453f;
}

// What a block works on: its sequence's lengths, all made safe.
struct Work {
  int len, q0, q_len, ctx, used;
};
__device__ inline Work work_of(const AttentionKernelArgs &a, int seq) {
  Work w;
  w.len = (int)clamp_to<int64_t>(a.lens[seq], 0, (int64_t)a.width << a.shift);
  w.q0 = seq;
  int q1 = seq + 1;
  if (a.q_start) {
    w.q0 = clamp_to(a.q_start[seq], 0, a.num_tokens);
    q1 = clamp_to(a.q_start[seq + 1], w.q0, a.num_tokens);
  }
  w.q_len = q1 - w.q0;
  w.ctx = w.len - w.q_len;
  w.used = clamp_to((int)(((int64_t)w.len + a.chunk - 1) / a.chunk), 1, a.splits);
  return w;
}

// One step of 32 keys (two tiles of 16) of a wave in LDS.  The loads go there
// directly (global_load_lds, 16 bytes a lane, lane after lane), so a step on
// its way costs no registers.  Where a lane's share of a tile is 16 bytes or
// more its 16-byte pieces lie at [piece][lane]; for D = 64 the tile lies as in
// the cache.
template <int D, int G>
struct Stage {
  static constexpr int NG = D / G;
  static constexpr int kTile = 8 * D;               // bytes of K, and of V, of 16 keys
  static constexpr int kScales = 32 * NG;           // bytes of K's scales, and of V's, of 16 keys
  static constexpr int kV = 2 * kTile, kKs = 4 * kTile, kVs = kKs + 2 * kScales;
  static constexpr int kBytes = kVs + 2 * kScales;  // 32 D + 128 NG
  static constexpr int kLoads = (D == 64 ? 2 : D / 32) + 1;  // load instructions of a step
  static constexpr int kVWords = D == 256 ? 8 : 4;  // V words of a lane and tile
};
constexpr int kStages = 2;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
typedef const __attribute__((address_space(4))) int32_t scalar_int32;  // read with scalar loads

// Keys that one block alone reads go past the caches (`once`), those that the
// blocks of other query rows read too do not: 8 x 131071 keys, 4 rows: 34.7 /
// 32.3 us without / with; 128 x 4000, 128 rows: 104 / 122.
constexpr int kNonTemporal = 2;
template <bool ONCE>
__device__ inline void copy16(const void *from, char *to) {
  __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)to, 16, 0, ONCE ? kNonTemporal : 0);
}

// Waits until at most N vector loads are on their way (s_waitcnt vmcnt).
template <int N>
__device__ inline void wait_loads() {
  issue_fence();
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
  issue_fence();
}

template <int N>
__device__ inline void read_words(uint32_t *to, const char *from) {
  if constexpr (N == 2) {
    const w2_t x = *reinterpret_cast<const w2_t *>(from);
    to[0] = x.x, to[1] = x.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const w4_t x = reinterpret_cast<const w4_t *>(from)[i];
      to[4 * i] = x.x, to[4 * i + 1] = x.y, to[4 * i + 2] = x.z, to[4 * i + 3] = x.w;
    }
  }
}

// V's scale on V's values, in fp16: see the top.
template <int D, int G, int RT>
constexpr bool scale_on_v() {
  return D / G * RT >= 8;
}

// Waves a SIMD should hold: what O (4 D RT / 64 registers), Q and a step's words
// leave of its 512 registers, without scratch.  Blocks of eight waves put two on
// every SIMD, so theirs are two or four.
template <int D, int G, int RT>
constexpr int waves_per_simd() {
  return D * RT <= 64 ? 4 : (D * RT <= 128 ? (D / G <= 2 ? 4 : 2) : (D * RT <= 256 ? 2 : 1));
}

template <int D, int RT>
constexpr int most_threads() {
  return D * RT <= 128 ? 512 : 256;
}

template <typename T, int D, int G, int RT, bool PAIR>
__global__ __launch_bounds__((most_threads<D, RT>()), (waves_per_simd<D, G, RT>())) void attention_kernel(AttentionKernelArgs a) {
  constexpr int NG = D / G, KJ = D / 32, NC = D / 64;
  constexpr bool kBiasInSum = NG * RT <= (D == 256 ? 4 : 8);  // else the registers are needed elsewhere
  constexpr bool kScaleV = scale_on_v<D, G, RT>();
  static_assert(!PAIR || (RT == 1 && !kScaleV));
  constexpr bool kTwo = !(kScaleV && T::kCoarse);  // terms of a probability, and of a scaled value
  constexpr int kRowStride = D + 4;          // floats; the 16 rows of a store fall in distinct banks
  extern __shared__ __align__(16) float lds[];
  const int waves = blockDim.x / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int lane = threadIdx.x % 64, li = lane % 16, la = lane / 16;

  // pieces of the same number first: all sequences have the first ones, only
  // long ones the last, so what runs at the end is what fills gaps
  const int seq = blockIdx.y, split = blockIdx.z;
  int rb = 0, head = blockIdx.x;
  if (a.row_blocks > 1) {
    rb = head % a.row_blocks;
    head /= a.row_blocks;
  }
  const int key0 = split * a.chunk;
  const int tile_shift = a.shift - 4;
  // The first step's page numbers come along with the lengths: whatever the
  // length is, the row of the table has an entry there (of any value behind
  // the sequence's end).
  scalar_int32 *row_of_table = (scalar_int32 *)(uintptr_t)(a.table + (int64_t)seq * a.width);
  const int first = key0 / kStepKeys + wave;
  const int32_t early[2] = {row_of_table[min(2 * first >> tile_shift, a.width - 1)],
                            row_of_table[min(2 * first + 1 >> tile_shift, a.width - 1)]};
  const Work w = work_of(a, seq);
  const int rows = min(w.q_len, a.max_q) * a.share;
  const int row0 = rb * 16 * RT;
  if (row0 >= rows || split >= w.used) return;
  const int key1 = split == a.splits - 1 ? w.len : min(w.len, key0 + a.chunk);

  const int step1 = (key1 + kStepKeys - 1) / kStepKeys;
  const int last_tile = (w.len - 1) >> 4;

  typedef Stage<D, G> St;
  char *stages = reinterpret_cast<char *>(lds) + wave * (kStages * St::kBytes);
  // first token of a tile in the cache's arrays of one head
  const auto token_of = [&](int tile, int32_t page) {
    const int64_t number = clamp_to(page, 0, a.num_pages - 1);
    return ((number * a.kv_heads + head) << a.shift) + ((tile & ((1 << tile_shift) - 1)) << 4);
  };
  // this lane's piece of the 8 NG pieces of scales: array, tile, place
  const uint16_t *my_scales = lane / (4 * NG) ? a.v_scales : a.k_scales;
  const bool my_tile = lane / (2 * NG) % 2;
  const int my_piece = lane % (2 * NG) * 8;
  const auto load_as = [&](auto once, int64_t token0, int64_t token1, char *to) {
    constexpr bool kOnce = decltype(once)::value;
    if constexpr (D == 64) {
      const int64_t mine = (lane / 32 ? token1 : token0) * (D / 2) + lane % 32 * 16;
      copy16<kOnce>(a.k_vals + mine, to);
      copy16<kOnce>(a.v_vals + mine, to + St::kV);
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < D / 128; ++h) {
          const int64_t token = t ? token1 : token0;
          copy16<kOnce>(a.k_vals + token * (D / 2) + (li * (D / 2) + la * (D / 8) + 16 * h), to + t * St::kTile + 1024 * h);
          copy16<kOnce>(a.v_vals + token * (D / 2) + (la * (2 * D) + li * (D / 8) + 16 * h), to + St::kV + t * St::kTile + 1024 * h);
        }
    }
    if (lane < 8 * NG) copy16<kOnce>(my_scales + (my_tile ? token1 : token0) * NG + my_piece, to + St::kKs);
  };
  const bool alone = a.row_blocks == 1;
  const auto load = [&](int64_t token0, int64_t token1, char *to) {
    if (alone)
      load_as(std::true_type(), token0, token1, to);
    else
      load_as(std::false_type(), token0, token1, to);
  };
  // the page numbers of a step's tiles, read one step before they are needed
  struct Pages {
    int tile[2];
    int32_t page[2];
  };
  const auto pages_of = [&](int s) {
    Pages p;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      p.tile[t] = min(2 * s + t, last_tile);
      p.page[t] = row_of_table[p.tile[t] >> tile_shift];
    }
    return p;
  };
  const auto load_step = [&](const Pages &p, char *to) {
    load(token_of(p.tile[0], p.page[0]), token_of(p.tile[1], p.page[1]), to);
  };
  Pages ahead = {};
  if (first < step1) {
    load(token_of(2 * first, early[0]), token_of(2 * first + 1, early[1]), stages);
    if (first + waves < step1) load_step(pages_of(first + waves), stages + St::kBytes);
    ahead = pages_of(first + 2 * waves);
  }

  // the query rows: lane (i, a) holds channels 32j + 8a .. +7 of row i
  typename T::vec q[RT][KJ];
  float bias[RT][NG];
  int limit[RT];          // last visible key (causal)
  uint64_t tree[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int row = row0 + 16 * r + (PAIR ? li % 8 : li);
    const bool has = row < rows;
    const int token = w.q0 + (has ? row / a.share : 0), qh = head * a.share + (has ? row % a.share : 0);
    const uint16_t *p = static_cast<const uint16_t *>(a.q) + token * a.q_token + qh * a.q_head + 8 * la;
    float s[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) s[g] = 0.0f;
#pragma unroll
    for (int j = 0; j < KJ; ++j) {
      w4_t x = *reinterpret_cast<const w4_t *>(p + 32 * j);
      if (!has) x = w4_t{0, 0, 0, 0};
      q[r][j] = __builtin_bit_cast(typename T::vec, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) s[32 * j / G] += T::to_float(x[e] & 0xFFFFu) + T::to_float(x[e] >> 16);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) bias[r][g] = -kOffset * sum4(s[g]);
    limit[r] = w.ctx + (token - w.q0);
    tree[r] = a.tree ? (uint64_t)a.tree[token] : 0;
  }

  f4_t o[RT][NC][4];
  // Scores are sums that start from minus the reference, so that their distance
  // to it is exact where it counts, however far from 0 both are.
  float less[RT];      // minus the reference
  uint64_t fresh[RT];  // the lanes whose row has seen no key yet
  float l[RT], extra[RT][kScaleV ? 1 : NG];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    less[r] = 0.0f;
    fresh[r] = ~uint64_t(0);
    l[r] = 0.0f;
#pragma unroll
    for (float &x : extra[r]) x = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][c][e] = f4_t{0, 0, 0, 0};
  }
  // fp16 terms use that type's range up to 2^15, bf16 terms need not
  // (-1, 0) and (0, -1) in bf16; in registers, as the compiler takes the second
  // for the constant -1.0 of the instruction, which is another number there
  const uint32_t without[2] = {in_vgpr(PAIR && li < 8 ? 0u : 0x0000BF80u), in_vgpr(PAIR && li < 8 ? 0u : 0xBF800000u)};
  constexpr float kHeadroom = kScaleV ? 15.0f - (float)kAttentionSlack : 0.0f;

  const Constants constants = {in_sgpr(T::kMask), in_vgpr(T::kSixteen), in_sgpr(BF16::kMask), in_vgpr(0xC1F84180u),
                               in_sgpr(0x000F000Fu), in_sgpr(0x00F000F0u), in_vgpr(0x64006400u)};
  struct {
    uint32_t k[2][KJ], v[2][St::kVWords];
    uint32_t ks[2][NG][2], vs[2][NG][2];  // fp16 scales of four keys
  } st;
  const auto read_k = [&](const char *from) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const char *p = from + t * St::kTile;
      if constexpr (D == 64) {
        read_words<2>(st.k[t], p + li * 32 + la * 8);
      } else {
#pragma unroll
        for (int h = 0; h < D / 128; ++h) read_words<4>(st.k[t] + 4 * h, p + 1024 * h + lane * 16);
      }
      read_words<2 * NG>(&st.ks[t][0][0], from + St::kKs + t * St::kScales + la * (8 * NG));
    }
  };
  const auto read_v = [&](const char *from) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const char *p = from + St::kV + t * St::kTile;
#pragma unroll
      for (int h = 0; h < (D + 127) / 128; ++h)
        read_words<4>(st.v[t] + 4 * h, p + 1024 * h + (D == 64 ? la * 128 + li / 2 * 16 : lane * 16));
      read_words<2 * NG>(&st.vs[t][0][0], from + St::kVs + t * St::kScales + la * (8 * NG));
    }
  };

  f4_t sc[RT][2];
  const auto scores = [&]() {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      typename T::vec kf[KJ];
#pragma unroll
      for (int j = 0; j < KJ; ++j) kf[j] = widen_k<T>(st.k[t][j], constants);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        f4_t sum = {less[r], less[r], less[r], less[r]};
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const float b = bias[r][g];
          f4_t acc = kBiasInSum ? f4_t{b, b, b, b} : f4_t{0, 0, 0, 0};
#pragma unroll
          for (int j = g * (G / 32); j < (g + 1) * (G / 32); ++j) acc = T::mfma(kf[j], q[r][j], acc);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float f = fp16_bits_to_float((st.ks[t][g][x / 2] >> (16 * (x % 2))) & 0xFFFFu);
            sum[x] = fmaf(f, kBiasInSum ? acc[x] : acc[x] + b, sum[x]);
          }
        }
        sc[r][t] = sum;
      }
    }
  };
  const auto values = [&](int s) {
    const int key = s * kStepKeys;
    const bool edge = key + kStepKeys > w.ctx;  // some key is not seen by every row
    if (edge) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int pos = key + 16 * t + 4 * la + x;
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            bool seen = pos < w.len;
            if (a.tree) {
              const int b = pos - w.ctx;
              seen = seen && (b < 0 || (b < 64 && ((tree[r] >> (b & 63)) & 1)));
            } else {
              seen = seen && pos <= limit[r];
            }
            if (!seen) sc[r][t][x] = -INFINITY;
          }
          // what lies behind the last key may be anything: 0 * that must be 0
          if (pos >= w.len) {
#pragma unroll
            for (int g = 0; g < NG; ++g) st.vs[t][g][x / 2] &= x % 2 ? 0x0000FFFFu : 0xFFFF0000u;
          }
        }
    }
    bool grows = false;
    float top[RT];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float m = sc[r][0][0];
#pragma unroll
      for (int x = 1; x < 8; ++x) m = maximum(m, sc[r][x / 4][x % 4]);
      top[r] = max4(m);
      grows |= top[r] > a.slack;
      if (fresh[r]) grows |= __builtin_amdgcn_inverse_ballot_w64(fresh[r]) && top[r] > -INFINITY;
    }
    if (__any(grows)) {
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const bool first = __builtin_amdgcn_inverse_ballot_w64(fresh[r]), seen = top[r] > -INFINITY;  // no key, or a NaN
        // up by the step's largest exactly: its distance is 0 now, whatever a last place of the score may be worth
        const float up = first ? (seen ? top[r] : 0.0f) : fmaxf(top[r], 0.0f);
        const float f = first ? 1.0f : __builtin_amdgcn_exp2f(-up * a.scale_log2);
        less[r] -= up;
        fresh[r] &= ~__ballot(seen);
#pragma unroll
        for (int x = 0; x < 8; ++x) sc[r][x / 4][x % 4] -= up;
        l[r] *= f;
#pragma unroll
        for (float &x : extra[r]) x *= f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][c][e] *= f;
      }
    }
    float p[RT][2][4];
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          p[r][t][x] = __builtin_amdgcn_exp2f(fmaf(sc[r][t][x], a.scale_log2, kHeadroom));
          l[r] += p[r][t][x];
        }
    // the probabilities, times V's scales of a group or not, in two terms
    typedef typename std::conditional<kScaleV, hf8_t, bf8_t>::type term_t;
    term_t high[RT], low[RT];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      typename std::conditional<kScaleV, h2_t, uint32_t>::type vq[2][2][4];  // [tile][token pair][e]
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t w0 = st.v[t][4 * (c / 2) + 2 * x], w1 = st.v[t][4 * (c / 2) + 2 * x + 1];
          const uint32_t upper = D == 64 ? (uint32_t)(li & 1) : (uint32_t)(c & 1);
          widen_v(__builtin_amdgcn_perm(w1, w0, upper ? 0x07060302u : 0x05040100u), constants, vq[t][x]);
        }
      constexpr int kSame = G < 64 ? G / 16 : 4;  // tiles of 16 channels of one group
#pragma unroll
      for (int e0 = 0; e0 < 4; e0 += kSame) {
        const int g = (64 * c + 16 * e0) / G;
        const auto words = [&](int e) {
          return w4_t{__builtin_bit_cast(uint32_t, vq[0][0][e]), __builtin_bit_cast(uint32_t, vq[0][1][e]),
                      __builtin_bit_cast(uint32_t, vq[1][0][e]), __builtin_bit_cast(uint32_t, vq[1][1][e])};
        };
        if constexpr (kScaleV) {
          if (c == 0 && e0 == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int x = 0; x < 8; x += 2) {
                const f2_t y = {p[r][x / 4][x % 4], p[r][x / 4][x % 4 + 1]};
                const h2_t first = __builtin_convertvector(y, h2_t);
                high[r][x] = first.x, high[r][x + 1] = first.y;
                if (!kTwo) continue;
                // one v_fma_mixlo/hi_f16 each
                low[r][x] = (_Float16)fmaf((float)first.x, -1.0f, y.x);
                low[r][x + 1] = (_Float16)fmaf((float)first.y, -1.0f, y.y);
              }
          }
#pragma unroll
          for (int e = e0; e < e0 + kSame; ++e) {
            h2_t rest[2][2];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const h2_t v = vq[x / 2][x % 2][e], scale = as_h2(st.vs[x / 2][g][x % 2]);
              vq[x / 2][x % 2][e] = v * scale;
              if (kTwo) rest[x / 2][x % 2] = __builtin_elementwise_fma(v, scale, -vq[x / 2][x % 2][e]);
            }
            const hf8_t first = __builtin_bit_cast(hf8_t, words(e));
#pragma unroll
            for (int r = 0; r < RT; ++r) o[r][c][e] = F16::mfma(first, high[r], o[r][c][e]);
            if constexpr (kTwo) {
              const hf8_t second = __builtin_bit_cast(hf8_t, rest);
#pragma unroll
              for (int r = 0; r < RT; ++r) o[r][c][e] = F16::mfma(second, high[r], o[r][c][e]);
#pragma unroll
              for (int r = 0; r < RT; ++r) o[r][c][e] = F16::mfma(first, low[r], o[r][c][e]);
            }
          }
        } else {
          if ((64 * c + 16 * e0) % G == 0) {
#pragma unroll
            for (int r = 0; r < RT; ++r)
#pragma unroll
              for (int x = 0; x < 8; x += 2) {
                const uint32_t scales = st.vs[x / 4][g][x % 4 / 2];
                const f2_t y = {p[r][x / 4][x % 4] * fp16_bits_to_float(scales & 0xFFFFu),
                                p[r][x / 4][x % 4 + 1] * fp16_bits_to_float(scales >> 16)};
                bf2_t first = __builtin_convertvector(y, bf2_t);
                const f2_t rest = {dot2(first, without[0], y.x), dot2(first, without[1], y.y)};
                const bf2_t second = __builtin_convertvector(rest, bf2_t);
                if (PAIR) first = second;
                high[r][x] = first.x, high[r][x + 1] = first.y;
                extra[r][g] = dot2(first, kPairBias, extra[r][g]);
                if constexpr (!PAIR) {
                  low[r][x] = second.x, low[r][x + 1] = second.y;
                  extra[r][g] = dot2(second, kPairBias, extra[r][g]);
                }
              }
          }
#pragma unroll
          for (int part = 0; part < (PAIR ? 1 : 2); ++part)
#pragma unroll
            for (int e = e0; e < e0 + kSame; ++e)
#pragma unroll
              for (int r = 0; r < RT; ++r)
                o[r][c][e] = BF16::mfma(__builtin_bit_cast(bf8_t, words(e)), part ? low[r] : high[r], o[r][c][e]);
        }
      }
    }
  };

  // Two steps are on their way or in use at any time; the last ones are not
  // followed by others, so there the wait is for everything.
  int at = 0;
  for (int s = first; s < step1; s += waves) {
    char *stage = stages + at;
    if (s + waves < step1) wait_loads<St::kLoads>(); else wait_loads<0>();
    read_k(stage);
    scores();
    read_v(stage);
    values(s);
    issue_fence();
    if (s + 2 * waves < step1) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): this stage is read
      issue_fence();
      load_step(ahead, stage);
      ahead = pages_of(s + 3 * waves);
    }
    at = St::kBytes - at;
  }
  __syncthreads();  // the stages make room for what follows

  // the waves join: references and sums first, then the outputs of one 16-row
  // tile at a time, each scaled to the common reference
  float *ml = lds;                         // [waves][16 * RT][2]
  float *ob = lds + waves * 16 * RT * 2;   // [waves][16][kRowStride]
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    less[r] = __builtin_amdgcn_inverse_ballot_w64(fresh[r]) ? -INFINITY : -less[r];  // now the reference
    l[r] = sum4(l[r]);
    if constexpr (!kScaleV) {
#pragma unroll
      for (float &x : extra[r]) x = sum4(x);
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][c][e] -= extra[r][(64 * c + 16 * e) / G];
    }
    if (la == 0) {
      ml[(wave * 16 * RT + 16 * r + li) * 2] = less[r];
      ml[(wave * 16 * RT + 16 * r + li) * 2 + 1] = l[r];
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    if (r) __syncthreads();
    float top = kLowest;
    for (int x = 0; x < waves; ++x) top = fmaxf(top, ml[(x * 16 * RT + 16 * r + li) * 2]);
    const float f = __builtin_amdgcn_exp2f(fmaf(less[r] - top, a.scale_log2, -kHeadroom));
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f4_t *>(ob + (wave * 16 + li) * kRowStride + 64 * c + 16 * e + 4 * la) = o[r][c][e] * f;
    __syncthreads();
    for (int at = threadIdx.x; at < (PAIR ? 8 : 16) * (D / 4); at += blockDim.x) {
      const int i = at / (D / 4), d = at % (D / 4) * 4, row = row0 + 16 * r + i;
      if (row >= rows) break;
      float m = kLowest, sum = 0.0f;
      for (int x = 0; x < waves; ++x) m = fmaxf(m, ml[(x * 16 * RT + 16 * r + i) * 2]);
      f4_t v = {0, 0, 0, 0};
      for (int x = 0; x < waves; ++x) {
        const float *e = ml + (x * 16 * RT + 16 * r + i) * 2;
        sum = fmaf(e[1], __builtin_amdgcn_exp2f(fmaf(e[0] - m, a.scale_log2, -kHeadroom)), sum);
        v += *reinterpret_cast<const f4_t *>(ob + (x * 16 + i) * kRowStride + d);
        if (PAIR) v += *reinterpret_cast<const f4_t *>(ob + (x * 16 + i + 8) * kRowStride + d);
      }
      const int64_t token = w.q0 + row / a.share;
      const int64_t at_row = token * (a.kv_heads * a.share) + head * a.share + row % a.share;
      if (w.used == 1) {
        const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
        v *= inv;
        const w2_t bits = {T::from_float(v[0]) | T::from_float(v[1]) << 16,
                           T::from_float(v[2]) | T::from_float(v[3]) << 16};
        *reinterpret_cast<w2_t *>(static_cast<uint16_t *>(a.out) + at_row * D + d) = bits;
        if (d == 0 && a.lse) a.lse[at_row] = lse_of(m, sum, a.scale_log2);
      } else {
        const int64_t part = (int64_t)split * a.num_tokens * (a.kv_heads * a.share) + at_row;
        *reinterpret_cast<f4_t *>(a.part_o + part * D + d) = v;
        if (d == 0) {
          a.part_ml[2 * part] = m;
          a.part_ml[2 * part + 1] = sum;
        }
      }
    }
  }
}

// Joins the pieces of a row: block (row of the sequence, sequence).  D/4
// neighbouring threads hold a row, 1024/D such groups take the pieces in turn.
template <typename T, int D>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionKernelArgs a) {
  constexpr int kGroups = 1024 / D;
  __shared__ f4_t part[256];
  __shared__ float weight[kMaxSplits], wave_m[4], wave_l[4];
  const int q_heads = a.kv_heads * a.share;
  const Work w = work_of(a, blockIdx.y);
  const int t = blockIdx.x / q_heads;
  if (t >= min(w.q_len, a.max_q) || w.used == 1) return;
  const int64_t rows = (int64_t)a.num_tokens * q_heads;
  const int64_t row = (int64_t)(w.q0 + t) * q_heads + blockIdx.x % q_heads;
  const int tid = threadIdx.x;
  float m = kLowest;
  for (int s = tid; s < w.used; s += 256) {
    const float e = a.part_ml[2 * (s * rows + row)];
    weight[s] = e;
    m = fmaxf(m, e);
  }
  for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  if (tid % 64 == 0) wave_m[tid / 64] = m;
  __syncthreads();
  m = fmaxf(fmaxf(wave_m[0], wave_m[1]), fmaxf(wave_m[2], wave_m[3]));
  float sum = 0.0f;
  for (int s = tid; s < w.used; s += 256) {
    const float f = __builtin_amdgcn_exp2f((weight[s] - m) * a.scale_log2);
    weight[s] = f;
    sum = fmaf(a.part_ml[2 * (s * rows + row) + 1], f, sum);
  }
  for (int d = 32; d; d >>= 1) sum += __shfl_xor(sum, d);
  if (tid % 64 == 0) wave_l[tid / 64] = sum;
  __syncthreads();
  sum = (wave_l[0] + wave_l[1]) + (wave_l[2] + wave_l[3]);
  const int group = tid / (D / 4), d = tid % (D / 4) * 4;
  f4_t v = {0, 0, 0, 0};
#pragma unroll 4
  for (int s = group; s < w.used; s += kGroups)
    v += *reinterpret_cast<const f4_t *>(a.part_o + (s * rows + row) * D + d) * weight[s];
  part[tid] = v;
  __syncthreads();
  if (group) return;
  for (int g = 1; g < kGroups; ++g) v += part[g * (D / 4) + tid];
  v *= sum == 0.0f ? 0.0f : 1.0f / sum;
  const w2_t bits = {T::from_float(v[0]) | T::from_float(v[1]) << 16, T::from_float(v[2]) | T::from_float(v[3]) << 16};
  *reinterpret_cast<w2_t *>(static_cast<uint16_t *>(a.out) + row * D + d) = bits;
  if (d == 0 && a.lse) a.lse[row] = lse_of(m, sum, a.scale_log2);
}

// The same for few pieces: D/4 neighbouring threads hold a row and take its
// pieces one after the other, 1024/D rows a block (16384 rows of 4 pieces: 20
// us with a block a row, 9 so).
constexpr int kFewSplits = 8;
template <typename T, int D>
__global__ __launch_bounds__(256) void attention_join_few_kernel(AttentionKernelArgs a) {
  const int q_heads = a.kv_heads * a.share;
  const Work w = work_of(a, blockIdx.y);
  const int i = blockIdx.x * (1024 / D) + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;  // row of the sequence
  if (i >= min(w.q_len, a.max_q) * q_heads || w.used == 1) return;
  const int64_t rows = (int64_t)a.num_tokens * q_heads, row = (int64_t)w.q0 * q_heads + i;
  float mo[kFewSplits], l[kFewSplits], m = kLowest;
  f4_t v[kFewSplits];
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s) {
    const int at = min(s, w.used - 1);  // loads without branches
    mo[s] = a.part_ml[2 * (at * rows + row)];
    l[s] = a.part_ml[2 * (at * rows + row) + 1];
    v[s] = *reinterpret_cast<const f4_t *>(a.part_o + (at * rows + row) * D + d);
    m = fmaxf(m, mo[s]);
  }
  f4_t o = {0, 0, 0, 0};
  float sum = 0.0f;
#pragma unroll
  for (int s = 0; s < kFewSplits; ++s)
    if (s < w.used) {
      const float f = __builtin_amdgcn_exp2f((mo[s] - m) * a.scale_log2);
      sum = fmaf(l[s], f, sum);
      o += v[s] * f;
    }
  o *= sum == 0.0f ? 0.0f : 1.0f / sum;
  const w2_t bits = {T::from_float(o[0]) | T::from_float(o[1]) << 16, T::from_float(o[2]) | T::from_float(o[3]) << 16};
  *reinterpret_cast<w2_t *>(static_cast<uint16_t *>(a.out) + row * D + d) = bits;
  if (d == 0 && a.lse) a.lse[row] = lse_of(m, sum, a.scale_log2);
}

template <typename T, int D, int G, int RT, bool PAIR>
hipError_t go(const AttentionKernelArgs &a, const AttentionPlan &p, hipStream_t stream) {
  const size_t join = sizeof(float) * p.waves * (16 * RT * 2 + 16 * (D + 4));
  const size_t stages = (size_t)p.waves * kStages * Stage<D, G>::kBytes;
  const size_t lds = join > stages ? join : stages;
  if (lds > 64 * 1024) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(attention_kernel<T, D, G, RT, PAIR>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((attention_kernel<T, D, G, RT, PAIR>), dim3((unsigned)a.row_blocks * a.kv_heads, a.num_seqs, p.splits),
                     dim3(64 * p.waves), lds, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  if (p.splits <= kFewSplits) {
    const unsigned rows = (unsigned)a.max_q * a.kv_heads * a.share, per = 1024 / D;
    hipLaunchKernelGGL((attention_join_few_kernel<T, D>), dim3((rows + per - 1) / per, a.num_seqs), dim3(256), 0, stream, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL((attention_join_kernel<T, D>), dim3((unsigned)a.max_q * a.kv_heads * a.share, a.num_seqs), dim3(256),
                     0, stream, a);
  return hipGetLastError();
}

template <typename T, int D, int G>
hipError_t by_rows(const AttentionKernelArgs &a, const AttentionPlan &p, hipStream_t stream) {
  if constexpr (D <= 128 && D / G >= 4)
    if (p.row_tiles == 2) return go<T, D, G, 2, false>(a, p, stream);
  if constexpr (!scale_on_v<D, G, 1>())
    if (a.max_q * a.share <= 8) return go<T, D, G, 1, true>(a, p, stream);
  return go<T, D, G, 1, false>(a, p, stream);
}

template <typename T>
hipError_t by_shape(const AttentionKernelArgs &a, const AttentionPlan &p, int d, int g, hipStream_t s) {
  if (d == 64) return g == 32 ? by_rows<T, 64, 32>(a, p, s) : by_rows<T, 64, 64>(a, p, s);
  if (d == 128)
    return g == 32 ? by_rows<T, 128, 32>(a, p, s) : g == 64 ? by_rows<T, 128, 64>(a, p, s) : by_rows<T, 128, 128>(a, p, s);
  return g == 32 ? by_rows<T, 256, 32>(a, p, s) : g == 64 ? by_rows<T, 256, 64>(a, p, s) : by_rows<T, 256, 128>(a, p, s);
}

}  // namespace

hipError_t launch_attention(const AttentionKernelArgs &a, const AttentionPlan &p, int32_t head_dim, int32_t group_size,
                            int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16 ? by_shape<F16>(a, p, head_dim, group_size, stream)
                          : by_shape<BF16>(a, p, head_dim, group_size, stream);
}

}  // namespace i4s
