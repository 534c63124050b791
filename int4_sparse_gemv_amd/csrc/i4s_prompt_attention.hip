// Attention of packed sequences over their own 16-bit keys and values
// (include/i4s_prompt.h), for gfx950.
//
// A block takes 128 or 256 query rows (tokens x query heads) of one sequence
// that read one KV head, 32 a wave; its waves share tiles of keys and values in
// LDS, filled with direct 16-byte loads ahead of their use.  Scores and outputs
// are computed transposed, so that no value moves between lanes on the way:
//   S^T = K Q^T: v_mfma_f32_32x32x16 with 32 keys as rows, 32 query rows as
//     columns and 16 channels.  Lane l = i + 32 h holds query row i and the
//     keys 8 x + 4 h + 0..3, x = 0..3, of a tile: its softmax is a loop over
//     registers and one exchange with lane l ^ 32.
//   O^T = V^T P^T: 32 channels as rows, 32 query rows as columns, 16 keys.  Its
//     B operand wants query row i and 8 keys in lane l: P's registers as they
//     are, for the keys 4 h + 0..3 and 8 + 4 h + 0..3.  Its A operand wants
//     channel i and the same keys: ds_read_b64_tr_b16 hands 4 keys x 16
//     channels of a row-major tile to 16 lanes, transposed.
// Scores are summed from minus the row's reference on (a score near its
// running maximum): exponents are exact differences however far from 0 the
// scores lie, and the reference follows the maximum only when that has grown
// by 8 powers of two, so O is scaled rarely.
//
// Roundings: scores, sums and outputs are fp32.  A probability is rounded to
// the values' type for its matrix instruction (at most 2^-8 of itself for
// bf16, 2^-11 for fp16), the sum takes it unrounded; the output is rounded once.  A
// second term for what the first leaves would double the second product, which bounds
// blocks of many rows: their outputs are 0.0021 (bf16; fp16 0.00026) off where their own
// rounding makes 0.0016 (0.0002).  Blocks of few rows wait for memory, but round as the
// others do: a short sequence has the same bits in a launch of either shape.
//
// Values that are not finite cost the usual call nothing: 0 times one is a NaN, in the
// rows that do not see it as in those whose probability of it is 0, and a block whose
// rows have a NaN at the end that is not their scores' goes through its keys again with
// such values apart.  Us, 8191 tokens, 40 heads: 803 back to back, with a NaN in the first
// key 2271, with nothing but infinities 6444.
//
// Long prompts are bound by the matrix cores, the LDS that feeds them (every wave
// reads all keys and values for its 32 rows: half of the LDS's cycles) and power.
// 8191 tokens, 40 heads of 128: 1225 us without the causal mask = 1.12 PFLOP/s, 661
// with it; large matrix products of the library reach 1.15 to 1.36, matrix instructions
// alone 1.9.  Us without the mask, step by step: operands read by the instruction that
// uses them 1400; four instructions ahead, V's first ones before the softmax, 1300
// (head dimension 256: 224, 178; two ahead 204; six the same as four); blocks of 256
// rows in two halves, one in its softmax while the other multiplies, 1275, with the
// loads' issue in the softmax 1231.  The tiles that a mask cuts, 40 prompts of 512
// tokens, 40 heads: with registers that spill 405, with less held from one to the next
// 285, without a look at each one's V for values that are not finite 263.  Tried and no
// faster: wave priorities for either part, waits between matrix instructions, 32-key
// tiles with the next scores ahead of this softmax; 64 rows a wave spill.
//
// 32 rows or fewer of a sequence and KV head (a token behind long keys) are bound
// by memory: there each wave of a block has tiles of 32 keys of its own, two of
// them, in its own time with no barrier, and all join in LDS; long keys are
// split over blocks, joined by a second launch.  Keys and values are read once,
// past the caches.  65536 keys of 8 KV heads of 128, 32 query heads: 49 us = 5.4
// TB/s (through the caches 64), 64 such sequences of 4096 keys 164 us = 6.6 (186).
// Us through the caches, waves x tiles ahead 3x3 / 4x2 / 5x2: 60.2 / 59.5 / 61.8, D =
// 64 38.1 / 36.8 / 39.6; blocks of four waves sharing tiles of 64 keys took 115.

#include <float.h>

#include <type_traits>

#include "i4s_gemv_common.h"
#include "i4s_prompt_internal.h"

namespace i4s {
namespace {

typedef float f16_t __attribute__((ext_vector_type(16)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));
typedef short s4_t __attribute__((ext_vector_type(4)));
typedef __bf16 b2_t __attribute__((ext_vector_type(2)));

struct Half {
  typedef _Float16 vec __attribute__((ext_vector_type(8)));
  typedef h2_t pair;
  static constexpr float kHeadroom = 7.0f;  // log2 of a probability's factor: 2^15 with the slack is finite
  static constexpr uint32_t kInf = 0x7C00u, kOne = 0x3C00u;
  static __device__ f16_t mfma(u4_t a, u4_t b, f16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(vec, a), __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
  static __device__ float dot(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2(__builtin_bit_cast(h2_t, a), __builtin_bit_cast(h2_t, b), c, false);
  }
};
struct Brain {
  typedef __bf16 vec __attribute__((ext_vector_type(8)));
  typedef b2_t pair;
  static constexpr float kHeadroom = 0.0f;  // fp32's exponents
  static constexpr uint32_t kInf = 0x7F80u, kOne = 0x3F80u;
  static __device__ f16_t mfma(u4_t a, u4_t b, f16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(vec, a), __builtin_bit_cast(vec, b), c, 0, 0, 0);
  }
  static __device__ float dot(uint32_t a, uint32_t b, float c) {
    return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(b2_t, a), __builtin_bit_cast(b2_t, b), c, false);
  }
};

// Two values rounded to nearest even, the first in the low half.
template <typename T>
__device__ inline uint32_t two(float a, float b) {
  const f2_t f = {a, b};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, typename T::pair));
}

// The value of the other lane that holds the same query row.
__device__ inline float other_half(float v, int lane) {
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto s = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t a = s[0], b = s[1];
  return __builtin_bit_cast(float, lane < 32 ? b : a);
}

__device__ inline float lse_of(float reference, float sum, float scale_log2, float headroom) {
  return sum == 0.0f ? -INFINITY
                     : fmaf(reference, scale_log2, __builtin_amdgcn_logf(sum) - headroom) * 0.6931471805599453f;
}

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
template <int AUX>  // 2: past the caches
__device__ inline void copy16(const void *from, char *to) {
  __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)to, 16, 0, AUX);
}
template <int N>
__device__ inline void wait_loads() {
  issue_fence();
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
  issue_fence();
}
// Waves meet: their LDS reads are done, their direct loads waited for.
__device__ inline void meet() {
  issue_fence();
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  issue_fence();
}

// Four keys x 16 channels of a row-major tile, transposed: lane i of 16 brings
// the address of four channels of key i / 4 and gets channel i of the four keys.
// The pointer's __restrict tells the compiler that direct loads on their way
// write elsewhere (the barriers see to that): it would wait for them here.
typedef __attribute__((address_space(3))) s4_t *lds_s4;
__device__ inline __attribute__((always_inline)) u2_t read_transposed(lds_s4 __restrict p) {
  return __builtin_bit_cast(u2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}

// What a block works on, all made safe.
struct Sequence {
  int q0, nq, k0, nk;
};
__device__ inline Sequence sequence_of(const PromptKernelArgs &a, int seq) {
  if (!a.q_start) return {0, a.num_tokens, 0, a.num_keys};
  Sequence s;
  s.q0 = clamp_to(a.q_start[seq], 0, a.num_tokens);
  s.nq = clamp_to(a.q_start[seq + 1], s.q0, a.num_tokens) - s.q0;
  s.k0 = clamp_to(a.k_start[seq], 0, a.num_keys);
  s.nk = clamp_to(a.k_start[seq + 1], s.k0, a.num_keys) - s.k0;
  return s;
}
// How many keys query token t sees.
__device__ inline int keys_seen(const PromptKernelArgs &a, const Sequence &s, int t) {
  return a.causal ? clamp_to(s.nk - s.nq + t + 1, 0, s.nk) : s.nk;
}

// Tiles of K and V in LDS: rows of 2 D bytes, the 16-byte pieces of a row
// exchanged by the row's number so that the rows that an instruction reads
// together lie in different banks: for K (16 bytes of 32 rows) by 16 rows (D = 64:
// by its 8 pieces), for V (32 bytes of 8 rows) by twice the row.  By 8 rows K's
// reads took twice the cycles (half of all LDS cycles were conflicts).
template <int D, int KEYS>
struct Tile {
  static constexpr int kPieces = D / 8;  // of a row
  static constexpr int kKeys = KEYS;
  static constexpr int kBytes = kKeys * D * 2;
  static __device__ int k_piece(int row, int piece) { return piece ^ (row & (kPieces < 16 ? 7 : 15)); }
  static __device__ int v_piece(int row, int piece) { return piece ^ ((row & 7) << 1 & (kPieces - 1)); }
};

constexpr float kSlack = 8.0f;  // log2: how far a probability may pass 2^kHeadroom

// How a tile is worked on: every row sees all of it; a mask cuts it; and, in the pass
// for values that are not finite, each value by what it is.
constexpr int kPlain = 0, kMasked = 1, kCareful = 2;

// A sum of values at another reference: infinities stay where their weight is 0.
__device__ inline float weigh(float f, float v) { return __builtin_fabsf(v) == INFINITY ? v : f * v; }
__device__ inline f4_t weigh(float f, f4_t v) { return {weigh(f, v.x), weigh(f, v.y), weigh(f, v.z), weigh(f, v.w)}; }

// The factor of an output row.  Where all probabilities are 0 the row is 0 already, or an infinity or a NaN that it sees.
__device__ inline float over(float sum) { return sum == 0.0f ? 1.0f : 1.0f / sum; }

// ROWS of a block.  32: all query rows of a sequence and KV head fit a wave; the
// waves of a block take the same rows and tiles of their own in turn, and join
// at the end.  128: four waves, two blocks a compute unit.  256: eight, in two
// halves half a step apart.
// D = 256: 32 keys a tile, for 64 the registers do not reach.
template <typename T, int D, int ROWS>
struct Shape {
  static constexpr bool kFew = ROWS == kPromptRows, kPaired = ROWS == 8 * kPromptRows;
  static constexpr int kWaves = kFew ? (D == 256 ? 2 : 4) : ROWS / kPromptRows;
  typedef Tile<D, kFew || D == 256 ? 32 : 64> L;
  static constexpr int kLoaders = kFew ? 1 : kWaves;            // waves that share a tile's loads
  static constexpr int kLoads = L::kBytes / 1024 / kLoaders;    // load instructions of a wave for K, and for V
  static constexpr int kStages = kPaired ? 4 : 2;               // tiles of K, and of V
  static constexpr int kTiles = (kFew ? kWaves : 1) * 2 * kStages * L::kBytes;
  static constexpr int kLds = kTiles + (kFew ? 0 : 64);         // and a word of each wave
  static constexpr int kRowFloats = D + 4;                      // of an output row where waves join
  static_assert(!kFew || kWaves * kPromptRows * kRowFloats * 4 + kWaves * kPromptRows * 8 <= kTiles, "joined in the tiles' LDS");
  static_assert(kLds <= 160 * 1024, "a compute unit has 160 KB");
};

template <typename T, int D, int ROWS>
__global__ __launch_bounds__((64 * Shape<T, D, ROWS>::kWaves), (ROWS != 4 * kPromptRows || D == 256 ? 1 : 2)) void prompt_kernel(
    PromptKernelArgs a) {
  typedef Shape<T, D, ROWS> S;
  constexpr bool FEW = S::kFew, PAIRED = S::kPaired;
  typedef typename S::L L;
  constexpr int NK = L::kKeys / 32, NC = D / 32, NQ = D / 16, kWaves = S::kWaves;
  constexpr int kRowsPerLoad = 64 / L::kPieces, kAhead = 4;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int li = lane & 31, lh = lane >> 5;

  // Groups of pairs (sequence, KV head) that share the L2s, in each the rows that
  // see the most keys first; pairs in turn, so that XCDs share out the heads.
  const int pairs = a.num_seqs * a.kv_heads, first_pair = blockIdx.x / (a.group * a.row_blocks) * a.group;
  const int many = pairs - first_pair < a.group ? pairs - first_pair : a.group, in = blockIdx.x - first_pair * a.row_blocks;
  const int pair = first_pair + in % many, rb = a.row_blocks - 1 - in / many;
  const int seq = pair / a.kv_heads, head = pair % a.kv_heads;
  const Sequence s = sequence_of(a, seq);
  const int tokens = s.nq < a.max_q ? s.nq : a.max_q;
  const int rows = tokens * a.share, block_row = rb * ROWS;
  if (block_row >= rows) return;

  // keys of this piece that any row of the block sees
  const int last_row = block_row + ROWS < rows ? block_row + ROWS - 1 : rows - 1;
  const int most = keys_seen(a, s, last_row / a.share);
  const int piece0 = blockIdx.y * a.chunk;
  const int piece1 = (int)blockIdx.y + 1 < a.splits && most - piece0 > a.chunk ? piece0 + a.chunk : most;
  if (blockIdx.y && piece0 >= most) return;

  const int first_row = block_row + (FEW ? 0 : wave * kPromptRows);
  const int row = first_row + li;
  const int safe = row < rows ? row : rows - 1;
  const int t = safe / a.share, q_head = head * a.share + (safe - t * a.share);
  const int seen = keys_seen(a, s, t) < piece1 ? keys_seen(a, s, t) : piece1;  // this lane's row sees the keys below
  const int wave_row = first_row < rows ? first_row : rows - 1;
  const int wave_last = wave_row + kPromptRows - 1 < rows ? wave_row + kPromptRows - 1 : rows - 1;
  const int any_sees = keys_seen(a, s, wave_last / a.share);

  u4_t q[NQ];
  {
    const uint16_t *p = static_cast<const uint16_t *>(a.q) + (int64_t)(s.q0 + t) * a.q_token + q_head * a.q_head + lh * 8;
#pragma unroll
    for (int c = 0; c < NQ; ++c) q[c] = *reinterpret_cast<const u4_t *>(p + 16 * c);
  }

  const char *kb = static_cast<const char *>(a.k) + 2 * (s.k0 * a.k_token + head * a.k_head);
  const char *vb = static_cast<const char *>(a.v) + 2 * (s.k0 * a.v_token + head * a.v_head);
  const uint32_t k_step = 2 * (uint32_t)a.k_token, v_step = 2 * (uint32_t)a.v_token;
  // this wave's pieces of 1024 bytes of K and of V
  char *const tiles = lds + (FEW ? wave * 2 * S::kStages * L::kBytes : 0);
  const int loader = FEW ? 0 : wave;
  char *const v_tiles = tiles + S::kStages * L::kBytes;
  // rows past the keys repeat the last: their scores are masked
  auto load_k = [&](int key, int stage, int lane) {
    const int first = key < s.nk ? key : s.nk - 1, left = s.nk - 1 - first;
    const char *k0 = kb + (int64_t)first * k_step;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int at = loader * S::kLoads + i, r = at * kRowsPerLoad + lane / L::kPieces, p = lane % L::kPieces;
      const int from = r < left ? r : left;
      copy16<FEW ? 2 : 0>(k0 + (uint32_t)(from * k_step + L::k_piece(r, p) * 16), tiles + stage * L::kBytes + at * 1024);
    }
  };
  auto load_v = [&](int key, int stage, int lane) {
    const int first = key < s.nk ? key : s.nk - 1, left = s.nk - 1 - first;
    const char *v0 = vb + (int64_t)first * v_step;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int at = loader * S::kLoads + i, r = at * kRowsPerLoad + lane / L::kPieces, p = lane % L::kPieces;
      const int from = r < left ? r : left;
      copy16<FEW ? 2 : 0>(v0 + (uint32_t)(from * v_step + L::v_piece(r, p) * 16), v_tiles + stage * L::kBytes + at * 1024);
    }
  };

  f16_t o[NC], every;  // every: `less` in each register
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[c][e] = 0;
#pragma unroll
  for (int e = 0; e < 16; ++e) every[e] = 0;
  float sum = 0, less = 0;  // less: minus the row's reference
  bool fresh = true;

  auto step = [&](int key, int stage, auto MODE, auto &&load) {
    constexpr bool masked = decltype(MODE)::value != kPlain, careful = decltype(MODE)::value == kCareful;
    // In the masked tiles addresses are worked out anew: kept from one to the next they
    // would not fit the registers.
    int own = lane;
    if constexpr (masked) asm volatile("" : "+v"(own));
    const int li = own & 31, lh = own >> 5;
    // V's operand: channels 32 c + li of the keys 16 x + 4 lh + 0..3 and + 8
    const int tr_row = (own & 15) / 4 + 4 * lh, tr_piece = (own >> 4 & 1) * 2 + (own & 3) / 2;
    auto read_v = [&](const char *tile, int c, int x) {
      u4_t r;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int key = 16 * x + 8 * y + tr_row;
        const char *p = tile + key * 2 * D + L::v_piece(tr_row, 4 * c + tr_piece) * 16 + (own & 1) * 8;
        const u2_t w = read_transposed((lds_s4)p);
        r[2 * y] = w.x, r[2 * y + 1] = w.y;
      }
      return r;
    };
    f16_t start = every;
    if constexpr (masked) {
      float one = less;
      asm volatile("" : "+v"(one));
#pragma unroll
      for (int e = 0; e < 16; ++e) start[e] = one;
    }
    // Operands are read kAhead instructions ahead of the one that uses them, V's
    // first ones before the softmax.
    constexpr int kScores = NK * NQ, kValues = 2 * NK * NC;
    f16_t p[NK];
    u4_t ahead[kAhead];
    auto read_k = [&](int i) {  // neighbouring products have sums of their own
      const char *row = tiles + stage * L::kBytes + (32 * (i % NK) + li) * 2 * D;
      return *reinterpret_cast<const u4_t *>(row + L::k_piece(li, 2 * (i / NK) + lh) * 16);
    };
    const char *const tile = v_tiles + stage * L::kBytes;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = read_k(i);
    issue_fence();
#pragma unroll
    for (int i = 0; i < kScores; ++i) {
      p[i % NK] = T::mfma(ahead[i % kAhead], q[i / NK], i < NK ? start : p[i % NK]);
      if (i + kAhead < kScores) ahead[i % kAhead] = read_k(i + kAhead);
      issue_fence();
    }
    if constexpr (PAIRED && !careful) {
      meet();  // the other half has its softmax behind it
      load(own);
    }
    if constexpr (!masked) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) ahead[i] = read_v(tile, i % NC, i / NC);
      issue_fence();
    }
    if constexpr (masked) {
      const int limit = seen - key - 4 * lh;
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) p[n][e] = 32 * n + 8 * (e / 4) + e % 4 < limit ? p[n][e] : -INFINITY;
    }
    float top = p[0][0];
#pragma unroll
    for (int n = 0; n < NK; ++n)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = __builtin_elementwise_maximum(top, p[n][e]);
    top = __builtin_elementwise_maximum(top, other_half(top, lane));
    const bool grown = top * a.scale_log2 > kSlack || (fresh && top != -INFINITY);
    if (__builtin_amdgcn_ballot_w64(grown)) {
      const float by = grown ? top : 0.0f;
      const float f = grown && fresh ? 0.0f : __builtin_amdgcn_exp2f(-by * a.scale_log2);
      fresh = fresh && !grown;
      sum *= f;
      less -= by;
      if constexpr (!masked) {
#pragma unroll
        for (int e = 0; e < 16; ++e) every[e] -= by;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[c][e] = careful ? weigh(f, o[c][e]) : o[c][e] * f;
#pragma unroll
      for (int n = 0; n < NK; ++n)
#pragma unroll
        for (int e = 0; e < 16; ++e) p[n][e] -= by;
    }
    u4_t w[NK][2];
#pragma unroll
    for (int n = 0; n < NK; ++n) {
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        p[n][e] = __builtin_amdgcn_exp2f(fmaf(p[n][e], a.scale_log2, T::kHeadroom));
        sum += p[n][e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) w[n][e / 4][e % 4] = two<T>(p[n][2 * e], p[n][2 * e + 1]);
    }
    if constexpr (!careful) {
      if constexpr (PAIRED) wait_loads<2 * S::kLoads>(), meet();
      if constexpr (masked) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) ahead[i] = read_v(tile, i % NC, i / NC);
        issue_fence();
      }
#pragma unroll
      for (int i = 0; i < kValues; ++i) {
        o[i % NC] = T::mfma(ahead[i % kAhead], w[i / NC / 2][i / NC % 2], o[i % NC]);
        if (i + kAhead < kValues) ahead[i % kAhead] = read_v(tile, (i + kAhead) % NC, (i + kAhead) / NC);
        issue_fence();
      }
      return;
    }
    // finite values as usual, in the same order; of others, whether the row sees a +inf
    // (-inf, either for a NaN) in the channel
    const int limit = seen - key - 4 * lh;
#pragma unroll 1
    for (int x = 0; x < 2 * NK; ++x) {
      u4_t weight;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        weight[e] = x == 0 ? w[0][0][e] : (x == 1 ? w[0][1][e] : (x == 2 ? w[NK - 1][0][e] : w[NK - 1][1][e]));
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        u4_t v = read_v(tile, c, x);
        float test = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) test = T::dot(v[e], 0u, test);
        if (__builtin_amdgcn_ballot_w64(test != 0.0f)) {
          u4_t sees, plus, minus;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int at = 16 * x + 8 * (e / 2) + 2 * (e % 2);
            sees[e] = (at < limit ? T::kOne : 0u) | (at + 1 < limit ? T::kOne << 16 : 0u);
            uint32_t keep = 0, up = 0, down = 0;
#pragma unroll
            for (int b = 0; b < 32; b += 16) {
              const uint32_t bits = v[e] >> b & 0xFFFFu, size = bits & 0x7FFFu;
              if (size < T::kInf) keep |= bits << b;
              if (size > T::kInf || bits == T::kInf) up |= T::kOne << b;
              if (size > T::kInf || bits == (T::kInf | 0x8000u)) down |= T::kOne << b;
            }
            v[e] = keep, plus[e] = up, minus[e] = down;
          }
          f16_t zero;
#pragma unroll
          for (int e = 0; e < 16; ++e) zero[e] = 0;
          f16_t count = T::mfma(plus, sees, zero);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (count[e] > 0) o[c][e] += INFINITY;
          issue_fence();
          count = T::mfma(minus, sees, zero);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (count[e] > 0) o[c][e] -= INFINITY;
        }
        o[c] = T::mfma(v, weight, o[c]);
        issue_fence();
      }
    }
  };

  // every row of the block sees the keys of the first tiles; the others are masked
  const int all_see = keys_seen(a, s, block_row / a.share);
  const int plain = (all_see < piece1 ? all_see : piece1) - L::kKeys;
  constexpr int kStride = FEW ? kWaves * L::kKeys : L::kKeys;
  const int first_key = piece0 + (FEW ? wave * L::kKeys : 0);
  int key = first_key, stage = 0;
  // tiles of the next step on their way while one is worked on
  auto next = [&](int own) {
    wait_loads<0>();
    if constexpr (FEW) {
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the other stage is read
      issue_fence();
    } else {
      meet();  // everybody's part of this step's tiles is here, and nobody reads the other stage
    }
    if (key + kStride < piece1) load_k(key + kStride, stage ^ 1, own), load_v(key + kStride, stage ^ 1, own);
  };
  auto begin = [&](int own) {
    if (key < piece1) load_k(key, 0, own), load_v(key, 0, own);
  };
  const auto no_load = [](int) {};
  if constexpr (PAIRED) {
    // While one half multiplies (a tile's probabilities with V, the next one's keys
    // with Q), the other works on its softmax, on the same four SIMDs.  Loads run
    // three tiles ahead of the keys' use, two of the values'.
    auto load = [&](int own) {
      load_k(key + 3 * kStride, (stage + 3) & 3, own);
      load_v(key + 2 * kStride, stage ^ 2, own);
    };
    auto turn = [&]() { key += kStride, stage = (stage + 1) & 3; };
    if (key < piece1) {
      load_k(key, 0, lane), load_k(key + kStride, 1, lane), load_v(key, 0, lane);
      load_k(key + 2 * kStride, 2, lane), load_v(key + kStride, 1, lane);
      wait_loads<2 * S::kLoads>();
      meet();
      if (wave >= kWaves / 2) meet();
    }
#pragma unroll 1
    while (key <= plain) {
      step(key, stage, std::integral_constant<int, kPlain>(), load);
      turn();
    }
#pragma unroll 1
    while (key < piece1) {
      if (key < any_sees) {
        step(key, stage, std::integral_constant<int, kMasked>(), load);
      } else {
        meet();
        load(lane);
        wait_loads<2 * S::kLoads>();
        meet();
      }
      turn();
    }
    if (piece0 < piece1 && wave < kWaves / 2) meet();
    wait_loads<0>();
  } else {
    begin(lane);
    if constexpr (D == 256) {
      // In the other half of the registers, which matrix instructions read as they are: left
      // to itself the compiler copied some of it in every step (4096 tokens, 16 heads: 182 us, so 171).
#pragma unroll
      for (int c = 0; c < NQ; ++c) asm volatile("" : "+a"(q[c]));
    }
    auto turn = [&]() { key += kStride, stage ^= 1; };
#pragma unroll 1
    while (key <= plain) {
      next(lane);
      step(key, stage, std::integral_constant<int, kPlain>(), no_load);
      turn();
    }
#pragma unroll 1
    while (key < piece1) {
      int own = lane;
      asm volatile("" : "+v"(own));
      next(own);
      if (key < any_sees) step(key, stage, std::integral_constant<int, kMasked>(), no_load);
      turn();
    }
  }

  // 0 times a value that is not finite is a NaN: a row has one where it does not see
  // such a value, or sees it at a probability that is 0 in fp32.  If any row has (and
  // not by its scores, which make its sum a NaN too), the keys are gone through again,
  // with care.  Blocks decide together, since they share tiles.
  float all = sum + other_half(sum, lane);
  bool lost = false;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 16; ++e) lost |= o[c][e] != o[c][e];
  bool again = __builtin_amdgcn_ballot_w64(lost && all == all) != 0;
  if constexpr (!FEW) {
    uint32_t *const votes = reinterpret_cast<uint32_t *>(lds + S::kTiles);
    if (lane == 0) votes[wave] = again;
    __syncthreads();
    uint32_t any = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) any |= votes[w];
    again = __builtin_amdgcn_readfirstlane(any) != 0;
  }
  if (__builtin_expect(again, 0)) {
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[c][e] = 0;
    sum = 0, less = 0, fresh = true;
    key = first_key, stage = 0;
    int own = lane;
    asm volatile("" : "+v"(own));
    begin(own);
#pragma unroll 1
    while (key < piece1) {
      asm volatile("" : "+v"(own));
      next(own);
      if (key < any_sees) step(key, stage, std::integral_constant<int, kCareful>(), no_load);
      key += kStride, stage ^= 1;
    }
    all = sum + other_half(sum, lane);
  }
  sum = all;
  if constexpr (FEW) {
    // the waves join: references and sums first, then outputs at a common reference
    wait_loads<0>();
    __syncthreads();
    float *const ml = reinterpret_cast<float *>(lds), *const rows_at = ml + kWaves * kPromptRows * 2;
    if (lh == 0) {
      ml[(wave * kPromptRows + li) * 2] = fresh ? -FLT_MAX : -less;
      ml[(wave * kPromptRows + li) * 2 + 1] = sum;
    }
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f4_t *>(rows_at + (wave * kPromptRows + li) * S::kRowFloats + 32 * c + 8 * e + 4 * lh) =
            f4_t{o[c][4 * e], o[c][4 * e + 1], o[c][4 * e + 2], o[c][4 * e + 3]};
    __syncthreads();
    constexpr int kFour = D / 4;  // lanes of an output row
    for (int at = threadIdx.x; at < (rows < kPromptRows ? rows : kPromptRows) * kFour; at += 64 * kWaves) {
      const int r = at / kFour, x = at % kFour * 4, tr = r / a.share;
      float top = -FLT_MAX, l = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, ml[(w * kPromptRows + r) * 2]);
      f4_t y = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float lw = ml[(w * kPromptRows + r) * 2 + 1];
        // a wave of weight 0 counts: values that its rows see may not be finite
        const float f = lw == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((ml[(w * kPromptRows + r) * 2] - top) * a.scale_log2);
        l += f * lw;
        y += weigh(f, *reinterpret_cast<const f4_t *>(rows_at + (w * kPromptRows + r) * S::kRowFloats + x));
      }
      const int64_t out_row = ((int64_t)(s.q0 + tr) * a.kv_heads + head) * a.share + (r - tr * a.share);
      if (a.splits > 1) {
        const int64_t to = (int64_t)blockIdx.y * a.num_tokens * a.kv_heads * a.share + out_row;
        *reinterpret_cast<f4_t *>(a.part_o + to * D + x) = y;
        if (x == 0) a.part_ml[2 * to] = top, a.part_ml[2 * to + 1] = l;
      } else {
        const float f = over(l);
        *reinterpret_cast<u2_t *>(static_cast<uint16_t *>(a.out) + out_row * D + x) =
            u2_t{two<T>(y.x * f, y.y * f), two<T>(y.z * f, y.w * f)};
        if (a.lse && x == 0) a.lse[out_row] = lse_of(top, l, a.scale_log2, T::kHeadroom);
      }
    }
    return;
  }
  if (row >= rows) return;
  const int64_t out_row = (int64_t)(s.q0 + t) * a.kv_heads * a.share + q_head;
  if (a.splits > 1) {
    const int64_t at = (int64_t)blockIdx.y * a.num_tokens * a.kv_heads * a.share + out_row;
    float *to = a.part_o + at * D + 4 * lh;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *reinterpret_cast<f4_t *>(to + 32 * c + 8 * e) =
            f4_t{o[c][4 * e], o[c][4 * e + 1], o[c][4 * e + 2], o[c][4 * e + 3]};
    if (lh == 0) {
      a.part_ml[2 * at] = fresh ? -FLT_MAX : -less;
      a.part_ml[2 * at + 1] = sum;
    }
    return;
  }
  const float f = over(sum);
  uint16_t *to = static_cast<uint16_t *>(a.out) + out_row * D + 4 * lh;
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<u2_t *>(to + 32 * c + 8 * e) =
          u2_t{two<T>(o[c][4 * e] * f, o[c][4 * e + 1] * f), two<T>(o[c][4 * e + 2] * f, o[c][4 * e + 3] * f)};
  if (a.lse && lh == 0) a.lse[out_row] = lse_of(-less, sum, a.scale_log2, T::kHeadroom);
}

// Joins the pieces of a row: a block a row.  Its threads take the pieces'
// references and sums first, then D / 4 lanes an output of a piece.
constexpr int kJoinThreads = 256;
template <typename T, int D>
__global__ __launch_bounds__(kJoinThreads) void prompt_join_kernel(PromptKernelArgs a) {
  constexpr int kLanes = D / 4, kGroups = kJoinThreads / kLanes;
  __shared__ float weight[kMaxPromptSplits];
  __shared__ float waves[2][kJoinThreads / 64];
  __shared__ f4_t part[kJoinThreads];
  const int heads = a.kv_heads * a.share, lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const Sequence s = sequence_of(a, blockIdx.y);
  const int tokens = s.nq < a.max_q ? s.nq : a.max_q;
  if ((int64_t)blockIdx.x >= (int64_t)tokens * heads) return;
  const int64_t row = (int64_t)s.q0 * heads + blockIdx.x, all = (int64_t)a.num_tokens * heads;
  const int seen = keys_seen(a, s, (int)(blockIdx.x / heads));
  const int used = clamp_to((int)(((int64_t)seen + a.chunk - 1) / a.chunk), 1, a.splits);
  auto across = [&](float v, bool largest, int at) {  // of the whole block
#pragma unroll
    for (int x = 1; x < 64; x *= 2) {
      const float y = __shfl_xor(v, x);
      v = largest ? fmaxf(v, y) : v + y;
    }
    if (lane == 0) waves[at][wave] = v;
    __syncthreads();
    v = waves[at][0];
#pragma unroll
    for (int x = 1; x < kJoinThreads / 64; ++x) v = largest ? fmaxf(v, waves[at][x]) : v + waves[at][x];
    return v;
  };
  float top = -FLT_MAX, sum = 0;
  for (int p = threadIdx.x; p < used; p += kJoinThreads) top = fmaxf(top, a.part_ml[2 * (p * all + row)]);
  top = across(top, true, 0);
  for (int p = threadIdx.x; p < used; p += kJoinThreads) {
    const float *ml = a.part_ml + 2 * (p * all + row);
    const float f = ml[1] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f((ml[0] - top) * a.scale_log2);  // no key: 0
    weight[p] = f;
    sum += f * ml[1];
  }
  sum = across(sum, false, 1);
  const int x = threadIdx.x % kLanes * 4, group = threadIdx.x / kLanes;
  f4_t o = {0, 0, 0, 0};
#pragma unroll 4
  for (int p = group; p < used; p += kGroups)
    o += weigh(weight[p], *reinterpret_cast<const f4_t *>(a.part_o + (p * all + row) * D + x));  // pieces of weight 0 too
  part[threadIdx.x] = o;
  __syncthreads();
  if (group) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) o += part[g * kLanes + threadIdx.x];
  const float f = over(sum);
  *reinterpret_cast<u2_t *>(static_cast<uint16_t *>(a.out) + row * D + x) =
      u2_t{two<T>(o.x * f, o.y * f), two<T>(o.z * f, o.w * f)};
  if (a.lse && threadIdx.x == 0) a.lse[row] = lse_of(top, sum, a.scale_log2, T::kHeadroom);
}

template <typename T, int D, int ROWS>
hipError_t launch_shape(const PromptKernelArgs &a, hipStream_t stream) {
  typedef Shape<T, D, ROWS> S;
  const unsigned blocks = (unsigned)((int64_t)a.num_seqs * a.kv_heads * a.row_blocks);
  hipLaunchKernelGGL((prompt_kernel<T, D, ROWS>), dim3(blocks, a.splits), dim3(64 * S::kWaves), S::kLds, stream, a);
  if (a.splits > 1) {
    const int64_t rows = (int64_t)a.max_q * a.kv_heads * a.share;
    hipLaunchKernelGGL((prompt_join_kernel<T, D>), dim3((unsigned)rows, a.num_seqs), dim3(kJoinThreads), 0, stream, a);
  }
  return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_dim(const PromptKernelArgs &a, const PromptPlan &p, hipStream_t stream) {
  if constexpr (D == 128)
    if (p.rows == 8 * kPromptRows) return launch_shape<T, D, 8 * kPromptRows>(a, stream);
  return p.rows == kPromptRows ? launch_shape<T, D, kPromptRows>(a, stream) : launch_shape<T, D, 4 * kPromptRows>(a, stream);
}

template <typename T>
hipError_t launch_type(const PromptKernelArgs &a, const PromptPlan &p, int32_t head_dim, hipStream_t stream) {
  if (head_dim == 64) return launch_dim<T, 64>(a, p, stream);
  if (head_dim == 128) return launch_dim<T, 128>(a, p, stream);
  return launch_dim<T, 256>(a, p, stream);
}

}  // namespace

hipError_t launch_prompt_attention(const PromptKernelArgs &a, const PromptPlan &p, int32_t head_dim, int32_t dtype,
                                   hipStream_t stream) {
  return dtype == I4S_F16 ? launch_type<Half>(a, p, head_dim, stream) : launch_type<Brain>(a, p, head_dim, stream);
}

}  // namespace i4s
