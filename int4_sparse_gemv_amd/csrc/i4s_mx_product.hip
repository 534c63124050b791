// Products y = X W^T of matrices in the microscaled 4-bit format (format:
// include/i4s_prompt.h), for gfx950.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies 16 weight rows by 16 tokens
// over 128 columns, 65536 operations in 16 cycles of a SIMD: lane 16 b + r
// brings row (token) r's columns 32 b .. 32 b + 31, 16 bytes, and their scale,
// one byte of a register that an immediate picks.  The format keeps both in that
// order: a tile's values are one 16-byte load per lane, its scales for four
// tiles one 4-byte load.  Lane 16 a + n of the result holds token n, rows 4 a
// .. 4 a + 3.  Sums are fp32 from first to last; a product of two codes and
// two powers of two is exact.

#include <type_traits>

#include "i4s_mx_common.h"

namespace i4s {
namespace {

typedef int i8_t __attribute__((ext_vector_type(8)));
typedef float f4_t __attribute__((ext_vector_type(4)));

// One matrix instruction: scale byte C of sa and sb.  Format 4 is e2m1, which
// takes half of the registers.
template <int C>
__device__ inline f4_t mx_mfma(u4_t a, uint32_t sa, u4_t b, uint32_t sb, f4_t c) {
  const i8_t wa = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0};
  const i8_t wb = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, 4, 4, C, (int)sa, C, (int)sb);
}

__device__ inline u4_t load16(const void *p) { return *static_cast<const u4_t *>(p); }
__device__ inline uint32_t load4(const void *p) { return *static_cast<const uint32_t *>(p); }

struct YHalf {
  typedef uint16_t type;
  static __device__ uint16_t of(float f) { return (uint16_t)float_to_fp16_bits(f); }
};
struct YBrain {
  typedef uint16_t type;
  static __device__ uint16_t of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
struct YFloat {
  typedef float type;
  static __device__ float of(float f) { return f; }
};

// ---------------------------------------------------------------------------
// few tokens: the weight's bytes are the time
//
// A block takes RT weight tiles and up to 16 * NT tokens; its waves take the
// groups of 512 columns in turn, the next one's tiles on their way while one is
// multiplied, and join their sums in LDS.
//
// 16-bit tokens are quantized on the way, each wave the columns that it
// multiplies: a token's 512 columns are one 16-byte load per lane, four
// neighbouring lanes hold a block, and codes and scales pass through the wave's
// own LDS into the matrix instruction's order.  Their loads go out first: they
// come from L2, and loads return in order.
//
// ONCE: no other block reads the same weights, which then pass by the caches.
// Us, so / through them: 50257 x 4096, 16 tokens 22.0 / 24.0, 37 tokens 29.1 / 30.6;
// 13824 x 5120, 48 tokens 11.9 / 12.8; 4096 x 4096, 16 tokens 3.8 / 3.7 (from the
// last-level cache); 200 tokens in four blocks, 9.8 / 9.2.
// Bound by memory: 50257 x 4096 with 16 tokens reads 5.8 TB/s behind 2.5 us of
// launch and first loads; more tokens cost their reads from L2 by every block, which
// for 48 are more than the weights (more weight tiles a block: registers do not
// reach; one and two waves a block: 33 to 36 us for 37 tokens).

// One group's tiles in registers.
template <int N>
struct Operand {
  u4_t v[N][4];
  uint32_t s[N];
};

template <int N, bool STREAM>
__device__ inline void load_operand(Operand<N> &o, const uint8_t *vals, const uint8_t *scales, int first, int tiles, int steps,
                                    int groups, int group, int lane) {
  const int left = steps - 4 * group;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t tile = first + i < tiles ? first + i : tiles - 1;
    const uint8_t *sp = scales + (tile * groups + group) * kMxGroupBytes + lane * 4;
    o.s[i] = STREAM ? __builtin_nontemporal_load(reinterpret_cast<const uint32_t *>(sp)) : load4(sp);
    const uint8_t *p = vals + (tile * steps + 4 * group) * kMxTileBytes + lane * 16;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (c < 2 || left > 2) {
        if constexpr (STREAM)
          o.v[i][c] = __builtin_nontemporal_load(reinterpret_cast<const u4_t *>(p + c * kMxTileBytes));
        else
          o.v[i][c] = load16(p + c * kMxTileBytes);
      }
  }
}

// 16-bit tokens, BATCH of them on their way together.  Us for 4 / 8 / 16: 13824 x
// 5120, 16 tokens 13.9 / 13.1 / 12.5; 4096 x 4096, 16: 7.1 / 6.7 / 7.0, one token 3.7 /
// 3.8 / 3.9; 22016 x 4096, 16: 17.2 / 16.2 / 19.0.
template <typename X, int BATCH>
struct Batch : X {
  static constexpr int kBatch = BATCH;
};
struct Given {  // tokens in the format
  static constexpr int kBatch = 1;
};

template <typename X, typename Y, int RT, int NT, int WAVES, bool ONCE>
__global__ __launch_bounds__(WAVES * 64) void mx_few_kernel(MxProductKernelArgs a) {
  constexpr bool kFused = !std::is_same<X, Given>::value;
  constexpr int kBatch = X::kBatch;
  __shared__ float sums[WAVES][RT * NT][72][4];  // 16 lanes and two empty places: rows read together lie in other banks
  __shared__ uint32_t own[kFused ? WAVES : 1][kFused ? 5 : 1][64][4];  // four tiles, and in the fifth place the scales
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int steps = mx_steps(a.cols), groups = mx_groups(a.cols), tiles = mx_row_tiles(a.rows);
  const int first = blockIdx.x * RT;
  f4_t acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f4_t{0, 0, 0, 0};

  u4_t raw[kBatch];
  auto load_tokens = [&](int g, int t0) {
    const int at = g * kMxGroup + lane * 8;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      raw[i] = u4_t{0, 0, 0, 0};
      if (t0 + i < a.tokens && at < a.cols)
        raw[i] = load16(static_cast<const uint16_t *>(a.x) + (t0 + i) * a.x_stride + at);
    }
  };
  Operand<RT> w;
  Operand<NT> x;
  auto load = [&](int g) {
    if constexpr (kFused) load_tokens(g, 0);
    load_operand<RT, ONCE>(w, a.w_vals, a.w_scales, first, tiles, steps, groups, g, lane);
    if constexpr (!kFused)
      load_operand<NT, false>(x, a.x_vals, a.x_scales, blockIdx.y * NT, mx_row_tiles(a.tokens), steps, groups, g, lane);
  };
  if (wave < groups) load(wave);
  for (int g = wave; g < groups; g += WAVES) {
    const Operand<RT> u = w;
    Operand<NT> t = x;
    if constexpr (kFused) {
      // lane = 16 c + 4 b + quad: step c, block b
      uint32_t *codes_at = &own[wave][lane / 16][lane / 4 % 4 * 16][lane % 4];
      uint8_t *scale_at = reinterpret_cast<uint8_t *>(own[wave][4]) + lane / 4 % 4 * 64 + lane / 16;
      for (int t0 = 0; t0 < a.tokens; t0 += kBatch) {
        if (t0) load_tokens(g, t0);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (t0 + i < a.tokens) {
            const uint32_t pair = quad_max(top_bits(raw[i]));
            const uint32_t byte = scale_byte<X>((pair & 0xFFFFu) > pair >> 16 ? pair & 0xFFFFu : pair >> 16);
            codes_at[(t0 + i) * 4] = byte == kMxNaN ? 0u : codes<X>(raw[i], scale_value(byte));
            if (lane % 4 == 0) scale_at[(t0 + i) * 4] = (uint8_t)byte;
          }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      t.s[0] = reinterpret_cast<const uint32_t *>(own[wave][4])[lane];
#pragma unroll
      for (int c = 0; c < 4; ++c) t.v[0][c] = load16(own[wave][c][lane]);
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (g + WAVES < groups) load(g + WAVES);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        acc[r][n] = mx_mfma<0>(u.v[r][0], u.s[r], t.v[n][0], t.s[n], acc[r][n]);
        acc[r][n] = mx_mfma<1>(u.v[r][1], u.s[r], t.v[n][1], t.s[n], acc[r][n]);
        if (steps - 4 * g > 2) {
          acc[r][n] = mx_mfma<2>(u.v[r][2], u.s[r], t.v[n][2], t.s[n], acc[r][n]);
          acc[r][n] = mx_mfma<3>(u.v[r][3], u.s[r], t.v[n][3], t.s[n], acc[r][n]);
        }
      }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<f4_t *>(sums[wave][r * NT + n][lane + lane / 16 * 2]) = acc[r][n];
  __syncthreads();
  // neighbouring rows of a token go out together
  typename Y::type *y = static_cast<typename Y::type *>(a.y);
  for (int at = threadIdx.x; at < RT * NT * 256; at += WAVES * 64) {
    const int row = at % (16 * RT), token = at / (16 * RT);
    const int r = row / 16, n = token / 16, from = row % 16 / 4 * 18 + token % 16;
    float s = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) s += sums[w][r * NT + n][from][row % 4];
    const int64_t out = (int64_t)first * 16 + row, t = (int64_t)blockIdx.y * NT * 16 + token;
    if (t < a.tokens && out < a.rows) y[t * a.y_stride + out] = Y::of(s);
  }
}

// ---------------------------------------------------------------------------
// many tokens: the matrix instructions are the time
//
// A block of WR x WC waves takes WR*RT weight tiles x WC*NT token tiles; a
// wave RT x NT of them.  Tiles go to LDS directly (global_load_lds), a step of
// 128 columns at a time, into a ring of kRing steps; scales a group of four
// steps at a time, into two areas.  A barrier before a step's loads sees to it
// that every wave has read the step whose place they take, and the waits before
// it that every wave's part of the step that is read next is there.
//
// 8191 x 13824 x 5120: 270 us = 4.3 PFLOP/s; 8192^3 235, 4.7.  Bound by power: matrix
// instructions alone on the same data run at 6.2 PFLOP/s and 1.5 GHz, and here
// too the clock falls to 1.5 GHz, with the matrix cores busy 54 to 64 % of the cycles.
// The stores take 5 us of a round of 256 blocks of 256 x 256.  All eight waves in
// step, reading and then multiplying: 7 to 14 % slower (8192^3: 292 us, half a
// step apart 257, with the loads among the products 250).  Four waves with
// 128 x 128 outputs each: the same as that.  128 neighbouring bytes of a token
// in a store instead of 64, or non-temporal ones: no faster.

constexpr int kRing = 4;

typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) const void global_void;
__device__ inline void copy16(const void *from, char *to) {
  __builtin_amdgcn_global_load_lds((global_void *)from, (lds_void *)to, 16, 0, 0);
}
template <int N>
__device__ inline void wait_loads() {
  issue_fence();
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | (N >> 4 << 14));
  issue_fence();
}
// Waves meet; LDS reads before it are done (their values are in use), direct
// loads have been waited for.
__device__ inline void meet() {
  issue_fence();
  __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  issue_fence();
}

template <int RT, int NT, int WR, int WC>
struct TileShape {
  static constexpr int kWaves = WR * WC, kThreads = 64 * kWaves;
  static constexpr int kA = WR * RT, kB = WC * NT;          // weight and token tiles of a block
  static constexpr int kStep = (kA + kB) * kMxTileBytes;    // LDS bytes of a step
  static constexpr int kScales = (kA + kB) * kMxGroupBytes; // LDS bytes of a group's scales
  static constexpr int kLds = kRing * kStep + 2 * kScales;
  static constexpr int kLoads = (kA + kB) / kWaves;         // load instructions of a wave and step
  static_assert((kA + kB) % kWaves == 0, "tiles of a step are dealt evenly");
  static constexpr bool kTwice = RT * NT <= 16;              // registers for two steps' operands
  static constexpr int kScaleLoads = (kScales / 1024 + kWaves - 1) / kWaves;
};

// The block's place: consecutive blocks go to the eight XCDs in turn; each XCD
// takes a contiguous range of places, ordered in bands of kBand weight tiles, so
// that blocks that run together share what its L2 holds.
constexpr int kBand = 8;
struct Place {
  int row, token;
};
__device__ inline Place place_of(int id, int rows, int tokens) {
  const int n = rows * tokens, per = n / 8, more = n % 8, xcd = id % 8;
  const int at = id / 8 + xcd * per + (xcd < more ? xcd : more);
  const int band = at / (kBand * tokens), in = at - band * kBand * tokens;
  const int wide = rows - band * kBand < kBand ? rows - band * kBand : kBand;
  return {band * kBand + in % wide, in / wide};
}

// Eight neighbouring values of y as 16 bits: of two 16-row tiles of a lane's
// token, rows 4 b .. 4 b + 3 of either in the lanes 16 b + n, lanes 16 b + n
// get the rows 8 b .. 8 b + 7 of the 32.
template <typename Y>
__device__ inline u4_t eight_rows(f4_t lo, f4_t hi) {
  u4_t r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = Y::of(lo[2 * i]) | (uint32_t)Y::of(lo[2 * i + 1]) << 16;
    const uint32_t y = Y::of(hi[2 * i]) | (uint32_t)Y::of(hi[2 * i + 1]) << 16;
    const auto s = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    const auto t = __builtin_amdgcn_permlane16_swap(s[0], s[1], false, false);
    r[i] = t[0], r[2 + i] = t[1];
  }
  return r;
}
// 16 bytes at the alignment of an element.
typedef u4_t loose_t __attribute__((aligned(2)));

template <typename Y, int RT, int NT, int WR, int WC>
__global__ __launch_bounds__(64 * WR *WC, 2) void mx_tile_kernel(MxProductKernelArgs a) {
  typedef TileShape<RT, NT, WR, WC> S;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), lane = threadIdx.x & 63;
  const int all = mx_steps(a.cols), groups_all = mx_groups(a.cols);
  const int row_tiles = mx_row_tiles(a.rows), token_tiles = mx_row_tiles(a.tokens);
  const Place place = place_of(blockIdx.x, (row_tiles + S::kA - 1) / S::kA, (token_tiles + S::kB - 1) / S::kB);
  const int row0 = place.row * S::kA, token0 = place.token * S::kB;
  const int last = all - 1;

  // the tiles that this wave brings
  const uint8_t *from[S::kLoads];
#pragma unroll
  for (int i = 0; i < S::kLoads; ++i) {
    const int t = wave * S::kLoads + i;
    if (t < S::kA) {
      const int64_t tile = row0 + t < row_tiles ? row0 + t : row_tiles - 1;
      from[i] = a.w_vals + tile * all * kMxTileBytes + lane * 16;
    } else {
      const int64_t tile = token0 + t - S::kA < token_tiles ? token0 + t - S::kA : token_tiles - 1;
      from[i] = a.x_vals + tile * all * kMxTileBytes + lane * 16;
    }
  }
  // and the scales: 16 lanes a tile
  const uint8_t *scales_from[S::kScaleLoads];
#pragma unroll
  for (int i = 0; i < S::kScaleLoads; ++i) {
    int t = (wave * S::kScaleLoads + i) * 4 + lane / 16;
    if (t >= S::kA + S::kB) t = S::kA + S::kB - 1;
    if (t < S::kA) {
      const int64_t tile = row0 + t < row_tiles ? row0 + t : row_tiles - 1;
      scales_from[i] = a.w_scales + tile * groups_all * kMxGroupBytes + lane % 16 * 16;
    } else {
      const int64_t tile = token0 + t - S::kA < token_tiles ? token0 + t - S::kA : token_tiles - 1;
      scales_from[i] = a.x_scales + tile * groups_all * kMxGroupBytes + lane % 16 * 16;
    }
  }
  char *const ring = lds;
  char *const scale_area = lds + kRing * S::kStep;
  auto load_tile = [&](int step, int i) {
    copy16(from[i] + (int64_t)(step < last ? step : last) * kMxTileBytes,
           ring + (step & (kRing - 1)) * S::kStep + (wave * S::kLoads + i) * kMxTileBytes);
  };
  auto load_step = [&](int step) {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) load_tile(step, i);
  };
  auto load_scales = [&](int group) {
    const int64_t at = (int64_t)(group < groups_all ? group : groups_all - 1) * kMxGroupBytes;
#pragma unroll
    for (int i = 0; i < S::kScaleLoads; ++i) {
      const int piece = wave * S::kScaleLoads + i;
      if (S::kScales / 1024 == S::kWaves * S::kScaleLoads || piece < S::kScales / 1024)
        copy16(scales_from[i] + at, scale_area + (group & 1) * S::kScales + piece * 1024);
    }
  };

  const int wr = wave / WC, wc = wave % WC;
  f4_t acc[RT][NT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[r][n] = f4_t{0, 0, 0, 0};

  auto run = [&](auto step) {
    for (int g = 0; g < groups_all; ++g) {
      step(4 * g, std::integral_constant<int, 0>());
      step(4 * g + 1, std::integral_constant<int, 1>());
      if (4 * g + 2 < all) {
        step(4 * g + 2, std::integral_constant<int, 2>());
        step(4 * g + 3, std::integral_constant<int, 3>());
      }
    }
  };
  if constexpr (S::kTwice) {
    // Operands in two sets of registers, read a step ahead between this step's
    // products, where a SIMD has one wave and nothing else to do meanwhile.
    u4_t va[2][RT], vb[2][NT];
    uint32_t sa[RT], sb[NT], next_sa[RT], next_sb[NT];
    auto read_a = [&](int set, int s, int r) {
      va[set][r] = load16(ring + (s & (kRing - 1)) * S::kStep + (wr * RT + r) * kMxTileBytes + lane * 16);
    };
    auto read_b = [&](int set, int s, int n) {
      vb[set][n] = load16(ring + (s & (kRing - 1)) * S::kStep + (S::kA + wc * NT + n) * kMxTileBytes + lane * 16);
    };
    auto read_scales = [&](uint32_t *pa, uint32_t *pb, int g) {
      const char *p = scale_area + (g & 1) * S::kScales + lane * 4;
#pragma unroll
      for (int r = 0; r < RT; ++r) pa[r] = load4(p + (wr * RT + r) * kMxGroupBytes);
#pragma unroll
      for (int n = 0; n < NT; ++n) pb[n] = load4(p + (S::kA + wc * NT + n) * kMxGroupBytes);
    };
    load_scales(0);
#pragma unroll
    for (int i = 0; i < kRing; ++i) load_step(i);
    wait_loads<(kRing - 1) * S::kLoads>();
    meet();
    read_scales(sa, sb, 0);
#pragma unroll
    for (int n = 0; n < NT; ++n) read_b(0, 0, n);
#pragma unroll
    for (int r = 0; r < RT; ++r) read_a(0, 0, r);
    run([&](int s, auto C) {
      constexpr int c = decltype(C)::value, set = c & 1;
      // two more steps (and scales) are on their way behind the next one
      wait_loads<2 * S::kLoads>();
      meet();  // this step's tiles are in registers: their place takes the fourth step from here
      if (c == 0) load_scales(s / 4 + 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = mx_mfma<c>(va[set][r], sa[r], vb[set][n], sb[n], acc[r][n]);
#pragma unroll
        for (int i = r * S::kLoads / RT; i < (r + 1) * S::kLoads / RT; ++i) load_tile(s + kRing, i);
        if (c == 3 && r == 0) read_scales(next_sa, next_sb, s / 4 + 1);
        read_a(set ^ 1, s + 1, r);
#pragma unroll
        for (int n = r * NT / RT; n < (r + 1) * NT / RT; ++n) read_b(set ^ 1, s + 1, n);
      }
      if (c == 3) {
#pragma unroll
        for (int r = 0; r < RT; ++r) sa[r] = next_sa[r];
#pragma unroll
        for (int n = 0; n < NT; ++n) sb[n] = next_sb[n];
      }
    });
  } else {
    // A SIMD has two waves, one of either half of the rows, and the halves are half a
    // step apart: while one multiplies, the other reads its operands from LDS.
    static_assert(WR == 2 && S::kWaves == 8, "wave and wave + 4 share a SIMD");
    load_scales(0);
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) load_step(i);
    uint32_t sa[RT], sb[NT];
    wait_loads<2 * S::kLoads>();
    meet();
    if (wr) meet();
    run([&](int s, auto C) {
      constexpr int c = decltype(C)::value;
      const char *base = ring + (s & (kRing - 1)) * S::kStep + lane * 16;
      if (c == 0) {
        const char *p = scale_area + (s / 4 & 1) * S::kScales + lane * 4;
#pragma unroll
        for (int r = 0; r < RT; ++r) sa[r] = load4(p + (wr * RT + r) * kMxGroupBytes);
#pragma unroll
        for (int n = 0; n < NT; ++n) sb[n] = load4(p + (S::kA + wc * NT + n) * kMxGroupBytes);
      }
      u4_t va[RT], vb[NT];
#pragma unroll
      for (int n = 0; n < NT; ++n) vb[n] = load16(base + (S::kA + wc * NT + n) * kMxTileBytes);
#pragma unroll
      for (int r = 0; r < RT; ++r) va[r] = load16(base + (wr * RT + r) * kMxTileBytes);
      // the next step's loads (and scales) are done behind this, one more step's on their way
      wait_loads<S::kLoads>();
      meet();  // the operands are in registers, and so are the other half's of the step before
      if (c == 0) load_scales(s / 4 + 1);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
#pragma unroll
        for (int n = 0; n < NT; ++n) acc[r][n] = mx_mfma<c>(va[r], sa[r], vb[n], sb[n], acc[r][n]);
#pragma unroll
        for (int i = r * S::kLoads / RT; i < (r + 1) * S::kLoads / RT; ++i) load_tile(s + kRing - 1, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      meet();
    });
    if (!wr) meet();
  }
  wait_loads<0>();

  // 16 bytes a lane, 64 neighbouring bytes of a token an instruction, at whatever
  // alignment y has
  typedef typename Y::type T;
  typedef typename std::conditional<sizeof(T) == 4, uint32_t, uint16_t>::type W;
  constexpr int kMany = 16 / sizeof(T), kTiles = kMany / 4;
  const int64_t row_at = (int64_t)(row0 + wr * RT) * 16 + lane / 16 * kMany;
  const int64_t token_at = (int64_t)(token0 + wc * NT) * 16 + lane % 16;
  T *const to = static_cast<T *>(a.y) + token_at * a.y_stride + row_at;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < RT; r += kTiles) {
      u4_t v;
      if constexpr (kTiles == 1)
        v = __builtin_bit_cast(u4_t, acc[r][n]);
      else
        v = eight_rows<Y>(acc[r][n], acc[r + 1][n]);
      T *const p = to + 16 * n * a.y_stride + 16 * r;
      const int64_t left = a.rows - (row_at + 16 * r);
      if (token_at + 16 * n >= a.tokens) continue;
      if (left >= kMany) {
        *reinterpret_cast<loose_t *>(p) = v;
      } else {
#pragma unroll
        for (int i = 0; i < kMany; ++i)
          if (i < left) reinterpret_cast<W *>(p)[i] = (W)(kTiles == 1 ? v[i % 4] : v[i / 2] >> (16 * (i % 2)));
      }
    }
}

template <typename X, typename Y, int RT, int NT, int WAVES, bool ONCE = true>
hipError_t launch_few_shape(const MxProductKernelArgs &a, hipStream_t stream) {
  const dim3 grid((mx_row_tiles(a.rows) + RT - 1) / RT, (mx_row_tiles(a.tokens) + NT - 1) / NT);
  hipLaunchKernelGGL((mx_few_kernel<X, Y, RT, NT, WAVES, ONCE>), grid, dim3(64 * WAVES), 0, stream, a);
  return hipGetLastError();
}

template <typename X, typename Y, int NT>
hipError_t launch_few_tokens(const MxProductKernelArgs &a, const MxProductPlan &p, hipStream_t stream) {
  if (p.waves == 4) return launch_few_shape<X, Y, 2, NT, 4>(a, stream);
  if constexpr (!std::is_same<X, Given>::value)
    if (p.row_tiles == 4) return launch_few_shape<X, Y, 4, NT, 8>(a, stream);
  return p.row_tiles == 1 ? launch_few_shape<X, Y, 1, NT, 8>(a, stream) : launch_few_shape<X, Y, 2, NT, 8>(a, stream);
}

template <typename Y>
hipError_t launch_few(const MxProductKernelArgs &a, const MxProductPlan &p, hipStream_t stream) {
  if (a.x) {
    if (a.tokens <= 4)
      return a.x_dtype == I4S_F16 ? launch_few_tokens<Batch<HalfX, 4>, Y, 1>(a, p, stream)
                                  : launch_few_tokens<Batch<BrainX, 4>, Y, 1>(a, p, stream);
    return a.x_dtype == I4S_F16 ? launch_few_tokens<Batch<HalfX, 8>, Y, 1>(a, p, stream)
                                : launch_few_tokens<Batch<BrainX, 8>, Y, 1>(a, p, stream);
  }
  switch (p.token_tiles) {
    case 1: return launch_few_tokens<Given, Y, 1>(a, p, stream);
    case 2: return launch_few_tokens<Given, Y, 2>(a, p, stream);
    case 3: return launch_few_tokens<Given, Y, 3>(a, p, stream);
    case 4: return launch_few_tokens<Given, Y, 4>(a, p, stream);
    default: return launch_few_shape<Given, Y, 2, 4, 4, false>(a, stream);
  }
}

template <typename Y, int RT, int NT, int WR, int WC>
hipError_t launch_tiles(const MxProductKernelArgs &a, hipStream_t stream) {
  typedef TileShape<RT, NT, WR, WC> S;
  const int64_t blocks = (int64_t)((mx_row_tiles(a.rows) + S::kA - 1) / S::kA) * ((mx_row_tiles(a.tokens) + S::kB - 1) / S::kB);
  hipLaunchKernelGGL((mx_tile_kernel<Y, RT, NT, WR, WC>), dim3((unsigned)blocks), dim3(S::kThreads), S::kLds, stream, a);
  return hipGetLastError();
}

template <typename Y>
hipError_t launch_product(const MxProductKernelArgs &a, const MxProductPlan &p, hipStream_t stream) {
  if (p.few) return launch_few<Y>(a, p, stream);
  if (p.tile == 256) return launch_tiles<Y, 8, 4, 2, 4>(a, stream);
  if (p.tile == 64) return launch_tiles<Y, 2, 4, 2, 2>(a, stream);
  return launch_tiles<Y, 4, 4, 2, 2>(a, stream);
}

}  // namespace

hipError_t launch_mx_product(const MxProductKernelArgs &a, const MxProductPlan &p, int32_t y_dtype, hipStream_t stream) {
  if (y_dtype == I4S_F16) return launch_product<YHalf>(a, p, stream);
  if (y_dtype == I4S_BF16) return launch_product<YBrain>(a, p, stream);
  return launch_product<YFloat>(a, p, stream);
}

}  // namespace i4s
