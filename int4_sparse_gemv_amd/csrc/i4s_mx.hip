// Quantization to the microscaled 4-bit format and reading it back (format:
// include/i4s_prompt.h), for gfx950.
//
// A wave takes 16 rows x 512 columns, the scales of a tile group, or 4 rows of it.  Sixteen
// neighbouring lanes hold 128 neighbouring columns of a row, eight each (16
// bytes), so four lanes hold a block, whose largest magnitude two DPP steps
// find as whole-number bits.  A lane's eight codes are four bytes of the
// block's sixteen, and the rows 4i .. 4i+3 of a load lie next to each other in
// the tile: every store covers whole 64-byte pieces.
//
// Bound by memory: 2 bytes read and 0.53 written a value.  Values are read, and
// written where they are read back, past the caches (non-temporal): they are used
// once.  Quantizing and reading back 13824 x 5120: 67 us for 358 MB = 5.4 TB/s
// (through the caches 79), 2000 x 11008 22 us (31); a large copy runs at 4.8 TB/s.

#include "i4s_mx_common.h"

namespace i4s {
namespace {

constexpr int kMxThreads = 64;  // blocks of a wave: few rows reach more compute units
// Up to so many tile groups take four waves each, of four rows.  Us of quantizing and
// reading back, four waves / one, x 11008: 64 rows 5.1 / 9.2, 500 (704 groups) 7.8 / 11.5;
// quantizing alone in four, 1000 (1386) 16.9 / 15.1, 2000 25.2 / 22.9.  1 x 4096 4.2 / 6.0.
constexpr unsigned kFewUnits = 1024;

template <typename X, int PARTS>  // PARTS of four rows by this wave, of the tile's four
__global__ __launch_bounds__(kMxThreads) void mx_quantize_kernel(MxQuantizeArgs a) {
  const int groups = mx_groups(a.cols), steps = mx_steps(a.cols);
  const int64_t tile = blockIdx.x / (unsigned)groups;
  const int group = blockIdx.x % (unsigned)groups;
  const int lane = threadIdx.x, col = lane % 16 * 8, sub = lane / 16, quad = lane % 4, block = lane % 16 / 4;
  const int left = steps - 4 * group < 4 ? steps - 4 * group : 4;  // tiles of this group
  const uint16_t *x = static_cast<const uint16_t *>(a.x);
  const int first = PARTS == 4 ? 0 : blockIdx.y * PARTS;
  u4_t v[4][PARTS];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const int64_t row = tile * kMxRows + 4 * (first + i) + sub;
      const int at = group * kMxGroup + c * kMxStep + col;
      v[c][i] = u4_t{0, 0, 0, 0};
      if (row < a.rows && at < a.cols)
        v[c][i] = __builtin_nontemporal_load(reinterpret_cast<const u4_t *>(x + row * a.stride + at));
    }
  uint32_t scales[PARTS] = {};
  uint8_t *vals = a.vals + (tile * steps + 4 * group) * kMxTileBytes + block * 256 + quad * 4;
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      const uint32_t pair = quad_max(top_bits(v[c][i]));
      const uint32_t top = (pair & 0xFFFFu) > pair >> 16 ? pair & 0xFFFFu : pair >> 16;
      const uint32_t byte = scale_byte<X>(top);
      scales[i] |= byte << (8 * c);
      const uint32_t word = byte == kMxNaN ? 0u : codes<X>(v[c][i], scale_value(byte));
      const int row = 4 * (first + i) + sub;
      if (c < left && tile * kMxRows + row < a.rows)
        *reinterpret_cast<uint32_t *>(vals + c * kMxTileBytes + row * 16) = word;
    }
  // the quad's lanes hold the same scale words: each stores one
  uint32_t word = scales[0];
#pragma unroll
  for (int i = 1; i < PARTS; ++i) word = quad == i ? scales[i] : word;
  const int row = 4 * (first + quad) + sub;
  if (quad < PARTS && tile * kMxRows + row < a.rows)
    *reinterpret_cast<uint32_t *>(a.scales + (tile * groups + group) * kMxGroupBytes + (block * 16 + row) * 4) = word;
}

// Values 2i and 2i + 1 of a word of codes.
typedef float f2_t __attribute__((ext_vector_type(2)));
template <int B>
__device__ inline f2_t two_values(uint32_t word) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(word, 1.0f, B);
}

struct AsHalf {
  typedef uint16_t type;
  static __device__ uint16_t of(float f) { return (uint16_t)float_to_fp16_bits(f); }
};
struct AsBrain {
  typedef uint16_t type;
  static __device__ uint16_t of(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};
struct AsFloat {
  typedef float type;
  static __device__ float of(float f) { return f; }
};

template <typename Y, int PARTS>
__global__ __launch_bounds__(kMxThreads) void mx_read_kernel(MxReadArgs a) {
  typedef typename Y::type T;
  const int groups = mx_groups(a.cols), steps = mx_steps(a.cols);
  const int64_t tile = blockIdx.x / (unsigned)groups;
  const int group = blockIdx.x % (unsigned)groups;
  const int lane = threadIdx.x, col = lane % 16 * 8, sub = lane / 16, quad = lane % 4, block = lane % 16 / 4;
  const uint8_t *vals = a.vals + (tile * steps + 4 * group) * kMxTileBytes + block * 256 + quad * 4;
  const uint8_t *scales = a.scales + (tile * groups + group) * kMxGroupBytes + block * 64;
  T *out = static_cast<T *>(a.out);
  const int first = PARTS == 4 ? 0 : blockIdx.y * PARTS;
#pragma unroll
  for (int i = 0; i < PARTS; ++i) {
    const int in = 4 * (first + i) + sub;
    const int64_t row = tile * kMxRows + in;
    if (row >= a.rows) continue;
    const uint32_t four = *reinterpret_cast<const uint32_t *>(scales + in * 4);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int at = group * kMxGroup + c * kMxStep + col;
      if (at >= a.cols) continue;
      const uint32_t word = *reinterpret_cast<const uint32_t *>(vals + c * kMxTileBytes + in * 16);
      const uint32_t byte = four >> (8 * c) & 255u;
      const float scale = byte == kMxNaN ? __builtin_nanf("") : scale_value(byte);
      const f2_t p[4] = {two_values<0>(word), two_values<1>(word), two_values<2>(word), two_values<3>(word)};
      constexpr int kMany = 16 / sizeof(T);  // 16 bytes a store: out's alignment
      typedef T vec __attribute__((ext_vector_type(kMany)));
#pragma unroll
      for (int h = 0; h < 8; h += kMany) {
        vec y;
#pragma unroll
        for (int e = 0; e < kMany; ++e) y[e] = Y::of(p[(h + e) / 2][e % 2] * scale);
        __builtin_nontemporal_store(y, reinterpret_cast<vec *>(out + row * a.cols + at + h));
      }
    }
  }
}

}  // namespace

static dim3 mx_blocks(int32_t rows, int32_t cols) { return dim3((unsigned)((int64_t)mx_row_tiles(rows) * mx_groups(cols))); }

template <typename X>
static hipError_t launch_quantize(const MxQuantizeArgs &a, hipStream_t stream) {
  dim3 grid = mx_blocks(a.rows, a.cols);
  if (grid.x <= kFewUnits) {
    grid.y = 4;
    hipLaunchKernelGGL((mx_quantize_kernel<X, 1>), grid, dim3(kMxThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((mx_quantize_kernel<X, 4>), grid, dim3(kMxThreads), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_mx_quantize(const MxQuantizeArgs &a, int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16 ? launch_quantize<HalfX>(a, stream) : launch_quantize<BrainX>(a, stream);
}

template <typename Y>
static hipError_t launch_read(const MxReadArgs &a, hipStream_t stream) {
  dim3 grid = mx_blocks(a.rows, a.cols);
  if (grid.x <= kFewUnits) {
    grid.y = 4;
    hipLaunchKernelGGL((mx_read_kernel<Y, 1>), grid, dim3(kMxThreads), 0, stream, a);
  } else {
    hipLaunchKernelGGL((mx_read_kernel<Y, 4>), grid, dim3(kMxThreads), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_mx_read(const MxReadArgs &a, int32_t dtype, hipStream_t stream) {
  if (dtype == I4S_F16) return launch_read<AsHalf>(a, stream);
  return dtype == I4S_BF16 ? launch_read<AsBrain>(a, stream) : launch_read<AsFloat>(a, stream);
}

}  // namespace i4s
