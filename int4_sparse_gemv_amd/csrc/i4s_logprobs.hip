// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits (include/i4s_serve.h), for gfx950.
//
// One pass: a block of 256 threads takes a slice of a row, 32 values per
// thread in registers, and computes from those registers the slice's maximum,
// the sums of exp(x - m) and (x - m) exp(x - m), and its largest k values;
// the slices of a row join through the running maximum m.  A block walks over
// the slices of its piece of the row; where there are few rows a row is split
// into pieces, which a second launch joins.
//
// Top k.  The k-th largest of the 64 lane maxima of a wave is a lower bound T
// of the k-th largest value, found bit by bit with ballots; the largest such
// T of the block's waves (and the k-th best of the slices before) leaves a
// few more than k candidates.  They go to LDS as 64-bit keys (value, then
// falling index), and a candidate's place is the number of keys above it.  Of
// the values equal to T only the first k of a wave in index order are taken,
// so that the number of candidates is bounded however many values are equal:
// fewer than k lanes of a wave have a maximum above T.
//
// Bound by: memory (2 or 4 bytes a value) when there are many rows, latency
// when there are few.

#include <float.h>

#include "i4s_serve_internal.h"

namespace i4s {
namespace {

typedef uint32_t w4_t __attribute__((ext_vector_type(4)));

constexpr int kBlock = 256, kBlockWaves = kBlock / 64;
constexpr int kValues = 32;                 // values of a thread in a slice
constexpr int kSlice = kBlock * kValues;    // values of a slice
constexpr int kMaxCandidates = kBlockWaves * (I4S_MAX_TOP_K * kValues) + I4S_MAX_TOP_K;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct LF16 {
  static constexpr int kSize = 2;
  static __device__ float get(const w4_t &v, int e) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)(v[e / 2] >> (16 * (e % 2))));
  }
  static __device__ float one(const void *p, int64_t i) { return (float)static_cast<const _Float16 *>(p)[i]; }
};
struct LBF16 {
  static constexpr int kSize = 2;
  static __device__ float get(const w4_t &v, int e) {
    return __builtin_bit_cast(float, e % 2 ? v[e / 2] & 0xFFFF0000u : v[e / 2] << 16);
  }
  static __device__ float one(const void *p, int64_t i) {
    return __builtin_bit_cast(float, (uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
  }
};
struct LF32 {
  static constexpr int kSize = 4;
  static __device__ float get(const w4_t &v, int e) {
    const uint32_t bits = v[e];
    return __builtin_bit_cast(float, bits);
  }
  static __device__ float one(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }
};

// A whole number that orders like the value (-0 as 0).
__device__ inline uint32_t order_of(float x) {
  const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ inline float value_of(uint32_t o) {
  return __builtin_bit_cast(float, o & 0x80000000u ? o ^ 0x80000000u : ~o);
}

__device__ inline float wave_max(float v) {
  for (int d = 32; d; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
__device__ inline float wave_add(float v) {
  for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The k-th largest of the 64 lanes' values.
__device__ inline uint32_t kth_of_wave(uint32_t o, int k) {
  uint32_t t = 0;
#pragma unroll 1
  for (int b = 31; b >= 0; --b) {
    const uint32_t next = t | 1u << b;
    if (__popcll(__ballot(o >= next)) >= k) t = next;
  }
  return t;
}

struct Stats {
  float m, l, t;  // maximum, sum of exp(x - m), sum of (x - m) exp(x - m)
};

// Takes s to the maximum `to` (at least s.m).
__device__ inline void raise(Stats &s, float to) {
  if (s.m == -INFINITY) {
    s.l = s.t = 0.0f;
  } else if (to > s.m) {
    const float d = s.m - to, f = __builtin_amdgcn_exp2f(d * kLog2e);
    s.t = f == 0.0f ? 0.0f : f * fmaf(d, s.l, s.t);
    s.l *= f;
  }
  s.m = to;
}

__device__ void write_row(const LogprobsArgs &a, int row, const Stats &s, float x, bool valid) {
  float lp, h;
  if (s.m == INFINITY) {  // a NaN or +inf among the values
    lp = h = NAN;
  } else if (s.m == -INFINITY) {
    lp = -INFINITY;
    h = 0.0f;
  } else {
    const float ln = __builtin_amdgcn_logf(s.l) * kLn2;
    lp = (x - s.m) - ln;
    h = fmaxf(ln - s.t / s.l, 0.0f);
  }
  a.logprobs[row] = valid ? lp : NAN;
  a.entropy[row] = h;
}

__device__ inline void write_top(const LogprobsArgs &a, int row, int i, uint64_t key, const Stats &s) {
  const int64_t at = (int64_t)row * a.top_k + i;
  a.top_ids[at] = (int32_t)~(uint32_t)key;
  const float x = value_of((uint32_t)(key >> 32));
  a.top_logprobs[at] = s.m == INFINITY ? NAN
                       : s.m == -INFINITY ? -INFINITY
                                          : (x - s.m) - __builtin_amdgcn_logf(s.l) * kLn2;
}

template <typename T>
__global__ __launch_bounds__(kBlock) void logprobs_kernel(LogprobsArgs a, int splits, int slices_per_split) {
  constexpr int kVec = 16 / T::kSize, kVecs = kValues / kVec;
  __shared__ uint64_t cand[kMaxCandidates];
  __shared__ uint64_t best[I4S_MAX_TOP_K];
  __shared__ float wave_m[kBlockWaves], wave_l[kBlockWaves], wave_t[kBlockWaves];
  __shared__ uint32_t wave_kth[kBlockWaves];
  __shared__ int count;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int row = blockIdx.x, split = blockIdx.y, k = a.top_k;
  const char *base = static_cast<const char *>(a.logits) + (int64_t)row * a.stride * T::kSize;
  // 16-byte vectors from the aligned address at or below the row's start:
  // value e of vector q is column q * kVec + e - pad
  const int pad = (int)((reinterpret_cast<uintptr_t>(base) & 15) / T::kSize);
  const int vectors = (a.vocab + pad + kVec - 1) / kVec;
  const int slices = (vectors + kBlock * kVecs - 1) / (kBlock * kVecs);
  const int s0 = split * slices_per_split, s1 = split == splits - 1 ? slices : min(slices, s0 + slices_per_split);

  const auto load = [&](w4_t(&v)[kVecs], float (&x)[kValues], int slice) {
    (void)v;
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const int q = (slice * kVecs + j) * kBlock + tid;
      const int col = q * kVec - pad;
      if (col >= 0 && col + kVec <= a.vocab) {
        v[j] = *reinterpret_cast<const w4_t *>(base + (int64_t)col * T::kSize);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[j * kVec + e] = T::get(v[j], e);
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
          x[j * kVec + e] = col + e >= 0 && col + e < a.vocab ? T::one(base, col + e) : -INFINITY;
      }
    }
  };

  Stats s = {-INFINITY, 0.0f, 0.0f};
  int held = 0;  // alternatives in `best`
  for (int slice = s0; slice < s1; ++slice) {
    w4_t raw[kVecs];
    float x[kValues];
    load(raw, x, slice);
    float top = -INFINITY;
#pragma unroll
    for (int e = 0; e < kValues; ++e) top = fmaxf(top, fminf(x[e], INFINITY));  // a NaN counts as +inf
    const float wm = wave_max(top);
    if (lane == 0) wave_m[wave] = wm;
    if (k) {
      const uint32_t kth = kth_of_wave(order_of(top), k);
      if (lane == 0) wave_kth[wave] = kth;
      if (tid == 0) count = 0;
    }
    __syncthreads();
    float m = s.m;
#pragma unroll
    for (int w = 0; w < kBlockWaves; ++w) m = fmaxf(m, wave_m[w]);
    raise(s, m);
    if (m != -INFINITY) {
#pragma unroll
      for (int e = 0; e < kValues; ++e) {
        const float d = fmaxf(x[e] - m, -150.0f);  // exp2 of less is 0; keeps 0 * -inf away
        const float p = __builtin_amdgcn_exp2f(d * kLog2e);
        s.l += p;
        s.t = fmaf(d, p, s.t);
      }
    }
    if (k) {
      uint32_t kth = 0;
#pragma unroll
      for (int w = 0; w < kBlockWaves; ++w) kth = max(kth, wave_kth[w]);
      // only what beats the k-th best of the slices before: its index is lower
      const uint32_t floor_key = held == k ? (uint32_t)(best[k - 1] >> 32) + 1 : 0;
      const bool ties = kth >= floor_key;
      kth = max(kth, floor_key);
      const bool any = order_of(top) >= kth;
      if (__any(any)) {
        int taken = 0;  // values equal to kth that this wave has taken
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const int col = ((slice * kVecs + j) * kBlock + tid) * kVec - pad;
          bool equal[kVec];
          int before = 0, mine = 0;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const uint32_t o = order_of(fminf(x[j * kVec + e], INFINITY));
            const bool inside = col + e >= 0 && col + e < a.vocab;
            equal[e] = ties && o == kth && inside;
            if (inside && (o > kth || (!ties && o == kth))) {
              const int at = atomicAdd(&count, 1);
              cand[at] = (uint64_t)o << 32 | ~(uint32_t)(col + e);
            }
            const uint64_t mask = __ballot(equal[e]);
            before += __popcll(mask & ((1ull << lane) - 1));
            mine += equal[e];
          }
          (void)mine;
          int nth = taken + before, all = 0;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            all += __popcll(__ballot(equal[e]));
            if (equal[e]) {
              if (nth < k) {
                const int at = atomicAdd(&count, 1);
                cand[at] = (uint64_t)kth << 32 | ~(uint32_t)(col + e);
              }
              ++nth;
            }
          }
          taken += all;
        }
      }
      __syncthreads();
      const int found = count;
      if (found) {
        if (tid < held) cand[found + tid] = best[tid];
        __syncthreads();
        const int n = found + held;
        for (int i = tid; i < n; i += kBlock) {
          const uint64_t key = cand[i];
          int above = 0;
          for (int j = 0; j < n; ++j) above += cand[j] > key;
          if (above < k) best[above] = key;
        }
        held = min(n, k);
      }
    }
    __syncthreads();
  }

  s.l = wave_add(s.l);
  s.t = wave_add(s.t);
  if (lane == 0) {
    wave_l[wave] = s.l;
    wave_t[wave] = s.t;
  }
  __syncthreads();
  s.l = s.t = 0.0f;
#pragma unroll
  for (int w = 0; w < kBlockWaves; ++w) {
    s.l += wave_l[w];
    s.t += wave_t[w];
  }
  if (splits == 1) {
    if (tid == 0) {
      const int64_t token = a.tokens[row];
      const bool valid = token >= 0 && token < a.vocab;
      write_row(a, row, s, valid ? T::one(base, token) : 0.0f, valid);
    }
    if (tid < k) write_top(a, row, tid, best[tid], s);
  } else {
    const int64_t part = (int64_t)row * splits + split;
    if (tid == 0) {
      float *p = a.part_stats + 4 * part;
      p[0] = s.m, p[1] = s.l, p[2] = s.t;
    }
    if (tid < k) a.part_keys[part * k + tid] = tid < held ? best[tid] : 0;
  }
}

// Joins the pieces of a row: one block per row.
template <typename T>
__global__ __launch_bounds__(1024) void logprobs_join_kernel(LogprobsArgs a, int splits) {
  extern __shared__ uint64_t keys[];
  const int row = blockIdx.x, tid = threadIdx.x, k = a.top_k, n = splits * k;
  for (int i = tid; i < n; i += blockDim.x) keys[i] = a.part_keys[(int64_t)row * n + i];
  Stats s = {-INFINITY, 0.0f, 0.0f};
  const float *p = a.part_stats + 4 * (int64_t)row * splits;
  float m = -INFINITY;
  for (int i = 0; i < splits; ++i) m = fmaxf(m, p[4 * i]);
  for (int i = 0; i < splits; ++i) {
    Stats o = {p[4 * i], p[4 * i + 1], p[4 * i + 2]};
    raise(o, m);
    s.l += o.l;
    s.t += o.t;
  }
  s.m = m;
  if (tid == 0) {
    const int64_t token = a.tokens[row];
    const bool valid = token >= 0 && token < a.vocab;
    const char *base = static_cast<const char *>(a.logits) + (int64_t)row * a.stride * T::kSize;
    write_row(a, row, s, valid ? T::one(base, token) : 0.0f, valid);
  }
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const uint64_t key = keys[i];
    if (!key) continue;  // a piece with fewer than k values
    int above = 0;
    for (int j = 0; j < n; ++j) above += keys[j] > key;
    if (above < k) write_top(a, row, above, key, s);
  }
}

template <typename T>
hipError_t go(const LogprobsArgs &a, const LogprobsPlan &p, hipStream_t stream) {
  hipLaunchKernelGGL((logprobs_kernel<T>), dim3(a.rows, p.splits), dim3(kBlock), 0, stream, a, p.splits, p.chunk / kSlice);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  const int keys = p.splits * a.top_k;
  const int threads = clamp_to((keys + 63) / 64 * 64, 64, 1024);
  hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3(a.rows), dim3(threads), sizeof(uint64_t) * (keys ? keys : 1), stream, a,
                     p.splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_token_logprobs(const LogprobsArgs &a, const LogprobsPlan &p, int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16 ? go<LF16>(a, p, stream) : dtype == I4S_BF16 ? go<LBF16>(a, p, stream) : go<LF32>(a, p, stream);
}

}  // namespace i4s
