// Log probabilities of given tokens, entropy and top alternatives of rows of
// logits (include/i4s_serve.h), for gfx950.
//
// A block streams over its piece of a row: 32 values a thread at a time (a
// segment), from which it takes the segment's maximum and adds exp(x - r) and
// (x - r) exp(x - r) to two sums.  The reference r is the thread's own largest
// value so far, so nothing waits for anything until the piece ends.  Where
// there are few rows they are split into pieces, which a second launch joins.
//
// Top k.  The threads fall into 64 groups (equal lanes of all waves); the k-th
// largest of the 64 group maxima is a lower bound T of the k-th largest value,
// found bit by bit with ballots.  Only threads and segments whose maximum
// reaches T are looked at again (about 64 ln(64 / (64 - k)) of them), and the
// values found get their places by counting the larger ones (value, then
// lower index).  Where more values reach T than there is room for (equal ones, as in
// a masked vocabulary) or a NaN hides maxima, the block finds the exact k-th
// value instead and takes the equal ones in order of their index.
//
// Bound by: memory (2 or 4 bytes a value) when there are many rows: 4093 x
// 50257 bf16, top 8: 412 MB in 82 us, 5.0 TB/s.  (The vector units are next:
// twelve instructions a value all told, one an exponential at a quarter of their
// rate.  Nothing may live in scratch: the argument struct, passed on to
// select_exact by reference, was written there by every thread of every block,
// 90 MB a call: 108 us.)  Few rows wait: 1 x 32000 fp16, one block of four
// segments, 5.9 us without and 8.3 to 9.9 with the top 1 to 20 (the bound, a second
// look, counting); 1 x 2048 3.3 and 5.6; 16 x 151643 fp32 10 us in 10 pieces of two
// segments and 5 us for their join.
//
// Errors, in nats: 2^-22 (1 + sum p |x - m|) of the exponentials (v_exp and the
// product with log2 e), as much of the logarithm, and fp32's own of the sums.

#include <float.h>

#include "i4s_serve_internal.h"

namespace i4s {
namespace {

typedef uint32_t w4_t __attribute__((ext_vector_type(4)));

constexpr int NT = 256;              // threads of a block
constexpr int kValues = 32;          // values of a thread in a segment
constexpr int kCandidates = 512;     // values that reach T
constexpr int kHits = 256;           // (thread, segment) pairs that reach T
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

// Sums of a thread, block or piece: with y = (x - e) log2(e'), e' Euler's
// number, l = sum 2^y and t = sum y 2^y.  m is the largest x; e is m, or the
// lowest finite value while there is nothing above -inf.
struct Stats {
  float m, e, l, t;
};
constexpr Stats kNothing = {-INFINITY, -FLT_MAX, 0.0f, 0.0f};

// Takes s to the reference `to`, at least s.e.
__device__ inline void raise(Stats &s, float to) {
  const float d = (s.e - to) * kLog2e, f = __builtin_amdgcn_exp2f(d);
  s.t = f == 0.0f ? 0.0f : f * fmaf(d, s.l, s.t);
  s.l *= f;
  s.e = to;
}

__device__ inline bool bad(const Stats &s) { return s.m == INFINITY || s.l != s.l; }  // +inf or NaN among the values

__device__ inline float logprob_of(const Stats &s, float x) {
  if (bad(s)) return NAN;
  if (s.m == -INFINITY) return -INFINITY;
  return (x - s.e) - __builtin_amdgcn_logf(s.l) * kLn2;
}

__device__ inline void write_row(const LogprobsArgs &a, int row, const Stats &s, bool valid, float x) {
  a.logprobs[row] = valid ? logprob_of(s, x) : NAN;
  float h = 0.0f;
  if (bad(s))
    h = NAN;
  else if (s.m != -INFINITY)
    h = fmaxf((__builtin_amdgcn_logf(s.l) - s.t / s.l) * kLn2, 0.0f);
  a.entropy[row] = h;
}

__device__ inline void write_top(const LogprobsArgs &a, int row, int i, uint64_t key, const Stats &s) {
  const int64_t at = (int64_t)row * a.top_k + i;
  a.top_ids[at] = (int32_t)~(uint32_t)key;
  a.top_logprobs[at] = logprob_of(s, value_of((uint32_t)(key >> 32)));
}

// A row as 16-byte vectors, from the start of the 128-byte line that holds its
// first value (a wave's loads then cover whole lines): value e of vector q is
// column q * kVec + e - pad.
template <typename T>
struct Row {
  static constexpr int kVec = 16 / T::kSize;
  const char *base;
  int pad, vocab;
  __device__ Row(const char *first, int n)
      : base(first), pad((int)((reinterpret_cast<uintptr_t>(first) & 127) / T::kSize)), vocab(n) {}
  __device__ int vectors() const { return (vocab + pad + kVec - 1) / kVec; }
  __device__ int column(int q) const { return q * kVec - pad; }
  __device__ int first_whole() const { return (pad + kVec - 1) / kVec; }
  __device__ int last_whole() const { return (vocab + pad) / kVec - 1; }
  __device__ bool whole(int q) const { return column(q) >= 0 && column(q) + kVec <= vocab; }
  __device__ w4_t vector(int q) const {
    return __builtin_nontemporal_load(reinterpret_cast<const w4_t *>(base + (int64_t)column(q) * T::kSize));
  }
  // the vector's values; -inf outside the row
  __device__ void load(int q, float (&x)[kVec]) const {
    if (whole(q)) {
      const w4_t v = vector(q);
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = T::get(v, e);
    } else {
#pragma unroll
      for (int e = 0; e < kVec; ++e) {
        const int c = column(q) + e;
        x[e] = c >= 0 && c < vocab ? T::one(base, c) : -INFINITY;
      }
    }
  }
  __device__ bool inside(int q, int e) const { return column(q) + e >= 0 && column(q) + e < vocab; }
};

__device__ inline uint32_t rank_order(float x) { return order_of(fminf(x, INFINITY)); }  // a NaN as +inf

// What the threads of a block share while they select.
struct Select {
  uint64_t cand[kCandidates], best[I4S_MAX_TOP_K];
  uint32_t hits[kHits];
  int n_cand, n_hits, wave_n[NT / 64];
};

__device__ inline int block_count(Select &s, int mine) {  // sum over the block, for every thread
  for (int d = 32; d; d >>= 1) mine += __shfl_xor(mine, d);
  __syncthreads();
  if (threadIdx.x % 64 == 0) s.wave_n[threadIdx.x / 64] = mine;
  __syncthreads();
  int n = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) n += s.wave_n[w];
  return n;
}

// The k best of vectors [q0, q1) into s.best by the exact k-th value; returns
// how many there are.  `bound`: a value that at least k values reach, or 0.
template <typename T>
__device__ __noinline__ int select_exact(Select &s, const char *first, int vocab, int q0, int q1, int k, uint32_t bound) {
  const Row<T> r(first, vocab);
  constexpr int kVec = Row<T>::kVec;
  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const auto count_from = [&](uint32_t least) {  // values of at least that order
    int n = 0;
    for (int q = q0 + tid; q < q1; q += NT) {
      float x[kVec];
      r.load(q, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) n += r.inside(q, e) && rank_order(x[e]) >= least;
    }
    return block_count(s, n);
  };
  k = min(k, count_from(0));
  uint32_t kth = bound;
  if (!bound || count_from(bound + 1) >= k) {
    kth = 0;
    for (int b = 31; b >= 0; --b)
      if (count_from(kth | 1u << b) >= k) kth |= 1u << b;
  }
  if (tid == 0) s.n_cand = 0;
  __syncthreads();
  for (int q = q0 + tid; q < q1; q += NT) {  // fewer than k are larger
    float x[kVec];
    r.load(q, x);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      const uint32_t o = rank_order(x[e]);
      if (r.inside(q, e) && o > kth) s.cand[atomicAdd(&s.n_cand, 1)] = (uint64_t)o << 32 | ~(uint32_t)(r.column(q) + e);
    }
  }
  __syncthreads();
  int have = s.n_cand;
  for (int q = q0; q < q1 && have < k; q += NT) {  // equal ones, in order
    const int mine = q + tid;
    uint32_t equal = 0;
    if (mine < q1) {
      float x[kVec];
      r.load(mine, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) equal |= (uint32_t)(r.inside(mine, e) && rank_order(x[e]) == kth) << e;
    }
    const int n = __popc(equal);
    int before = n;  // inclusive over the wave
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(before, d);
      if (lane >= d) before += o;
    }
    __syncthreads();
    if (lane == 63) s.wave_n[wave] = before;
    __syncthreads();
    int at = have + before - n, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
      if (w < wave) at += s.wave_n[w];
      all += s.wave_n[w];
    }
    for (int e = 0; e < kVec; ++e)
      if (equal >> e & 1 && at < k) s.cand[at++] = (uint64_t)kth << 32 | ~(uint32_t)(r.column(mine) + e);
    have = min(have + all, k);
  }
  __syncthreads();
  return have;
}

// Orders s.cand[0..n) into s.best; every thread of the block.
__device__ inline void place(Select &s, int n, int k) {
  for (int i = threadIdx.x; i < n; i += NT) {
    const uint64_t key = s.cand[i];
    int above = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) above += s.cand[j] > key;
    if (above < k) s.best[above] = key;
  }
  __syncthreads();
}

template <typename T>
__global__ __launch_bounds__(NT) void logprobs_kernel(LogprobsArgs a, int splits, int segments) {
  typedef Row<T> R;
  constexpr int kVec = R::kVec, kVecs = kValues / kVec, kWaves = NT / 64;
  extern __shared__ float seg_max[];  // [segments][NT], only with top_k
  __shared__ Select sel;
  __shared__ float thread_m[NT], wave_l[kWaves], wave_t[kWaves];
  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int row = blockIdx.x, split = blockIdx.y, k = a.top_k;
  const R r(static_cast<const char *>(a.logits) + (int64_t)row * a.stride * T::kSize, a.vocab);
  const int q0 = split * segments * (NT * kVecs);
  const int q1 = min(r.vectors(), q0 + segments * (NT * kVecs));

  const int64_t token = tid == 0 ? a.tokens[row] : -1;
  const bool valid = token >= 0 && token < a.vocab;
  const float token_x = valid ? T::one(r.base, token) : 0.0f;

  // The next segment's vectors load while this one is added up.  Vectors that
  // are not whole are replaced afterwards; the loads themselves have no branch.
  const int first_whole = r.first_whole(), last_whole = r.last_whole();
  const bool any_whole = first_whole <= last_whole;
  w4_t v[kVecs] = {};
  const auto fetch = [&](int q) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) v[j] = r.vector(clamp_to(q + j * NT + tid, first_whole, last_whole));
  };
  Stats s = kNothing;
  const auto add = [&](const auto &x) {  // the largest of x
    constexpr int n = sizeof(x) / sizeof(float);
    float top = x[0];
#pragma unroll
    for (int e = 1; e < n; ++e) top = fmaxf(top, x[e]);  // passes over NaN
    if (top > s.e) raise(s, top);
    float l[2] = {0.0f, 0.0f}, t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < n; ++e) {
      const float y = (x[e] - s.e) * kLog2e, p = __builtin_amdgcn_exp2f(y);
      l[e % 2] += p;
      t[e % 2] = fmaf(fmaxf(y, -200.0f), p, t[e % 2]);  // exp2 of less is 0: keeps -inf * 0 away
    }
    s.l += l[0] + l[1];
    s.t += t[0] + t[1];
    return top;
  };
  if (any_whole) fetch(q0);
  for (int seg = 0, q = q0; q < q1; ++seg, q += NT * kVecs) {
    const bool edge = q < first_whole || q + NT * kVecs - 1 > last_whole, more = any_whole && q + NT * kVecs < q1;
    float top = -INFINITY;
    if (!edge) {
      float x[kValues];
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[j * kVec + e] = T::get(v[j], e);
      if (more) fetch(q + NT * kVecs);
      top = add(x);
    } else {  // vector by vector: a wave passes over those behind the row's end
#pragma unroll
      for (int j = 0; j < kVecs; ++j)
        if (q + j * NT + 64 * wave < q1) {
          float x[kVec];
#pragma unroll
          for (int e = 0; e < kVec; ++e) x[e] = T::get(v[j], e);
          if (!r.whole(q + j * NT + tid)) r.load(q + j * NT + tid, x);
          top = fmaxf(top, add(x));
        }
      if (more) fetch(q + NT * kVecs);
    }
    if (k) seg_max[seg * NT + tid] = top;
    s.m = fmaxf(s.m, top);
  }

  thread_m[tid] = s.m;
  if (tid == 0) sel.n_cand = sel.n_hits = 0;
  __syncthreads();
  float group = thread_m[lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) group = fmaxf(group, thread_m[64 * w + lane]);
  const float m = wave_max(group);
  raise(s, fmaxf(m, -FLT_MAX));
  s.l = wave_add(s.l);
  s.t = wave_add(s.t);
  if (lane == 0) {
    wave_l[wave] = s.l;
    wave_t[wave] = s.t;
  }
  uint32_t kth = 0;
  if (k) {
    kth = kth_of_wave(order_of(group), k);
    if (order_of(s.m) >= kth)
      for (int seg = 0, q = q0; q < q1; ++seg, q += NT * kVecs)
        if (order_of(seg_max[seg * NT + tid]) >= kth) {
          const int at = atomicAdd(&sel.n_hits, 1);
          if (at < kHits) sel.hits[at] = seg * NT + tid;
        }
  }
  __syncthreads();
  s.m = m;
  s.l = s.t = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    s.l += wave_l[w];
    s.t += wave_t[w];
  }
  int held = 0;
  if (k) {
    const int hits = sel.n_hits;
    bool exact = hits > kHits || s.l != s.l;
    if (!exact) {
      for (int i = tid; i < hits * kVecs; i += NT) {
        const int seg = sel.hits[i / kVecs] / NT, who = sel.hits[i / kVecs] % NT;
        const int q = q0 + (seg * kVecs + i % kVecs) * NT + who;
        float x[kVec];
        r.load(q, x);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const uint32_t o = order_of(x[e]);
          if (o >= kth && r.inside(q, e)) {
            const int at = atomicAdd(&sel.n_cand, 1);
            if (at < kCandidates) sel.cand[at] = (uint64_t)o << 32 | ~(uint32_t)(r.column(q) + e);
          }
        }
      }
      __syncthreads();
      held = sel.n_cand;
      exact = held > kCandidates;
    }
    if (exact) {
      __syncthreads();
      held = select_exact<T>(sel, r.base, r.vocab, q0, q1, k, s.l != s.l ? 0 : kth);
    }
    place(sel, held, k);
    held = min(held, k);
  }
  if (splits == 1) {
    if (tid == 0) write_row(a, row, s, valid, token_x);
    if (tid < k) write_top(a, row, tid, sel.best[tid], s);
  } else {
    const int64_t part = (int64_t)row * splits + split;
    if (tid == 0) {
      float *p = a.part_stats + 4 * part;
      p[0] = s.m, p[1] = s.e, p[2] = s.l, p[3] = s.t;
    }
    if (tid < k) a.part_keys[part * k + tid] = tid < held ? sel.best[tid] : 0;
  }
}

// Joins the pieces of a row: one block per row.  The k best of splits * k keys
// (at most 64 * 32) the same way: a bound from the lane maxima, then counting.
template <typename T>
__global__ __launch_bounds__(NT) void logprobs_join_kernel(LogprobsArgs a, int splits) {
  constexpr int kMine = 8;  // 64 * 32 / 256
  __shared__ Select sel;
  __shared__ uint32_t thread_top[256];
  const int row = blockIdx.x, tid = threadIdx.x, k = a.top_k, n = splits * k;
  Stats s = kNothing;
  const float *p = a.part_stats + 4 * (int64_t)row * splits;
  // each lane takes a piece, then the lanes join
  const int lane = tid % 64;
  if (lane < splits) s = {p[4 * lane], p[4 * lane + 1], p[4 * lane + 2], p[4 * lane + 3]};
  const float m = wave_max(s.m), e = wave_max(s.e);
  raise(s, e);
  s.l = wave_add(s.l);
  s.t = wave_add(s.t);
  s.m = m;
  if (tid == 0) {
    const int64_t token = a.tokens[row];
    const bool valid = token >= 0 && token < a.vocab;
    const char *base = static_cast<const char *>(a.logits) + (int64_t)row * a.stride * T::kSize;
    const float x = valid ? T::one(base, token) : 0.0f;
    write_row(a, row, s, valid, x);
    sel.n_cand = 0;
  }
  if (!k) return;
  uint64_t key[kMine];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kMine; ++j) {
    key[j] = tid + 256 * j < n ? a.part_keys[(int64_t)row * n + tid + 256 * j] : 0;
    top = max(top, (uint32_t)(key[j] >> 32));
  }
  thread_top[tid] = top;
  __syncthreads();
  const uint32_t kth = kth_of_wave(max(max(thread_top[lane], thread_top[64 + lane]),
                                       max(thread_top[128 + lane], thread_top[192 + lane])), k);
#pragma unroll
  for (int j = 0; j < kMine; ++j)
    if (key[j] && (uint32_t)(key[j] >> 32) >= kth) {
      const int at = atomicAdd(&sel.n_cand, 1);
      if (at < kCandidates) sel.cand[at] = key[j];
    }
  __syncthreads();
  int found = sel.n_cand;
  if (found <= kCandidates) {
    place(sel, found, k);
  } else {  // many equal ones: every key against every other
#pragma unroll
    for (int j = 0; j < kMine; ++j)
      if (key[j]) {
        int above = 0;
        for (int i = 0; i < n; ++i) above += a.part_keys[(int64_t)row * n + i] > key[j];
        if (above < k) sel.best[above] = key[j];
      }
    __syncthreads();
  }
  if (tid < k) write_top(a, row, tid, sel.best[tid], s);
}

template <typename T>
hipError_t go(const LogprobsArgs &a, const LogprobsPlan &p, hipStream_t stream) {
  const size_t lds = a.top_k ? sizeof(float) * p.segments * NT : 0;
  hipLaunchKernelGGL((logprobs_kernel<T>), dim3(a.rows, p.splits), dim3(NT), lds, stream, a, p.splits, p.segments);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.splits == 1) return e;
  hipLaunchKernelGGL((logprobs_join_kernel<T>), dim3(a.rows), dim3(256), 0, stream, a, p.splits);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_token_logprobs(const LogprobsArgs &a, const LogprobsPlan &p, int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16    ? go<LF16>(a, p, stream)
         : dtype == I4S_BF16 ? go<LBF16>(a, p, stream)
                             : go<LF32>(a, p, stream);
}

}  // namespace i4s
