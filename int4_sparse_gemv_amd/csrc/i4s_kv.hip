// The paged 4-bit KV cache: block tables and slot maps from request lengths,
// and the kernels that write tokens into the cache and read them back.  The
// format is that of include/i4s_serve.h.

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>

#include "i4s_serve_internal.h"

namespace i4s {
namespace {

typedef uint32_t u4_t __attribute__((ext_vector_type(4)));
typedef float f4_t __attribute__((ext_vector_type(4)));
typedef float f8_t __attribute__((ext_vector_type(8)));

constexpr float kScaleMax = 9352.0f;  // largest fp16 whose 7-fold is finite in fp16

// ---------------------------------------------------------------------------
// block tables and slot maps
//
// Every block sums the lengths of all requests by itself (n is at most a few
// thousand 4-byte words, which stay in L2): exclusive sums of the new tokens
// and of the new pages go to LDS, and each thread then finds the owner of a
// token, or of a new page, by bisection there.  So one launch does it all,
// with no block waiting for another: a token's page is either in the part of
// the table that the call does not write, or follows from the page sums and
// the free list without reading the table.
//
// Bound by: latency.  16 requests of one token each 3.1 us (one block, a few
// dependent loads), 512 requests of about 76000 tokens together 7.0 us.

struct Sums {
  long long tokens, pages;
};

__global__ __launch_bounds__(1024) void kv_extend_kernel(ExtendArgs a) {
  extern __shared__ int32_t lds[];
  __shared__ Sums wave_sums[16];
  __shared__ int32_t any_flags;
  int32_t *token_start = lds;              // [n + 1]
  int32_t *page_start = lds + a.n + 1;     // [n + 1]
  const int threads = blockDim.x, tid = threadIdx.x, lane = tid % 64, wave = tid / 64, waves = threads / 64;
  const int page = 1 << a.shift;
  if (tid == 0) any_flags = 0;

  const int per = (a.n + threads - 1) / threads;
  const int first = min(tid * per, a.n), last = min(first + per, a.n);
  Sums mine = {0, 0};
  int32_t flags = 0;
  for (int i = first; i < last; ++i) {
    const long long have = a.lens[i], more = a.new_lens[i];
    if (have < 0 || more < 0 || have + more > 0x7FFFFFFFll) {
      flags |= I4S_KV_BAD_LENGTH;
      continue;
    }
    const long long old_pages = (have + page - 1) >> a.shift, pages = (have + more + page - 1) >> a.shift;
    if (pages > a.width) flags |= I4S_KV_ROW_FULL;
    mine.tokens += more;
    mine.pages += pages - old_pages;
  }
  Sums sum = mine;  // inclusive over the wave
  for (int d = 1; d < 64; d <<= 1) {
    const long long t = __shfl_up(sum.tokens, d), p = __shfl_up(sum.pages, d);
    if (lane >= d) {
      sum.tokens += t;
      sum.pages += p;
    }
  }
  if (lane == 63) wave_sums[wave] = sum;
  __syncthreads();
  if (flags) atomicOr(&any_flags, flags);
  Sums before = {sum.tokens - mine.tokens, sum.pages - mine.pages}, total = {0, 0};
  for (int w = 0; w < waves; ++w) {
    if (w < wave) {
      before.tokens += wave_sums[w].tokens;
      before.pages += wave_sums[w].pages;
    }
    total.tokens += wave_sums[w].tokens;
    total.pages += wave_sums[w].pages;
  }
  const int32_t count = *a.free_count;
  __syncthreads();
  int32_t all = any_flags;
  if (count < 0 || count > a.free_entries) all |= I4S_KV_BAD_COUNT;
  if (total.pages > (count < 0 ? 0 : count)) all |= I4S_KV_NO_PAGES;
  if (total.tokens > a.capacity) all |= I4S_KV_NO_SLOTS;
  const bool fine = all == 0;

  if (blockIdx.x == 0) {
    if (tid == 0) {
      *a.flags = all;
      *a.free_count_out = fine ? count - (int32_t)total.pages : count;
      a.q_start[a.n] = fine ? (int32_t)total.tokens : 0;
    }
    long long t = before.tokens;
    for (int i = first; i < last; ++i) {
      const int32_t have = a.lens[i], more = a.new_lens[i];
      a.lens_out[i] = fine ? have + more : have;
      a.q_start[i] = fine ? (int32_t)t : 0;
      t += more;
    }
  }
  if (fine) {
    Sums at = before;
    for (int i = first; i < last; ++i) {
      const long long have = a.lens[i], more = a.new_lens[i];
      token_start[i] = (int32_t)at.tokens;
      page_start[i] = (int32_t)at.pages;
      at.tokens += more;
      at.pages += ((have + more + page - 1) >> a.shift) - ((have + page - 1) >> a.shift);
    }
  }
  __syncthreads();

  // the last request that starts at or before place v: the owner of v
  const auto owner = [&](const int32_t *start, int32_t v) {
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
  };
  const int32_t tokens = fine ? (int32_t)total.tokens : 0, pages = fine ? (int32_t)total.pages : 0;
  const int64_t step = (int64_t)gridDim.x * threads;
  for (int64_t v = (int64_t)blockIdx.x * threads + tid; v < a.capacity; v += step) {
    if (v >= tokens) {
      a.slots[v] = -1;
      a.positions[v] = 0;
      continue;
    }
    const int i = owner(token_start, (int32_t)v);
    const int32_t have = a.lens[i];
    const int32_t pos = have + ((int32_t)v - token_start[i]);
    const int32_t old_pages = (int32_t)(((int64_t)have + page - 1) >> a.shift), p = pos >> a.shift;
    const int32_t number = p < old_pages ? a.table[(int64_t)i * a.width + p]
                                         : a.free_pages[count - 1 - (page_start[i] + (p - old_pages))];
    // a number that no cache can have must not come round to another page's slots
    const bool real = number >= 0 && number <= 0x7FFFFFFF >> a.shift;
    a.slots[v] = real ? (number << a.shift) + (pos & (page - 1)) : -1;
    a.positions[v] = pos;
    if (v < pages) {  // every new page holds a new token, so pages <= tokens
      const int j = owner(page_start, (int32_t)v);
      const int32_t entry = (int32_t)(((int64_t)a.lens[j] + page - 1) >> a.shift) + ((int32_t)v - page_start[j]);
      a.table[(int64_t)j * a.width + entry] = a.free_pages[count - 1 - (int32_t)v];
    }
  }
}

// ---------------------------------------------------------------------------
// element types

struct Half {
  static __device__ float to_float(uint32_t bits) { return (float)__builtin_bit_cast(_Float16, (uint16_t)bits); }
  static __device__ uint32_t from_float(float f) { return __builtin_bit_cast(uint16_t, (_Float16)f); }
};
struct Bfloat {
  static __device__ float to_float(uint32_t bits) { return __builtin_bit_cast(float, bits << 16); }
  static __device__ uint32_t from_float(float f) { return __builtin_bit_cast(uint16_t, (__bf16)f); }
};

template <typename T>
__device__ inline f8_t load8(const uint16_t *p) {
  const u4_t w = __builtin_nontemporal_load(reinterpret_cast<const u4_t *>(p));
  f8_t x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = T::to_float(w[i] & 0xFFFFu);
    x[2 * i + 1] = T::to_float(w[i] >> 16);
  }
  return x;
}

// ---------------------------------------------------------------------------
// writing tokens
//
// A block takes 256 / (D/8) neighbouring tokens of one head, D/8 neighbouring
// lanes a token: a lane quantizes 8 channels (one 16-byte load), the group
// maximum goes across the G/8 lanes of a group with DPP.  Neighbouring tokens
// mostly lie in one page, where their K rows, the V words of four tokens and
// their scales lie next to each other, so stores fill whole lines.  For K the
// lane's 8 nibbles are one word of the row.  For V the four lanes that hold
// channels 16e + 8b .. +7 (e = 0..3) of one 64-channel block exchange their
// words and make two of the eight 16-bit halves each, and pairs of lanes join
// these into whole words.
//
// Bound by: memory, 2 bytes read and a little over half a byte written a
// value.  8191 tokens x 40 heads of 128, bf16, G = 64, sliced out of a fused
// product: 213 MB in 45 us, 4.7 TB/s (57 us with
// ordinary loads: k and v are read once); 16 tokens x 32 heads 2.8 us.

template <int CTRL>
__device__ inline uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kXor7 = 0x141, kXor8 = 0x128, kXor15 = 0x140;  // of the lane number

// The 8 nibbles (in channel order) and the scale of the lane's channels.
// Quotients are a product with an approximate reciprocal and one correction
// with the exact remainder: a quotient that has few bits (a whole number and a
// half, half a step of a subnormal scale) comes out exactly, and the others lie
// further from such a border (2^-12 of a step) than the error, so rounding
// gives what it gives for the correctly rounded quotient.
__device__ inline float quotient(float x, float divisor, float reciprocal) {
  const float q = x * reciprocal;
  return fmaf(fmaf(-q, divisor, x), reciprocal, q);
}

// The low bytes of a, b, c, d.
__device__ inline uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_amdgcn_perm(__builtin_amdgcn_perm(d, c, 0x0C0C0400u), __builtin_amdgcn_perm(b, a, 0x0C0C0400u), 0x05040100u);
}

// n[e] of the lane's channels e = 0..7: the nibble in the low byte.
template <int G>
__device__ inline void quantize8(f8_t x, uint32_t (&n)[8], uint32_t &scale_bits) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = __builtin_elementwise_maximum(m, fabsf(x[e]));  // passes a NaN on
  if (__any(m != m)) {
    m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = x[e] == x[e] ? x[e] : 0.0f;
      m = fmaxf(m, fabsf(x[e]));
    }
  }
  const auto with = [&](uint32_t o) { m = __builtin_elementwise_maximum(m, __builtin_bit_cast(float, o)); };
  with(dpp<kXor1>(__builtin_bit_cast(uint32_t, m)));
  with(dpp<kXor2>(__builtin_bit_cast(uint32_t, m)));
  if constexpr (G > 32) with(dpp<kXor7>(__builtin_bit_cast(uint32_t, m)));  // the other four lanes of eight
  if constexpr (G > 64) with(dpp<kXor15>(__builtin_bit_cast(uint32_t, m)));  // the other eight of sixteen
  float amax7 = quotient(fminf(m, 7.0f * kScaleMax), 7.0f, 1.0f / 7.0f);
  // rounded to fp32 here: joined into one instruction with the conversion it
  // would miss quotients half way between two subnormal scales
  asm("" : "+v"(amax7));
  const _Float16 h = (_Float16)amax7;
  const float s = (float)h, r = s > 0.0f ? __builtin_amdgcn_rcpf(s) : 0.0f, most = 7.0f * s;
  scale_bits = __builtin_bit_cast(uint16_t, h);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // adding 1.5 * 2^23 + 8 rounds to a whole number (half to even) and leaves n + 8 in the low bits
    const float u = quotient(__builtin_amdgcn_fmed3f(x[e], -most, most), s, r) + 12582920.0f;
    n[e] = __builtin_bit_cast(uint32_t, u);
  }
}

// Where a thread works: a token (clamped, all lanes of a wave stay for the
// exchanges) and its slot.
template <int D>
struct Place {
  static constexpr int kLanes = D / 8, kTokens = 256 / kLanes;
  int token, l, head, slot;
  bool has, inside;
  __device__ Place(const i4s_kv_cache &c, const int32_t *slots, int tokens, int shift) {
    // the heads of the same tokens run next to each other: they lie in the same rows of k and v
    const int block = blockIdx.x / c.kv_heads;
    const int64_t t = (int64_t)block * kTokens + threadIdx.x / kLanes;
    has = t < tokens;
    token = has ? (int)t : tokens - 1;
    l = threadIdx.x % kLanes;
    head = blockIdx.x - block * c.kv_heads;
    slot = slots[token];
    inside = slot >= 0 && (slot >> shift) < c.num_pages;
  }
};

template <typename T, int D, int G>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs a, int shift) {
  const Place<D> at(a.cache, a.slots, a.tokens, shift);
  const int token = at.token, l = at.l, head = at.head, slot = at.slot, heads = a.cache.kv_heads, page_size = 1 << shift;
  const f8_t xk = load8<T>(static_cast<const uint16_t *>(a.k) + token * a.k_token + head * a.k_head + 8 * l);
  const f8_t xv = load8<T>(static_cast<const uint16_t *>(a.v) + token * a.v_token + head * a.v_head + 8 * l);
  uint32_t sk, sv, nk[8], nv[8];
  quantize8<G>(xk, nk, sk);
  quantize8<G>(xv, nv, sv);
  // K: slot k of the word takes element (0,2,4,6,1,3,5,7)[k]; V for now in order
  const uint32_t word = low_bytes(nk[0], nk[4], nk[1], nk[5]) | low_bytes(nk[2], nk[6], nk[3], nk[7]) << 4;
  const uint32_t wv = low_bytes(nv[0], nv[2], nv[4], nv[6]) | low_bytes(nv[1], nv[3], nv[5], nv[7]) << 4;

  // V: lane l holds block c = l / 8, e = l % 8 / 2, b = l % 2; it collects the
  // words of the four e and makes halves x = 2e and 2e + 1 of i = 8b + x
  const int e = l % 8 / 2, b = l % 2, c = l / 8;
  uint32_t halves[2] = {0, 0};
  const uint32_t mirrored = dpp<kXor7>(wv);
  const uint32_t words[4] = {wv, dpp<kXor2>(wv), dpp<kXor3>(mirrored), dpp<kXor1>(mirrored)};  // of lanes l ^ 2d
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t two = words[d] >> (8 * e);
    const int from = e ^ d;
    halves[0] |= (two & 15u) << (4 * from);
    halves[1] |= (two >> 4 & 15u) << (4 * from);
  }
  const uint32_t other[2] = {dpp<kXor8>(halves[0]), dpp<kXor8>(halves[1])};
  if (!at.has || !at.inside) return;

  const int64_t base = (int64_t)(slot >> shift) * heads + head;
  const int off = slot & (page_size - 1);
  uint32_t *kv = reinterpret_cast<uint32_t *>(a.cache.k_vals + (base * page_size + off) * (D / 2));
  kv[(D / 32) * (l % 4) + l / 4] = word;
  uint32_t *vv = reinterpret_cast<uint32_t *>(a.cache.v_vals + (base * page_size + (off & ~3)) * (D / 2)) + (off & 3);
  if constexpr (D == 64) {
    vv[4 * (4 * b + e)] = halves[0] | halves[1] << 16;
  } else {
    // the lane of the other 64-channel block of a pair has the words' other halves: one word each
    const bool upper = c & 1;
    const uint32_t word_v = upper ? other[1] | halves[1] << 16 : halves[0] | other[0] << 16;
    vv[4 * (((8 * b + 2 * e + upper) * (D / 64) + c) / 2)] = word_v;
  }
  if (l % (G / 8) == 0) {
    const int64_t to = (base * page_size + (off & ~3)) * (D / G) + (l / (G / 8)) * 4 + (off & 3);
    a.cache.k_scales[to] = (uint16_t)sk;
    a.cache.v_scales[to] = (uint16_t)sv;
  }
}

// ---------------------------------------------------------------------------
// reading tokens: the same lanes the other way round
//
// Bound by: memory.  The same 8191 tokens: 213 MB in 34 us, 6.3 TB/s (the cache,
// just written, comes out of the last-level cache; 41 us with ordinary stores);
// as fp32 382 MB in 109 us, 3.5 TB/s (129 us with stores past the caches);
// 16 tokens 2.9 us.

template <typename T>
__device__ inline void store8(void *p, int64_t at, const f8_t &x) {
  u4_t w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = T::from_float(x[2 * i]) | T::from_float(x[2 * i + 1]) << 16;
  __builtin_nontemporal_store(w, reinterpret_cast<u4_t *>(static_cast<uint16_t *>(p) + at));
}
struct Float {};
template <>
__device__ inline void store8<Float>(void *p, int64_t at, const f8_t &x) {
  // two vectors of 16 bytes: the outputs have that alignment.  Not past the caches,
  // where each store would fill half lines only
  f4_t *to = reinterpret_cast<f4_t *>(static_cast<float *>(p) + at);
  to[0] = f4_t{x[0], x[1], x[2], x[3]};
  to[1] = f4_t{x[4], x[5], x[6], x[7]};
}

template <typename T, int D, int G>
__global__ __launch_bounds__(256) void kv_read_kernel(ReadArgs a, int shift) {
  const Place<D> place(a.cache, a.slots, a.tokens, shift);
  const int token = place.token, l = place.l, head = place.head, slot = place.slot;
  const int heads = a.cache.kv_heads, page_size = 1 << shift;
  const bool inside = place.inside;
  const int64_t base = (int64_t)(inside ? slot >> shift : 0) * heads + head;
  const int off = inside ? slot & (page_size - 1) : 0;

  const uint32_t *kv = reinterpret_cast<const uint32_t *>(a.cache.k_vals + (base * page_size + off) * (D / 2));
  const uint32_t word = kv[(D / 32) * (l % 4) + l / 4];
  const uint16_t *vv = reinterpret_cast<const uint16_t *>(a.cache.v_vals + (base * page_size + (off & ~3)) * (D / 2));
  const int e = l % 8 / 2, b = l % 2, c = l / 8;
  uint32_t two = 0;  // halves x = 2e and 2e + 1 of i = 8b + x
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int half = (8 * b + 2 * e + k) * (D / 64) + c;
    two |= (uint32_t)vv[(half / 2) * 8 + (off & 3) * 2 + half % 2] << (16 * k);
  }
  const int64_t at = (base * page_size + (off & ~3)) * (D / G) + (l / (G / 8)) * 4 + (off & 3);
  const float sk = Half::to_float(a.cache.k_scales[at]), sv = Half::to_float(a.cache.v_scales[at]);
  const uint32_t mirrored = dpp<kXor7>(two);
  const uint32_t words[4] = {two, dpp<kXor2>(two), dpp<kXor3>(mirrored), dpp<kXor1>(mirrored)};  // of lanes l ^ 2d
  f8_t xk, xv;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const float q = (float)((int)((word >> (4 * (x / 2 + 4 * (x % 2)))) & 15u) - 8);
    xk[x] = inside ? sk * q : 0.0f;
  }
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const uint32_t other = words[d];
    // the lane e ^ d holds halves 2(e^d) and 2(e^d) + 1; channel x of this lane is nibble e of half x
    const float q0 = (float)((int)((other >> (4 * e)) & 15u) - 8), q1 = (float)((int)((other >> (16 + 4 * e)) & 15u) - 8);
    const float v0 = inside ? sv * q0 : 0.0f, v1 = inside ? sv * q1 : 0.0f;
#pragma unroll
    for (int f = 0; f < 4; ++f)
      if ((e ^ d) == f) {
        xv[2 * f] = v0;
        xv[2 * f + 1] = v1;
      }
  }
  if (!place.has) return;
  const int64_t to = ((int64_t)token * heads + head) * D + 8 * l;
  store8<T>(a.k, to, xk);
  store8<T>(a.v, to, xv);
}

dim3 grid_of(int tokens, int heads, int head_dim) {
  const int per = 256 / (head_dim / 8);
  return dim3((unsigned)((tokens + (int64_t)per - 1) / per * heads));
}

template <template <typename, int, int> class Launch, typename T, typename A>
hipError_t by_shape(const A &a, hipStream_t s) {
  const int d = a.cache.head_dim, g = a.cache.group_size;
  if (d == 64) return g == 32 ? Launch<T, 64, 32>::go(a, s) : Launch<T, 64, 64>::go(a, s);
  if (d == 128)
    return g == 32 ? Launch<T, 128, 32>::go(a, s) : g == 64 ? Launch<T, 128, 64>::go(a, s) : Launch<T, 128, 128>::go(a, s);
  return g == 32 ? Launch<T, 256, 32>::go(a, s) : g == 64 ? Launch<T, 256, 64>::go(a, s) : Launch<T, 256, 128>::go(a, s);
}

template <typename T, int D, int G>
struct Append {
  static hipError_t go(const AppendArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kv_append_kernel<T, D, G>), grid_of(a.tokens, a.cache.kv_heads, D), dim3(256), 0, s, a,
                       page_shift(a.cache.page_size));
    return hipGetLastError();
  }
};

template <typename T, int D, int G>
struct Read {
  static hipError_t go(const ReadArgs &a, hipStream_t s) {
    hipLaunchKernelGGL((kv_read_kernel<T, D, G>), grid_of(a.tokens, a.cache.kv_heads, D), dim3(256), 0, s, a,
                       page_shift(a.cache.page_size));
    return hipGetLastError();
  }
};

}  // namespace

hipError_t launch_kv_extend(const ExtendArgs &a, hipStream_t stream) {
  const int threads = a.n <= 256 && a.capacity <= 4096 ? 256 : 1024;
  const int64_t blocks = clamp_to<int64_t>(((int64_t)a.capacity + threads - 1) / threads, 1, 256);
  const size_t lds = 2 * sizeof(int32_t) * ((size_t)a.n + 1);
  hipLaunchKernelGGL(kv_extend_kernel, dim3((unsigned)blocks), dim3(threads), lds, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_append(const AppendArgs &a, int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16 ? by_shape<Append, Half>(a, stream) : by_shape<Append, Bfloat>(a, stream);
}

hipError_t launch_kv_read(const ReadArgs &a, int32_t dtype, hipStream_t stream) {
  return dtype == I4S_F16    ? by_shape<Read, Half>(a, stream)
         : dtype == I4S_BF16 ? by_shape<Read, Bfloat>(a, stream)
                             : by_shape<Read, Float>(a, stream);
}

}  // namespace i4s
