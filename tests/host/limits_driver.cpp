// Driver for the CPU build of the serving operators' host layer: every size
// that include/i4s_serve.h bounds is accepted at its border and refused behind
// it.  Prints "ok <n> checks".

#include <cstdio>

#include "i4s_hip_stub.h"
#include "i4s_serve_stub.h"

namespace {

int g_checks = 0, g_fails = 0;

#define TAKES(call) expect((call), I4S_OK, #call, __LINE__)
#define REFUSES(call) expect((call), I4S_ERR_INVALID_ARGUMENT, #call, __LINE__)
void expect(i4s_status got, i4s_status want, const char *what, int line) {
  ++g_checks;
  if (got == want) return;
  ++g_fails;
  std::fprintf(stderr, "line %d: %s gives %d: %s\n", line, what, (int)got, i4s_last_error());
}

// Addresses far enough apart for every size used here; nothing is read there.
template <typename T> T *fake(uint64_t n) { return reinterpret_cast<T *>(static_cast<uintptr_t>(n) << 48); }

i4s_kv_cache cache_of(int pages, int page, int heads, int dim, int group) {
  i4s_kv_cache c{};
  c.num_pages = pages, c.page_size = page, c.kv_heads = heads, c.head_dim = dim, c.group_size = group;
  c.k_vals = fake<uint8_t>(1), c.v_vals = fake<uint8_t>(2), c.k_scales = fake<uint16_t>(3), c.v_scales = fake<uint16_t>(4);
  return c;
}

i4s_status extend(int n, int width, int page, int entries, int capacity) {
  return i4s_kv_extend(fake<int32_t>(1), n, width, page, fake<int32_t>(2), fake<int32_t>(3), fake<int32_t>(4), entries,
                       fake<int32_t>(5), capacity, fake<int32_t>(6), fake<int32_t>(7), fake<int32_t>(8), fake<int32_t>(9),
                       fake<int32_t>(10), fake<int32_t>(11), nullptr);
}

i4s_status append(int heads, int dim, int tokens, int64_t kt, int64_t kh) {
  const i4s_kv_cache c = cache_of(1, 16, heads, dim, 32);
  return i4s_kv_append(&c, fake<void>(5), fake<void>(6), I4S_F16, kt, kh, 8, 8, fake<int32_t>(7), tokens, nullptr);
}

i4s_status read(int heads, int dim, int tokens) {
  const i4s_kv_cache c = cache_of(1, 16, heads, dim, 32);
  return i4s_kv_read(&c, fake<int32_t>(7), tokens, I4S_F32, fake<void>(5), fake<void>(6), nullptr);
}

struct Attention {
  int kv_heads = 1, page = 16, q_heads = 1, tokens = 1, seqs = 1, width = 1, max_q = 1, max_len = 0;
  int64_t token_stride = 64, head_stride = 64;
  bool tree = false;
  i4s_status run() const {
    const i4s_kv_cache c = cache_of(1, page, kv_heads, 64, 32);
    i4s_attention_args a{};
    a.cache = &c, a.q = fake<void>(5), a.q_token_stride = token_stride, a.q_head_stride = head_stride, a.dtype = I4S_F16;
    a.q_heads = q_heads, a.num_tokens = tokens, a.num_seqs = seqs, a.table = fake<int32_t>(6), a.table_width = width;
    a.lens = fake<int32_t>(7), a.q_start = fake<int32_t>(8), a.max_q = max_q, a.max_len = max_len, a.scale = 1.0f;
    a.tree_mask = tree ? fake<int64_t>(9) : nullptr, a.out = fake<void>(10), a.lse = fake<float>(11);
    a.workspace = fake<void>(12), a.workspace_bytes = uint64_t(1) << 47;
    return i4s_attention(&a, nullptr);
  }
};

i4s_status scores(int rows, int vocab, int64_t stride, int top) {
  return i4s_token_logprobs(fake<void>(1), I4S_F16, rows, vocab, stride, fake<int64_t>(2), top, fake<float>(3), fake<float>(4),
                            fake<int32_t>(5), fake<float>(6), fake<void>(7), uint64_t(1) << 47, nullptr);
}

}  // namespace

int main() {
  const int64_t far = int64_t(1) << 40;
  const int most = 0x7FFFFFFF;
  i4s_kv_sizes sz;
  for (int page : {16, 32, 64, 128, 256}) {
    TAKES(i4s_kv_cache_sizes(most / page, page, 1024, 64, 64, &sz));
    REFUSES(i4s_kv_cache_sizes(most / page + 1, page, 1024, 64, 64, &sz));
  }
  TAKES(i4s_kv_cache_sizes(1, 16, 1, 128, 128, &sz));
  for (int heads : {0, 1025}) REFUSES(i4s_kv_cache_sizes(1, 16, heads, 64, 64, &sz));
  REFUSES(i4s_kv_cache_sizes(0, 16, 1, 64, 64, &sz));
  for (int page : {0, 8, 24, 512}) REFUSES(i4s_kv_cache_sizes(1, page, 1, 64, 64, &sz));

  TAKES(extend(0, 1, 16, 0, 0));
  TAKES(extend(I4S_KV_MAX_REQUESTS, most, 256, most, most));
  REFUSES(extend(I4S_KV_MAX_REQUESTS + 1, 1, 16, 1, 1));
  REFUSES(extend(1, 0, 16, 1, 1));
  REFUSES(extend(1, 1, 8, 1, 1));
  REFUSES(extend(1, 1, 512, 1, 1));
  REFUSES(extend(1, 1, 16, -1, 1));
  REFUSES(extend(1, 1, 16, 1, -1));

  for (int dim : {64, 128, 256})
    for (int heads : {1, 40, 1024}) {
      // the largest count with heads * (dim * tokens + 2048) below 2^34
      const int64_t tokens = (((int64_t(1) << 34) - 1) / heads - 2048) / dim;
      TAKES(append(heads, dim, (int)tokens, 8, 8));
      REFUSES(append(heads, dim, (int)tokens + 1, 8, 8));
      TAKES(read(heads, dim, (int)tokens));
      REFUSES(read(heads, dim, (int)tokens + 1));
    }
  TAKES(append(2, 64, 2, far, far));
  REFUSES(append(2, 64, 2, far + 8, 8));
  REFUSES(append(2, 64, 2, 8, far + 8));
  TAKES(append(2, 64, 2, 0, 0));
  REFUSES(append(2, 64, 2, -8, 8));
  REFUSES(append(2, 64, 2, 8, 12));

  Attention a;
  TAKES(a.run());
  for (int64_t s : {int64_t(0), far}) {
    a = Attention(), a.token_stride = s;
    TAKES(a.run());
    a = Attention(), a.head_stride = s;
    TAKES(a.run());
  }
  a = Attention(), a.token_stride = far + 8;
  REFUSES(a.run());
  a = Attention(), a.head_stride = far + 8;
  REFUSES(a.run());
  a = Attention(), a.q_heads = 65536;
  TAKES(a.run());
  a.q_heads = 65537;
  REFUSES(a.run());
  a = Attention(), a.seqs = 65535;
  TAKES(a.run());
  a.seqs = 65536;
  REFUSES(a.run());
  for (int page : {16, 256}) {
    a = Attention(), a.page = page, a.width = (1 << 30) / page;
    TAKES(a.run());
    a.max_len = most;
    TAKES(a.run());
    ++a.width;
    REFUSES(a.run());
  }
  a = Attention(), a.max_q = 1 << 20;
  TAKES(a.run());
  a.q_heads = 7;
  TAKES(a.run());
  a.q_heads = 8;
  REFUSES(a.run());
  a = Attention(), a.max_q = (1 << 20) + 1;
  REFUSES(a.run());
  a = Attention(), a.max_q = 0;
  REFUSES(a.run());
  a = Attention(), a.max_q = I4S_MAX_TREE, a.tree = true;
  TAKES(a.run());
  ++a.max_q;
  REFUSES(a.run());
  a = Attention(), a.max_len = -1;
  REFUSES(a.run());
  a = Attention(), a.width = 0;
  REFUSES(a.run());

  TAKES(scores((1 << 23) - 1, 1, 1, 1));
  REFUSES(scores(1 << 23, 1, 1, 1));
  TAKES(scores(2, I4S_MAX_VOCAB, far, I4S_MAX_TOP_K));
  REFUSES(scores(2, I4S_MAX_VOCAB + 1, far, 1));
  REFUSES(scores(2, 100, far + 1, 1));
  REFUSES(scores(2, 100, 99, 1));
  REFUSES(scores(2, 100, 100, I4S_MAX_TOP_K + 1));
  TAKES(scores(2, 31, 31, 31));
  REFUSES(scores(2, 31, 31, 32));
  if (g_fails) return 1;
  std::printf("ok %d checks\n", g_checks);
  return 0;
}
