// Driver for the CPU build of the serving operators' host layer
// (i4s_serve_api.cpp) against the stand-ins, built with AddressSanitizer and
// UndefinedBehaviorSanitizer: valid calls reach their launcher once, with the
// arguments they should have; calls with nothing to do launch nothing; the
// launch shapes hold what the kernels assume over a sweep of sizes; and a
// device of another architecture is refused.  Prints "ok <n> checks".

#include <cstdio>
#include <cstring>

#include "i4s_hip_stub.h"
#include "i4s_serve_stub.h"

namespace {

int g_checks = 0, g_fails = 0;

#define CHECK(cond)                                                                                     \
  do {                                                                                                  \
    ++g_checks;                                                                                         \
    if (!(cond)) {                                                                                      \
      ++g_fails;                                                                                        \
      std::fprintf(stderr, "%s:%d: CHECK(%s) failed; last error: %s\n", __FILE__, __LINE__, #cond,   \
                   i4s_last_error());                                                                   \
    }                                                                                                   \
  } while (0)

template <typename T> T *fake(uint64_t gib) { return reinterpret_cast<T *>(static_cast<uintptr_t>(gib) << 32); }

i4s_kv_cache cache_of(int pages, int page, int heads, int dim, int group) {
  i4s_kv_cache c{};
  c.num_pages = pages, c.page_size = page, c.kv_heads = heads, c.head_dim = dim, c.group_size = group;
  c.k_vals = fake<uint8_t>(100), c.v_vals = fake<uint8_t>(200), c.k_scales = fake<uint16_t>(300);
  c.v_scales = fake<uint16_t>(400);
  return c;
}

i4s_attention_args args_of(const i4s_kv_cache &c, int seqs, int max_q, int share, int width, int max_len) {
  i4s_attention_args a{};
  a.cache = &c;
  a.q = fake<void>(500), a.q_token_stride = (int64_t)c.kv_heads * share * c.head_dim, a.q_head_stride = c.head_dim;
  a.dtype = I4S_F16, a.q_heads = c.kv_heads * share, a.num_tokens = seqs * max_q, a.num_seqs = seqs;
  a.table = fake<int32_t>(600), a.table_width = width, a.lens = fake<int32_t>(700), a.q_start = fake<int32_t>(800);
  a.max_q = max_q, a.max_len = max_len, a.scale = 0.1f, a.out = fake<void>(900);
  a.workspace = fake<void>(1000), a.workspace_bytes = uint64_t(1) << 50;
  return a;
}

void attention_shapes(i4s_status expect) {
  for (int dim : {64, 128, 256})
    for (int group : {32, 64, 128})
      for (int heads : {1, 8, 40})
        for (int share : {1, 5, 8})
          for (int seqs : {1, 3, 64, 5000})
            for (int max_q : {1, 2, 16, 300})
              for (int len : {1, 31, 1024, 1025, 4097, 131071, 1 << 30}) {
                if (group > dim) continue;
                const i4s_kv_cache c = cache_of(1000, 256, heads, dim, group);
                i4s_attention_args a = args_of(c, seqs, max_q, share, 1 << 22, len);
                const int before = serve_stub_launches();
                uint64_t bytes = 0;
                CHECK(i4s_attention_workspace_size(&a, &bytes) == I4S_OK);
                const i4s_status st = i4s_attention(&a, nullptr);
                CHECK(st == expect);
                if (expect != I4S_OK) {
                  CHECK(serve_stub_launches() == before);
                  continue;
                }
                CHECK(serve_stub_launches() == before + 1);
                const i4s::AttentionPlan &p = serve_stub_plan();
                const i4s::AttentionKernelArgs &k = serve_stub_attention();
                CHECK(p.row_tiles == 1 || (p.row_tiles == 2 && dim / group >= 4));  // what is instantiated
                CHECK(p.waves == 4 || (p.waves == 8 && p.row_tiles == 1 && dim <= 128));
                CHECK((int64_t)p.row_blocks * 16 * p.row_tiles >= (int64_t)max_q * share);
                CHECK(p.chunk > 0 && p.chunk % (i4s::kStepKeys * p.waves) == 0);
                CHECK(p.splits >= 1 && p.splits <= i4s::kMaxSplits);
                CHECK((int64_t)p.chunk * (p.splits - 1) < len && (int64_t)p.chunk * p.splits >= len);
                CHECK((int64_t)p.chunk * p.splits < (int64_t(1) << 31) - 4096);  // key positions are 32-bit
                CHECK((p.splits > 1) == (bytes > 0));
                if (bytes) {
                  const uint64_t rows = (uint64_t)a.num_tokens * a.q_heads;
                  CHECK(bytes == 4 * (uint64_t)p.splits * rows * (dim + 2) + 4 * (uint64_t)p.splits * rows * 2);
                  CHECK(k.part_ml == k.part_o + (uint64_t)p.splits * rows * dim);
                }
                CHECK(k.share == share && k.row_blocks == p.row_blocks && k.splits == p.splits && k.shift == 8);
              }
}

void others(i4s_status expect) {
  const i4s_kv_cache c = cache_of(10, 32, 4, 64, 64);
  int before = serve_stub_launches();
  const int one = expect == I4S_OK;
  CHECK(i4s_kv_append(&c, fake<void>(1), fake<void>(2), I4S_BF16, 256, 64, 256, 64, fake<int32_t>(3), 5, nullptr) == expect);
  CHECK(i4s_kv_read(&c, fake<int32_t>(3), 5, I4S_F32, fake<void>(1), fake<void>(2), nullptr) == expect);
  CHECK(i4s_kv_extend(fake<int32_t>(1), 3, 4, 64, fake<int32_t>(2), fake<int32_t>(3), fake<int32_t>(4), 5, fake<int32_t>(5), 6,
                      fake<int32_t>(6), fake<int32_t>(7), fake<int32_t>(8), fake<int32_t>(9), fake<int32_t>(10),
                      fake<int32_t>(11), nullptr) == expect);
  CHECK(serve_stub_launches() == before + 3 * one);
  if (one) CHECK(serve_stub_extend().shift == 6 && serve_stub_extend().capacity == 6);
  for (int dtype : {I4S_F16, I4S_BF16, I4S_F32})
    for (int rows : {1, 2, 16, 100, 256, 257, 4093})
      for (int vocab : {1, 100, 8192, 8193, 32768, 50257, 151643, 1 << 20, I4S_MAX_VOCAB})
        for (int top : {0, 1, 32}) {
          if (top > vocab) continue;
          uint64_t bytes = 0;
          CHECK(i4s_token_logprobs_workspace_size(dtype, rows, vocab, top, &bytes) == I4S_OK);
          const i4s::LogprobsPlan p = i4s::logprobs_plan(dtype, rows, vocab, top);
          CHECK(p.splits >= 1 && p.splits <= i4s::kMaxLogprobsSplits && p.segments >= 1 && p.segments <= i4s::kMaxSegments);
          // every row fits, wherever in a 128-byte line it begins
          CHECK((int64_t)p.splits * p.segments * i4s::kSegment >= (int64_t)vocab + 128 / (dtype == I4S_F32 ? 4 : 2) - 1);
          CHECK(bytes == (p.splits > 1 ? (uint64_t)rows * p.splits * (16 + 8 * top) : 0));
          before = serve_stub_launches();
          CHECK(i4s_token_logprobs(fake<void>(1), dtype, rows, vocab, vocab, fake<int64_t>(100), top, fake<float>(101),
                                   fake<float>(102), fake<int32_t>(103), fake<float>(104), fake<void>(105), bytes,
                                   nullptr) == expect);
          CHECK(serve_stub_launches() == before + one);
          if (one && p.splits > 1)
            CHECK((const char *)serve_stub_logprobs().part_stats ==
                  (const char *)fake<void>(105) + 8ull * rows * p.splits * top);
        }
}

void nothing_to_do() {
  const int before = serve_stub_launches();
  const i4s_kv_cache c = cache_of(10, 32, 4, 64, 64);
  CHECK(i4s_kv_append(&c, nullptr, nullptr, I4S_F16, 0, 0, 0, 0, nullptr, 0, nullptr) == I4S_OK);
  CHECK(i4s_kv_read(&c, nullptr, 0, I4S_F16, nullptr, nullptr, nullptr) == I4S_OK);
  i4s_attention_args a = args_of(c, 0, 1, 1, 4, 0);
  CHECK(i4s_attention(&a, nullptr) == I4S_OK);
  CHECK(i4s_token_logprobs(nullptr, I4S_F16, 0, 5, 5, nullptr, 0, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) ==
        I4S_OK);
  CHECK(serve_stub_launches() == before);
}

}  // namespace

int main(int argc, char **argv) {
  i4s_status expect = I4S_OK;
  if (argc == 3 && !std::strcmp(argv[1], "--arch")) {
    i4s_stub_set_arch(argv[2]);
    expect = I4S_ERR_UNSUPPORTED;
  }
  attention_shapes(expect);
  others(expect);
  nothing_to_do();
  if (g_fails) return 1;
  std::printf("ok %d checks\n", g_checks);
  return 0;
}
