// Driver for the CPU build of the prompt's host layer (i4s_prompt_api.cpp)
// against the stand-ins, built with AddressSanitizer and
// UndefinedBehaviorSanitizer: valid calls reach their launchers with the
// arguments they should have; the launch shapes hold what the kernels assume
// over a sweep of sizes, the largest included; and a device of another
// architecture is refused.  Prints "ok <n> checks".

#include <cstdio>
#include <cstring>

#include "i4s_hip_stub.h"
#include "i4s_prompt_stub.h"

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

template <typename T> T *fake(uint64_t at) { return reinterpret_cast<T *>(static_cast<uintptr_t>(at) << 44); }

i4s_mx mx_of(int32_t rows, int32_t cols, uint64_t at) { return {rows, cols, fake<uint8_t>(at), fake<uint8_t>(at + 1)}; }

void format(i4s_status expect) {
  for (int32_t rows : {1, 15, 17, 4096, 50257, 1 << 18, 1 << 24})
    for (int32_t cols : {32, 256, 288, 4096, 1 << 13, 1 << 20}) {
      i4s_mx_buffers sz{};
      const bool fits = (int64_t)((rows + 15) / 16) * ((cols + 511) / 512) <= 4ll * i4s::kMaxBlocks;
      CHECK(i4s_mx_sizes(rows, cols, &sz) == (fits ? I4S_OK : I4S_ERR_INVALID_ARGUMENT));
      if (!fits) continue;
      CHECK(sz.vals >= (uint64_t)rows * cols / 2 && sz.scales >= (uint64_t)rows * cols / 32);
      // a block of a wave for each: 32-bit grids
      CHECK((int64_t)((rows + 15) / 16) * ((cols + 511) / 512) * 64 < (int64_t(1) << 32));
      const i4s_mx m = mx_of(rows, cols, 1);
      const int before = prompt_stub_launches();
      CHECK(i4s_mx_quantize(fake<void>(100), I4S_BF16, cols, &m, nullptr) == expect);
      CHECK(i4s_mx_read(&m, I4S_F32, fake<void>(100), nullptr) == expect);
      CHECK(prompt_stub_launches() == before + (expect == I4S_OK ? 2 : 0));
      if (expect == I4S_OK) CHECK(prompt_stub_quantize().rows == rows && prompt_stub_quantize().stride == cols);
    }
}

void products(i4s_status expect) {
  for (int32_t tokens : {1, 2, 15, 16, 17, 32, 33, 64, 65, 256, 257, 4096, 8191, 1 << 20, 1 << 24})
    for (int32_t rows : {1, 16, 4000, 4096, 4097, 8192, 8193, 16384, 16385, 50257, 1 << 20, 1 << 24})
      for (int32_t cols : {32, 4064, 4096, 4128, 1 << 17, 1 << 20})
        for (bool given : {false, true}) {
          const i4s_mx w = mx_of(rows, cols, 1), x = mx_of(tokens, cols, 3);
          i4s_mx_product_args a{};
          a.w = &w, a.tokens = tokens, a.y = fake<void>(200), a.y_stride = rows, a.y_dtype = I4S_F16;
          a.x_values = fake<void>(100), a.x_stride = cols, a.x_dtype = I4S_F16;
          if (given) a.x = &x;
          uint64_t bytes = 0;
          const bool fits = (int64_t)((rows + 15) / 16) * ((cols + 511) / 512) <= 4ll * i4s::kMaxBlocks &&
                            (int64_t)((tokens + 15) / 16) * ((cols + 511) / 512) <= 4ll * i4s::kMaxBlocks &&
                            (int64_t)((tokens + 127) / 128) * ((rows + 127) / 128) <= i4s::kMaxBlocks;
          CHECK(i4s_mx_product_workspace_size(&a, &bytes) == (fits ? I4S_OK : I4S_ERR_INVALID_ARGUMENT));
          if (!fits) continue;
          a.workspace = fake<void>(300), a.workspace_bytes = bytes;
          const int before = prompt_stub_launches();
          CHECK(i4s_mx_product(&a, nullptr) == expect);
          if (expect != I4S_OK) {
            CHECK(prompt_stub_launches() == before);
            continue;
          }
          const i4s::MxProductPlan &p = prompt_stub_product_plan();
          const i4s::MxProductKernelArgs &k = prompt_stub_product();
          CHECK(prompt_stub_launches() == before + 1 + p.quantize);
          CHECK(!(given && p.quantize) && (bytes > 0) == p.quantize);
          CHECK(p.token_tiles == (tokens + 15) / 16);
          const bool fused = !given && !p.quantize;
          CHECK((k.x != nullptr) == fused && (k.x_vals != nullptr) == !fused && (k.x_scales != nullptr) == !fused);
          if (p.quantize) CHECK(k.x_vals == (uint8_t *)a.workspace && k.x_scales + i4s::mx_scales_bytes(tokens, cols) == k.x_vals + bytes);
          if (p.few) {  // what is instantiated
            CHECK((p.row_tiles == 1 && p.waves == 8) || (p.row_tiles == 2 && (p.waves == 8 || p.waves == 4)) ||
                  (p.row_tiles == 4 && p.waves == 8 && fused));
            CHECK(p.token_tiles <= 4 || (p.row_tiles == 2 && p.waves == 4));
            CHECK((p.token_tiles + 3) / 4 <= 65535);  // grid.y
          } else {
            CHECK(p.tile == 64 || p.tile == 128 || p.tile == 256);
          }
          if (fused) CHECK(p.few && tokens <= 16);
          // the order of the sums does not depend on how the tokens are given
          const i4s::MxProductPlan q = i4s::mx_product_plan(tokens, rows, cols, !given);
          CHECK(q.few == p.few && q.tile == p.tile && (!p.few || q.waves == p.waves));
        }
}

void attention(i4s_status expect) {
  for (int dim : {64, 128, 256})
    for (int heads : {1, 8, 40, 1024})
      for (int share : {1, 5, 8, 64})
        for (int seqs : {1, 3, 64, 65535})
          for (int max_q : {1, 2, 16, 129, 2048, 1 << 20, 1 << 24})
            for (int max_k : {0, 1, 512, 513, 8191, 131071, 1 << 30})
              for (int keys : {0, 1, 65536, 1 << 30}) {
                i4s_prompt_args a{};
                a.q = fake<void>(100), a.k = fake<void>(200), a.v = fake<void>(5000);
                a.dtype = I4S_BF16, a.head_dim = dim, a.q_heads = heads * share, a.kv_heads = heads;
                a.k_token_stride = 8, a.v_token_stride = 1 << 23;
                a.q_head_stride = a.k_head_stride = a.v_head_stride = dim;
                a.num_tokens = 1 << 20, a.num_keys = keys, a.num_seqs = seqs, a.max_q = max_q, a.max_k = max_k;
                a.causal = 1, a.scale = 1e38f, a.out = fake<void>(400), a.q_start = fake<int32_t>(50), a.k_start = fake<int32_t>(51);
                const int64_t blocks = ((int64_t)max_q * share + 127) / 128 * heads * seqs;
                const bool fits = blocks <= i4s::kMaxBlocks && a.q_heads <= 65536;
                uint64_t bytes = 0;
                CHECK(i4s_prompt_attention_workspace_size(&a, &bytes) == (fits ? I4S_OK : I4S_ERR_INVALID_ARGUMENT));
                if (!fits) continue;
                a.workspace = fake<void>(500), a.workspace_bytes = bytes;
                const int before = prompt_stub_launches();
                CHECK(i4s_prompt_attention(&a, nullptr) == expect);
                CHECK(prompt_stub_launches() == before + (expect == I4S_OK));
                if (expect != I4S_OK) continue;
                const i4s::PromptPlan &p = prompt_stub_plan();
                const i4s::PromptKernelArgs &k = prompt_stub_attention();
                const int64_t len = max_k > 0 && max_k < keys ? max_k : keys;
                CHECK((p.rows == 32) == ((int64_t)max_q * share <= 32));
                CHECK(p.rows == 32 || p.rows == 128 || (p.rows == 256 && dim == 128));  // what is instantiated
                CHECK((int64_t)p.row_blocks * p.rows >= (int64_t)max_q * share);
                CHECK((int64_t)p.row_blocks * heads * seqs * 2 * p.rows < (int64_t(1) << 31));  // threads of the grid, at most
                CHECK(p.group >= 8 && (int64_t)p.group * p.row_blocks < (int64_t(1) << 30));
                CHECK(p.chunk > 0 && p.chunk % i4s::kPromptKeys == 0);
                CHECK(p.splits >= 1 && p.splits <= i4s::kMaxPromptSplits);
                CHECK((int64_t)p.chunk * p.splits >= len && ((int64_t)p.chunk * (p.splits - 1) < len || len == 0));
                CHECK((int64_t)p.chunk * p.splits < (int64_t(1) << 31));  // where pieces begin
                CHECK((p.splits > 1) == (bytes > 0));
                if (p.splits > 1) {
                  CHECK(p.chunk >= 512 || p.splits == 2);
                  CHECK((int64_t)max_q * a.q_heads * 256 < (int64_t(1) << 31));  // threads of the joining launch
                  CHECK(bytes == 4ull * p.splits * a.num_tokens * a.q_heads * (dim + 2));
                  CHECK(k.part_o == a.workspace && k.part_ml == k.part_o + (uint64_t)p.splits * a.num_tokens * a.q_heads * dim);
                }
                CHECK(k.share == share && k.splits == p.splits && k.chunk == p.chunk && k.group == p.group);
                CHECK(k.scale_log2 > 0 && k.scale_log2 <= 3.4028235e38f);
              }
}

void one_sequence(i4s_status expect) {  // needs no starts
  i4s_prompt_args a{};
  a.q = fake<void>(100), a.k = fake<void>(200), a.v = fake<void>(300), a.out = fake<void>(400);
  a.head_dim = 64, a.q_heads = a.kv_heads = 1, a.num_tokens = a.num_keys = 9, a.max_q = 9, a.num_seqs = 1, a.scale = 1;
  CHECK(i4s_prompt_attention(&a, nullptr) == expect);
  if (expect == I4S_OK) CHECK(!prompt_stub_attention().q_start && !prompt_stub_attention().k_start);
  a.num_seqs = 2;
  CHECK(i4s_prompt_attention(&a, nullptr) == I4S_ERR_INVALID_ARGUMENT);
}

void nothing_to_do() {
  const int before = prompt_stub_launches();
  const i4s_mx none = {0, 64, nullptr, nullptr}, w = mx_of(20, 64, 1);
  CHECK(i4s_mx_quantize(nullptr, I4S_F16, 64, &none, nullptr) == I4S_OK);
  CHECK(i4s_mx_read(&none, I4S_F16, nullptr, nullptr) == I4S_OK);
  i4s_mx_product_args p{};
  p.w = &w, p.x_stride = 64, p.y_stride = 20;
  CHECK(i4s_mx_product(&p, nullptr) == I4S_OK);
  p.w = &none, p.tokens = 5;
  CHECK(i4s_mx_product(&p, nullptr) == I4S_OK);
  i4s_prompt_args a{};
  a.head_dim = 64, a.q_heads = a.kv_heads = 1, a.max_q = 1, a.scale = 1;
  CHECK(i4s_prompt_attention(&a, nullptr) == I4S_OK);
  a.num_tokens = 5;
  CHECK(i4s_prompt_attention(&a, nullptr) == I4S_OK);  // no sequences
  CHECK(prompt_stub_launches() == before);
}

}  // namespace

int main(int argc, char **argv) {
  i4s_status expect = I4S_OK;
  if (argc == 3 && !std::strcmp(argv[1], "--arch")) {
    i4s_stub_set_arch(argv[2]);
    expect = I4S_ERR_UNSUPPORTED;
  }
  format(expect);
  products(expect);
  attention(expect);
  one_sequence(expect);
  nothing_to_do();
  if (g_fails) return 1;
  std::printf("ok %d checks\n", g_checks);
  return 0;
}
