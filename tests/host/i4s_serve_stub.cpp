// Stand-ins for the kernel launchers of the serving operators, so that their
// host layer (i4s_serve_api.cpp) can be built for the CPU alone; see
// i4s_hip_stub.cpp.  A launch is counted and its arguments are kept.  Test
// infrastructure only.

#include "i4s_serve_stub.h"

namespace {
int g_launches = 0;
i4s::AttentionKernelArgs g_attention{};
i4s::AttentionPlan g_plan{};
i4s::LogprobsArgs g_logprobs{};
i4s::ExtendArgs g_extend{};
}  // namespace

int serve_stub_launches() { return g_launches; }
const i4s::AttentionKernelArgs &serve_stub_attention() { return g_attention; }
const i4s::AttentionPlan &serve_stub_plan() { return g_plan; }
const i4s::LogprobsArgs &serve_stub_logprobs() { return g_logprobs; }
const i4s::ExtendArgs &serve_stub_extend() { return g_extend; }

namespace i4s {

hipError_t launch_kv_extend(const ExtendArgs &a, hipStream_t) {
  ++g_launches;
  g_extend = a;
  return hipSuccess;
}
hipError_t launch_kv_append(const AppendArgs &, int32_t, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_kv_read(const ReadArgs &, int32_t, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_attention(const AttentionKernelArgs &a, const AttentionPlan &p, int32_t, int32_t, int32_t, hipStream_t) {
  ++g_launches;
  g_attention = a;
  g_plan = p;
  return hipSuccess;
}
hipError_t launch_token_logprobs(const LogprobsArgs &a, const LogprobsPlan &, int32_t, hipStream_t) {
  ++g_launches;
  g_logprobs = a;
  return hipSuccess;
}

}  // namespace i4s
