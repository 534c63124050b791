// Stand-ins for the kernel launchers of the prompt's operators, so that their
// host layer (i4s_prompt_api.cpp) can be built for the CPU alone; see
// i4s_hip_stub.cpp.  A launch is counted and its arguments are kept.  Test
// infrastructure only.

#include "i4s_prompt_stub.h"

namespace {
int g_launches = 0;
i4s::MxQuantizeArgs g_quantize{};
i4s::MxProductKernelArgs g_product{};
i4s::MxProductPlan g_product_plan{};
i4s::PromptKernelArgs g_attention{};
i4s::PromptPlan g_plan{};
}  // namespace

int prompt_stub_launches() { return g_launches; }
const i4s::MxQuantizeArgs &prompt_stub_quantize() { return g_quantize; }
const i4s::MxProductKernelArgs &prompt_stub_product() { return g_product; }
const i4s::MxProductPlan &prompt_stub_product_plan() { return g_product_plan; }
const i4s::PromptKernelArgs &prompt_stub_attention() { return g_attention; }
const i4s::PromptPlan &prompt_stub_plan() { return g_plan; }

namespace i4s {

hipError_t launch_mx_quantize(const MxQuantizeArgs &a, int32_t, hipStream_t) {
  ++g_launches;
  g_quantize = a;
  return hipSuccess;
}
hipError_t launch_mx_read(const MxReadArgs &, int32_t, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
hipError_t launch_mx_product(const MxProductKernelArgs &a, const MxProductPlan &p, int32_t, hipStream_t) {
  ++g_launches;
  g_product = a;
  g_product_plan = p;
  return hipSuccess;
}
hipError_t launch_prompt_attention(const PromptKernelArgs &a, const PromptPlan &p, int32_t, int32_t, hipStream_t) {
  ++g_launches;
  g_attention = a;
  g_plan = p;
  return hipSuccess;
}

}  // namespace i4s
