/* What the CPU stand-in for the prompt's launchers (i4s_prompt_stub.cpp) saw.
 * Test infrastructure only. */
#pragma once

#include "i4s_prompt_internal.h"

int prompt_stub_launches();
const i4s::MxQuantizeArgs &prompt_stub_quantize();
const i4s::MxProductKernelArgs &prompt_stub_product();
const i4s::MxProductPlan &prompt_stub_product_plan();
const i4s::PromptKernelArgs &prompt_stub_attention();
const i4s::PromptPlan &prompt_stub_plan();
