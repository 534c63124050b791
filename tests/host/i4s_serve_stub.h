/* What the CPU stand-in for the serving launchers (i4s_serve_stub.cpp) saw.
 * Test infrastructure only. */
#pragma once

#include "i4s_serve_internal.h"

int serve_stub_launches();
const i4s::AttentionKernelArgs &serve_stub_attention();
const i4s::AttentionPlan &serve_stub_plan();
const i4s::LogprobsArgs &serve_stub_logprobs();
const i4s::ExtendArgs &serve_stub_extend();
