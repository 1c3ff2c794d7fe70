// Device functions shared by the vocabulary losses' kernels.
#pragma once

#include "loss_internal.h"

namespace zl {

constexpr float kLog2e = 1.4426950408889634f;

// A value as bf16 parts: x = p0 + p1 + p2 up to fp32's rounding (each part
// holds the next 8 bits; the rests are exact differences). An infinity and
// a value that would round to one keep the parts finite or zero.
__device__ __forceinline__ void split(float x, __nv_bfloat16 (&part)[3]) {
  part[0] = __float2bfloat16_rn(x);
  if (isinf(__bfloat162float(part[0])) && !isinf(x)) part[0] = __float2bfloat16_rz(x);
  if (isinf(x)) {
    part[1] = part[2] = __float2bfloat16_rn(0.0f);
    return;
  }
  const float r = x - __bfloat162float(part[0]);
  part[1] = __float2bfloat16_rn(r);
  part[2] = __float2bfloat16_rn(r - __bfloat162float(part[1]));
}

// Programmatic launches: every kernel of a call lets the next one start when
// its own blocks run, and waits for the one before it (complete, and so for all
// before that) before it touches what they wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace zl
