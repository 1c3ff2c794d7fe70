// Device functions shared by the vocabulary losses' kernels.
#pragma once

#include "loss_internal.h"

namespace zl {

constexpr float kLog2e = 1.4426950408889634f;

// Programmatic launches: every kernel of a call lets the next one start when
// its own blocks run, and waits for the one before it (complete, and so for all
// before that) before it touches what they wrote.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace zl
