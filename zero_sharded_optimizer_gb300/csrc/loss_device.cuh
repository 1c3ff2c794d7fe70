// Device functions shared by the vocabulary losses' kernels.
#pragma once

#include "launch.cuh"
#include "loss_internal.h"

namespace zl {

constexpr float kLog2e = 1.4426950408889634f;

}  // namespace zl
