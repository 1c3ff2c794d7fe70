// Device functions shared by the vocabulary losses' kernels.
#pragma once

#include "launch.cuh"
#include "loss_internal.h"

namespace zl {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eRest = 1.4426950408889634 - double(kLog2e);

// 2^x for x <= 0, by the series of 2^f around the nearest whole exponent: off by a
// rounding or two in either direction, where the hardware's exponential is a little
// low on average (4.8e-8), which adds up over sums that are rescaled again and again.
__device__ __forceinline__ float exp2_even(float x) {
  const float n = fmaxf(rintf(x), -127.0f), f = fmaxf(x, -127.0f) - n;  // (-inf: zero)
  constexpr double kLn2 = 0.69314718055994530942;
  // the terms ln2^k / k!
  constexpr double c2 = kLn2 * kLn2 / 2, c3 = c2 * kLn2 / 3, c4 = c3 * kLn2 / 4, c5 = c4 * kLn2 / 5, c6 = c5 * kLn2 / 6,
                   c7 = c6 * kLn2 / 7;
  float p = fmaf(float(c7), f, float(c6));
  p = fmaf(p, f, float(c5));
  p = fmaf(p, f, float(c4));
  p = fmaf(p, f, float(c3));
  p = fmaf(p, f, float(c2));
  p = fmaf(p, f, float(kLn2));
  p = fmaf(p, f, 1.0f);
  const float y = n <= -127.0f ? 0.0f : p * __int_as_float((int(n) + 127) << 23);
  return x == x ? y : x;
}

}  // namespace zl
