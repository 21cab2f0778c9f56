// What the masked attention kernels share: the capped score.
#pragma once

#include "ps_common.cuh"

namespace ps {

constexpr float kLog2e = 1.4426950408889634f;

// cap * log2(e) * tanh(y) with 2 y log2(e) = raw * arg: tanh(y) = 1 - 2 / (e^2y + 1). A
// large y gives exactly 1 (the reciprocal of inf is 0), a large negative one exactly -1.
__device__ __forceinline__ float capped(float raw, float arg, float cap_log2) {
  const float e = fast_exp2(raw * arg);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 1.f));
  return fmaf(r, -2.f * cap_log2, cap_log2);
}

}  // namespace ps
