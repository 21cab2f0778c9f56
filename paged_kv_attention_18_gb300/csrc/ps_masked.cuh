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

// The same on two scores whose |y| = |raw| scale / cap is at most 1, without special
// functions: tanh(y) = y P(y^2), P of degree 5 fitted to a largest relative error of
// 2^-20.6 over |y| <= 1 (a cap of 50 is 72 in log2 units: 2^-14.4 on the score). `y_of` is
// scale / cap. `top` is raised to the largest y^2: above 1 the result does not hold.
__device__ __forceinline__ float2 capped_small2(float2 raw, float y_of, float cap_log2,
                                                float& top) {
  const float2 y = fmul2(raw, make_float2(y_of, y_of));
  const float2 t = fmul2(y, y);
  top = fmax3(top, t.x, t.y);
  auto two = [](float c) { return make_float2(c, c); };
  float2 q = ffma2(t, two(-0.003067068289965391f), two(0.016743160784244537f));
  q = ffma2(q, t, two(-0.051605746150016785f));
  q = ffma2(q, t, two(0.13281437754631042f));
  q = ffma2(q, t, two(-0.3332904279232025f));
  q = ffma2(q, t, two(0.9999994039535522f));
  return fmul2(fmul2(y, two(cap_log2)), q);
}

}  // namespace ps
