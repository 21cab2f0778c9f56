// What the masked attention kernels share: the capped score, with and without special
// functions.
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

// cap * log2(e) * tanh(y) + c on two scores y = raw * scale / cap of small size, without
// special functions: y P(y^2) cap log2(e), P fitted to tanh(y) / y over |y| <= 1/2 within
// 2^-20.7 relative (a cap of 50 is 72 in log2 units: 2^-15.6 on the largest such score). `k`
// holds P's coefficients times cap * log2(e), highest first.
__device__ __forceinline__ float2 capped_poly2(float2 y, const float* k, float2 c) {
  const float2 t = fmul2(y, y);
  float2 q = ffma2(t, make_float2(k[0], k[0]), make_float2(k[1], k[1]));
  q = ffma2(q, t, make_float2(k[2], k[2]));
  q = ffma2(q, t, make_float2(k[3], k[3]));
  return ffma2(y, q, c);
}
constexpr float kTanh4[4] = {-0.04440223425626755f, 0.13190299272537231f,
                                        -0.33326318860054016f, 0.999999463558197f};

}  // namespace ps
