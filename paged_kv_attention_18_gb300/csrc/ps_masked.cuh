// What the masked attention kernels share: the capped score, with and without special
// functions. Its error is within 2^-20 of the score, or in the tile kernel 2^-15 in log2 units if
// that is more (caps up to kLargeCapLog2).
#pragma once

#include "ps_common.cuh"
#include "ps_launch.h"

namespace ps {

constexpr float kLog2e = 1.4426950408889634f;

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

// cap * log2(e) * tanh(y) of a raw score, y = raw * scale / cap: tanh(y) = 1 - 2 / (e^2y + 1). A
// large y gives exactly 1 (the reciprocal of inf is 0), a large negative one exactly -1. The
// cancellation costs 2^-22 of 1 whatever y: nothing beside a large y, but all of a score that is
// small beside its cap.
__device__ __forceinline__ float capped_far(float raw, const MaskedAttnParams& p) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(fast_exp2(raw * p.cap_arg) + 1.f));
  return fmaf(r, -2.f * p.cap_log2, p.cap_log2);
}

// The same of any raw score, by the polynomial up to |y| = 1/2.
__device__ __forceinline__ float capped(float raw, const MaskedAttnParams& p) {
  const float y = raw * p.cap_y, t = y * y;
  const float near = y * fmaf(fmaf(fmaf(t, p.tanh4[0], p.tanh4[1]), t, p.tanh4[2]), t, p.tanh4[3]);
  return fabsf(y) > 0.5f ? capped_far(raw, p) : near;
}

// The scores of a warp's lanes, N each (even), capped in place, without special functions where
// the polynomial serves all of them.
template <int N>
__device__ __forceinline__ void cap_scores(float* s, const MaskedAttnParams& p) {
  bool far = false;
#pragma unroll
  for (int e = 0; e < N; ++e) far |= fabsf(s[e] * p.cap_y) > 0.5f;
  if (__any_sync(0xffffffffu, far)) {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] = capped(s[e], p);
  } else {
    const float2 cap_y2 = make_float2(p.cap_y, p.cap_y);
#pragma unroll
    for (int e = 0; e < N; e += 2) {
      const float2 x = capped_poly2(fmul2(make_float2(s[e], s[e + 1]), cap_y2), p.tanh4,
                                    make_float2(0.f, 0.f));
      s[e] = x.x;
      s[e + 1] = x.y;
    }
  }
}

}  // namespace ps
