// pa_score.cuh -- the capped score of pa_extend_scored and pa_decode_scored.
#pragma once

#include <cmath>

#include "pa_common.cuh"

namespace pa {

// tanh on [-1, 1] as t P(t^2), P of degree 5 fitted to the least largest relative error, 5.9e-7
// (2^-20.7): in the exponent of a weight of a score capped at 50 that is 3e-5 at most, where the
// weight's rounding to bf16 is 2^-8.
constexpr float kTanh0 = 0.99999941f, kTanh1 = -0.33329042f, kTanh2 = 0.13281434f,
                kTanh3 = -0.05160567f, kTanh4 = 0.01674311f, kTanh5 = -0.00306706f;

// On [-1/2, 1/2] four terms come as near (5.5e-7).
constexpr float kTanhHalf0 = 0.99999946f, kTanhHalf1 = -0.33326318f, kTanhHalf2 = 0.13190297f,
                kTanhHalf3 = -0.04440223f;

__device__ __forceinline__ float tanh_within_1(float t) {
  const float u = t * t;
  float y = fmaf(u, kTanh5, kTanh4);
  y = fmaf(u, y, kTanh3);
  y = fmaf(u, y, kTanh2);
  y = fmaf(u, y, kTanh1);
  y = fmaf(u, y, kTanh0);
  return t * y;
}

// tanh anywhere: 1 - 2 / (1 + e^2t) past 1, where its error of some 2^-23 is one of the result, too.
__device__ __forceinline__ float tanh_any(float t) {
  const float far = 1.f - __fdividef(2.f, 1.f + ex2(t * (2.f * kLog2e)));
  return fabsf(t) <= 1.f ? tanh_within_1(t) : far;
}

// What a product is multiplied by under a cap, kept where its own products with a pool's scales are finite, so
// that a product of 0 scores 0; a score that this bounds lies far past its cap (products above 1e-19).
inline float scale_over_cap(float sm_scale, float softcap) {
  return fminf(fmaxf(sm_scale / softcap, -1e20f), 1e20f);
}

// A slope in the log2 domain, kept where its product with any distance is finite: a key that is
// infinitely far below every other has weight 0 all the same.
__device__ __forceinline__ float slope_log2(float slope) {
  return fminf(fmaxf(slope * kLog2e, -1e25f), 1e25f);
}

}  // namespace pa
