// pa_attend_scored.cuh -- pa_extend_scored: the kernels of pa_attend.cuh with scores that a tanh caps,
// that fall with distance, or with a prefix whose tokens all see one another.
#pragma once

#include <cfloat>
#include <cmath>

#define PA_ATTEND_SCORED true
#include "pa_attend.cuh"

namespace pa {

template <int kScore>
pa_status run_attend_scored(const ScoredCall &x) {
  const Plan plan = make_plan(x.s, x.T, x.sms);
  AttendParams p = make_params(x.s, plan, x.out, x.offsets, x.T, x.k_scale, x.v_scale, x.bt, x.sl, true,
                               x.window, x.sm_scale, x.workspace, x.err);
  p.slopes = x.score.slopes;
  p.prefix_lens = x.score.prefix_lens;
  if (kScore & kCap) {
    // (0 with sm_scale 0, whatever the products)
    p.c = fabsf(scale_over_cap(x.sm_scale, x.score.softcap));
    p.cap2 = x.score.softcap * kLog2e;
    // tanh's coefficients; on bf16 pools with c^(2 i + 1) in them, as far as fp32 holds all of them: six
    // for c >= 2^-11 (heads of 128: caps up to 180), four for scores up to half the cap to 2^-16 (caps
    // up to 5,800), two for scores up to a fiftieth of it below.  Scores beyond, and all those of caps
    // below 3.5e-4 and of a c whose powers leave fp32 (with the usual scales: below 1e-15), go through
    // the exponential.
    const double c = x.s.kv_dtype == PA_KV_BF16 ? p.c : 1.0;
    const double six[6] = {kTanh0, kTanh1, kTanh2, kTanh3, kTanh4, kTanh5};
    const double four[6] = {kTanhHalf0, kTanhHalf1, kTanhHalf2, kTanhHalf3}, two[6] = {1.0, -1.0 / 3};
    auto fits = [&](const double *k) {                   // no coefficient that counts leaves fp32
      double power = p.cap2 * c;
      for (int i = 0; i < 6; ++i, power *= c * c)
        if (k[i] != 0.0 && !(fabs(k[i] * power) >= FLT_MIN && fabs(k[i] * power) <= FLT_MAX)) return false;
      return c <= 0x1p8;
    };
    const double *small = c >= 0x1p-16 && fits(four) ? four : two;
    const double *large = c >= 0x1p-11 && fits(six) ? six : small;
    p.reach4 = !fits(small) ? -1.f : small == four ? 0.5f : 0.02f;
    p.reach6 = large == six ? 1.f : p.reach4;
    double power = p.cap2 * c;
    for (int i = 0; i < 6; ++i, power *= c * c) {
      const float y = static_cast<float>(large[i] * power), z = static_cast<float>(small[i] * power);
      p.tanh6[i] = make_float2(y, y);
      if (i < 4) p.tanh4[i] = make_float2(z, z);
    }
  }
  CUtensorMap maps[3];
  if (!make_maps(x.s, plan, x.q, x.T, x.k_pool, x.v_pool, maps)) return PA_ERR_CUDA;
  return launch_kind<kScore>(x.s, plan, p, maps, x.stream);
}

}  // namespace pa
