// pa_attend_scored.cuh -- pa_extend_scored: the kernels of pa_attend.cuh with scores that a tanh caps,
// that fall with distance, or with a prefix whose tokens all see one another.
#pragma once

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
    p.c = fmaxf(fabsf(x.sm_scale / x.score.softcap), 1e-30f);
    p.cap2 = x.score.softcap * kLog2e;
    const float tanh[6] = {kTanh0, kTanh1, kTanh2, kTanh3, kTanh4, kTanh5};
    for (int i = 0; i < 6; ++i) p.near[i] = make_float2(p.cap2 * tanh[i], p.cap2 * tanh[i]);
  }
  CUtensorMap maps[3];
  if (!make_maps(x.s, plan, x.q, x.T, x.k_pool, x.v_pool, maps)) return PA_ERR_CUDA;
  return launch_kind<kScore>(x.s, plan, p, maps, x.stream);
}

}  // namespace pa
