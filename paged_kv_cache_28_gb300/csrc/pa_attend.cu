// pa_attend.cu -- pa_extend and pa_cross_attend: the kernels of pa_attend.cuh with plain scores.
#define PA_ATTEND_SCORED false
#include "pa_attend.cuh"

namespace pa {

size_t attend_workspace_bytes(const pa_shape &s, int T, int sms) {
  const Plan plan = make_plan(s, T, sms);
  // a worker counts its tiles in 32 bits (2^28 of them would take minutes)
  const int64_t units = (static_cast<int64_t>(T) / plan.tok + s.B) * s.Hkv;
  const int64_t tiles = static_cast<int64_t>(s.max_blocks) * s.block_size / kKeys + 4;
  return units * tiles / plan.workers < (int64_t(1) << 28) ? plan.total : 0;
}

pa_status run_attend(const pa_shape &s, void *out, const void *q, const int32_t *offsets, int T,
                     const void *k_pool, const void *v_pool, const float *k_scale,
                     const float *v_scale, const int32_t *bt, const int32_t *sl, bool causal,
                     int window, float sm_scale, void *workspace, int sms, int32_t *err,
                     cudaStream_t stream) {
  const Plan plan = make_plan(s, T, sms);
  const AttendParams p = make_params(s, plan, out, offsets, T, k_scale, v_scale, bt, sl, causal, window,
                                     sm_scale, workspace, err);
  CUtensorMap maps[3];
  if (!make_maps(s, plan, q, T, k_pool, v_pool, maps)) return PA_ERR_CUDA;
  return launch_kind<0>(s, plan, p, maps, stream);
}

}  // namespace pa
