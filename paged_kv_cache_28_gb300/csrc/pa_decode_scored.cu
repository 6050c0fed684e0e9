// pa_decode_scored.cu -- single-token decode attention with changed scores (pa_decode_scored).
//
//     a_t = sm_scale <q[b][h], K_b[t]>,  with a cap: a_t = cap tanh(a_t / cap),
//     a_t = a_t - slope_h (L - 1 - t),   out[b][h] = sum_t softmax_t(a_t) V_b[t]
//
// pa_decode's split decode and merge, with the scores changed where they leave the matrix product:
// a lane holds 4 or 8 scores of a 16-token tile, so that a cap costs it some ten instructions a score
// beside the 2 x 16 rows that the tile loads from HBM, which stay what bounds it.
#include "pa_decode.cuh"
#include "pa_extend.h"

namespace pa {
namespace {

constexpr bool kScored = true;    // what PA_DISPATCH instantiates

pa_status dispatch(const pa_shape &s, int heads, const Params &p, const CUtensorMap &mk,
                   const CUtensorMap &mv, cudaStream_t stream) {
  const int nt = (p.G + 7) / 8;
  const int kind = kind_of(s, heads);
  PA_DISPATCH_ALL(launch_segments, p, mk, mv, stream)
  return PA_ERR_UNSUPPORTED;
}

}  // namespace

pa_status run_decode_scored(const pa_shape &s, void *out, const void *q, const void *k_pool,
                            const void *v_pool, const float *k_scale, const float *v_scale,
                            const int32_t *bt, const int32_t *sl, int window, const pa_score &score,
                            float sm_scale, void *workspace, int num_splits, int32_t *err,
                            cudaStream_t stream) {
  const WorkspaceLayout w = splitkv_layout(s, num_splits);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int heads = heads_per_unit(s, nullptr);
  const pa_shape v = unit_view(s, heads);
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, k_pool, v, heads) || !make_pool_map(&mv, v_pool, v, heads))
    return PA_ERR_CUDA;
  Params p = make_params(v, static_cast<float *>(out), q, k_scale, v_scale, bt, sl, nullptr, sm_scale,
                         err);
  p.window = window;
  if (score.softcap > 0.f) {
    p.sl2 = sm_scale / score.softcap;
    p.cap2 = score.softcap * kLog2e;
  }
  p.slopes = score.slopes;
  p.prefix_out = reinterpret_cast<int32_t *>(ws + w.prefix);
  p.lse_part = reinterpret_cast<float *>(ws + w.lse);
  p.o_part = reinterpret_cast<float *>(ws + w.o_part);
  p.num_splits = num_splits;
  const pa_status st = dispatch(v, heads, p, mk, mv, stream);
  return st == PA_OK ? launch_merge(s, static_cast<uint16_t *>(out), workspace, num_splits, stream) : st;
}

}  // namespace pa
