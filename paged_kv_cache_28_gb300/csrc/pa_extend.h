// pa_extend.h -- host-side interfaces between the C ABI (pa_api.cu) and the kernels of the
// calls with several new tokens per sequence (pa_rope.cu, pa_attend.cu), with changed scores
// (pa_attend_scored.cuh, pa_decode_scored.cu) and of reading the cache back (pa_read.cu).  Arguments reaching these functions are already validated.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "pa.h"

namespace pa {

// pa_extend (causal) and pa_cross_attend; `sms`: SMs of the device, as the workspace was sized.
// 0 bytes: more work than a call takes.
size_t attend_workspace_bytes(const pa_shape &s, int T, int sms);
pa_status run_attend(const pa_shape &s, void *out, const void *q, const int32_t *offsets, int T,
                     const void *k_pool, const void *v_pool, const float *k_scale,
                     const float *v_scale, const int32_t *bt, const int32_t *sl, bool causal,
                     int window, float sm_scale, void *workspace, int sms, int32_t *err,
                     cudaStream_t stream);

// pa_extend_scored: causal, with a window and changed scores; the workspace is pa_extend's.
struct ScoredCall {
  const pa_shape &s;
  void *out;
  const void *q;
  const int32_t *offsets;
  int T;
  const void *k_pool, *v_pool;
  const float *k_scale, *v_scale;
  const int32_t *bt, *sl;
  int window;
  const pa_score &score;
  float sm_scale;
  void *workspace;
  int sms;
  int32_t *err;
  cudaStream_t stream;
};
// what changes the scores (a prefix alone: neither); a file each, which compile side by side
constexpr int kCap = 1, kBias = 2;
template <int kScore>
pa_status run_attend_scored(const ScoredCall &x);
pa_status run_decode_scored(const pa_shape &s, void *out, const void *q, const void *k_pool,
                            const void *v_pool, const float *k_scale, const float *v_scale,
                            const int32_t *bt, const int32_t *sl, int window, const pa_score &score,
                            float sm_scale, void *workspace, int num_splits, int32_t *err,
                            cudaStream_t stream);

// axes: which position each pair turns by (pa_rope_axes_and_cache), or null
pa_status run_rope_and_cache(const pa_shape &s, const pa_rope &rope, const pa_rope_axes *axes,
                             const float *cos_sin,
                             const int32_t *positions, void *q_out, const void *q,
                             const void *k_new, const void *v_new, void *k_pool, void *v_pool,
                             float *k_scale, float *v_scale, const int64_t *slot_mapping,
                             int32_t *err, cudaStream_t stream);

// k_out or v_out may be null
pa_status run_read_cache(const pa_shape &s, void *k_out, void *v_out, const void *k_pool,
                         const void *v_pool, const float *k_scale, const float *v_scale,
                         const int32_t *bt, const int32_t *sl, const int32_t *offsets, int T,
                         const int32_t *starts, int32_t *err, cudaStream_t stream);

}  // namespace pa
