// pa_decode_scored.cu -- single-token decode attention with changed scores (pa_decode_scored).
//
//     a_t = sm_scale <q[b][h], K_b[t]>,  with a cap: a_t = cap tanh(a_t / cap),
//     a_t = a_t - slope_h (L - 1 - t),   out[b][h] = sum_t softmax_t(a_t) V_b[t]
//
// pa_decode's split decode with the scores changed where they leave the matrix product: a lane holds
// 4 or 8 scores of a 16-token tile, and a cap costs it some ten instructions a score beside the rows
// that the tile loads.  HBM bounds bf16 and large E4M3 batches, restoring the codes 4-bit ones.
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

// Joins the pieces of query head blockIdx.x's unit: kWarps warps take every kWarps-th of them, a lane
// D / 32 channels, and meet in shared memory.  A long sequence of a small batch has tens of pieces,
// and their loads' latency is what this takes: nine windowed sequences of a 4-bit cache 44 -> 31 us
// with eight warps a head, against pa_decode's merge by a CTA per KV head.  Of 64 sequences most
// heads are finished already, and 4,096 CTAs of eight warps took 5 us to come and go.
template <int D, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) merge_scored_kernel(uint16_t *out, const int32_t *prefix,
                                                           const float *o_part, const float *lse_part,
                                                           int B, int Hq, int Hkv, int G, int num_splits) {
  constexpr int E = D / 32, kBatch = 4;
  __shared__ float top[kWarps], dens[kWarps], nums[kWarps][D];
  pdl_trigger();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / Hq, h = blockIdx.x - b * Hq, kvh = h / G;
  // the KV heads that the decode served at a time, and this head's row among theirs
  const int heads = prefix[B + 1] == 2 ? 2 : 1, unit = kvh / heads;
  const int row = h - unit * heads * G, rows = G * heads;
  const int start_b = prefix[b], nt = (prefix[b + 1] - start_b) / (Hkv / heads), total = prefix[B];
  const int W = max(1, (total + num_splits - 1) / num_splits);
  uint16_t *o = out + static_cast<size_t>(blockIdx.x) * D;
  if (nt == 0) {
    for (int i = threadIdx.x; i < D / 2; i += 32 * kWarps) reinterpret_cast<uint32_t *>(o)[i] = 0u;
    return;
  }
  const int start = start_b + unit * nt, p0 = start / W, p1 = (start + nt - 1) / W;
  if (p0 == p1) return;                                  // finished inside one segment
  float M = -INFINITY, den = 0.f, num[E] = {};
  for (int s0 = p0 + warp; s0 <= p1; s0 += kBatch * kWarps) {
    float l[kBatch], x[kBatch][E], most = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int s = s0 + i * kWarps;
      const size_t at = (static_cast<size_t>(s) * 2 + (s == p0 ? 1 : 0)) * rows + row;
      l[i] = s <= p1 ? __ldg(lse_part + at) : -INFINITY;
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = s <= p1 ? __ldg(o_part + at * D + 32 * e + lane) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) most = fmaxf(most, l[i]);
    const float r = M == -INFINITY ? 0.f : expf(M - most);
    M = most;
    den *= r;
#pragma unroll
    for (int e = 0; e < E; ++e) num[e] *= r;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float w = l[i] == -INFINITY ? 0.f : expf(l[i] - M);
      den += w;
#pragma unroll
      for (int e = 0; e < E; ++e) num[e] = fmaf(w, x[i][e], num[e]);
    }
  }
  if (lane == 0) {
    top[warp] = M;
    dens[warp] = den;
  }
#pragma unroll
  for (int e = 0; e < E; ++e) nums[warp][32 * e + lane] = num[e];
  __syncthreads();
  M = -INFINITY;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) M = fmaxf(M, top[w]);
  for (int i = threadIdx.x; i < D / 2; i += 32 * kWarps) {
    float2 sum = make_float2(0.f, 0.f);
    den = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      // a warp without a piece has nothing; a NaN's den is NaN, and comes through
      const float f = dens[w] == 0.f ? 0.f : expf(top[w] - M);
      den = fmaf(f, dens[w], den);
      sum.x = fmaf(f, nums[w][2 * i], sum.x);
      sum.y = fmaf(f, nums[w][2 * i + 1], sum.y);
    }
    reinterpret_cast<uint32_t *>(o)[i] = pack_bf16(sum.x / den, sum.y / den);
  }
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
    p.sl2 = scale_over_cap(sm_scale, score.softcap);
    p.cap2 = score.softcap * kLog2e;
  }
  p.slopes = score.slopes;
  p.prefix_out = reinterpret_cast<int32_t *>(ws + w.prefix);
  p.lse_part = reinterpret_cast<float *>(ws + w.lse);
  p.o_part = reinterpret_cast<float *>(ws + w.o_part);
  p.num_splits = num_splits;
  const pa_status st = dispatch(v, heads, p, mk, mv, stream);
  if (st != PA_OK) return st;
  const bool many = s.B * s.Hq >= 1024;
  auto merge = s.D == 128 ? (many ? merge_scored_kernel<128, 2> : merge_scored_kernel<128, 8>)
                          : (many ? merge_scored_kernel<64, 2> : merge_scored_kernel<64, 8>);
  return launch_pdl(merge, dim3(s.B * s.Hq), dim3(many ? 64 : 256), 0, stream, static_cast<uint16_t *>(out),
                    p.prefix_out, p.o_part, p.lse_part, s.B, s.Hq, s.Hkv, s.Hq / s.Hkv,
                    num_splits) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace pa
