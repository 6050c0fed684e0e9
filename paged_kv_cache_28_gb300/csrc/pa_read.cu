// pa_read.cu -- cached rows as dense bf16 tensors (pa_read_cache).
//
//     out[offsets[b] + i][h][:] = bf16(code * scale[block][h]),   block of position starts[b] + i
//
// (bf16 pools: the row itself.)  One pass, each byte read once and written once, so HBM bounds it;
// a CTA takes consecutive rows of K or of V, whose places it finds first (a warp looks through the
// offsets 32 at a time), and then every thread has four 32-byte pieces of rows on their way at once.
#include <algorithm>

#include "pa_common.cuh"
#include "pa_extend.h"
#include "pa_internal.h"

namespace pa {
namespace {

struct ReadParams {
  uint16_t *out[2];                     // K's and V's
  const uint8_t *pool[2];
  const float *scale[2];
  const int32_t *offsets, *starts, *seq_lens, *block_tables;
  int32_t *err;
  int B, Hkv, T, bs, max_blocks, nblocks;
  int rows;                             // output rows of a CTA
  bool wide;                            // the outputs are 32-byte aligned
};

constexpr int kThreads = 256, kMaxRows = 64;
constexpr int kLeft = -2, kZeros = -1;  // a row of no sequence; a row that reads zeros

// Sequence b's row t: its row in the pool, or kZeros.
__device__ __forceinline__ int pool_row(const ReadParams &p, int b, int t, int first, int32_t *err) {
  const int64_t pos = static_cast<int64_t>(p.starts ? p.starts[b] : 0) + (t - first);
  const int64_t held = static_cast<int64_t>(p.max_blocks) * p.bs;
  if (pos < 0 || pos >= p.seq_lens[b] || pos >= held) {
    set_err(err, PA_DEVERR_SEQ_LEN);
    return kZeros;
  }
  const int block = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + pos / p.bs];
  if (block < 0 || block >= p.nblocks) {
    set_err(err, PA_DEVERR_BLOCK_ID);
    return kZeros;
  }
  return block * p.bs + static_cast<int>(pos % p.bs);
}

// The last sequence whose first row is at most t (a warp, all lanes): the bound moves by 32 looks at
// a time, so that 16,384 sequences take three loads.
__device__ __forceinline__ int find_sequence(const int32_t *offsets, int B, int t, int lane) {
  int lo = 0, hi = B;                                    // offsets[lo] <= t, or lo = 0
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int at = lo + lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, at < hi && offsets[at] <= t);
    const int last = below ? 31 - __clz(below) : 0;
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

template <int KIND>
__device__ __forceinline__ void restore16(const uint8_t *src, float scale, uint32_t (&o)[8]) {
  if constexpr (KIND == PA_KV_BF16) {
    const uint4 a = reinterpret_cast<const uint4 *>(src)[0], b = reinterpret_cast<const uint4 *>(src)[1];
    o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
    o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
  } else if constexpr (KIND == PA_KV_FP8_E4M3) {
    const uint4 a = *reinterpret_cast<const uint4 *>(src);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = e4m3x2_to_float2(w[i >> 1] >> (16 * (i & 1)));
      o[i] = pack_bf16(__fmul_rn(v.x, scale), __fmul_rn(v.y, scale));
    }
  } else {
    const uint2 a = *reinterpret_cast<const uint2 *>(src);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c = (i < 4 ? a.x : a.y) >> (8 * (i & 3));
      o[i] = pack_bf16(__fmul_rn(static_cast<float>(static_cast<int>(c & 15u) - 8), scale),
                       __fmul_rn(static_cast<float>(static_cast<int>(c >> 4 & 15u) - 8), scale));
    }
  }
}

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  __shared__ int row_of[kMaxRows];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int which = blockIdx.y;                          // K or V
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - t0));
  int32_t *err = which == 0 ? p.err : nullptr;             // both have the same errors
  if (blockIdx.x == 0 && err)                            // offsets that fall or leave the rows
    for (int b = tid; b < p.B; b += kThreads) {
      const int q0 = p.offsets[b], q1 = p.offsets[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > p.T) set_err(err, PA_DEVERR_QUERY);
    }
  for (int r = warp; r < n; r += kThreads / 32) {
    const int t = static_cast<int>(t0) + r;
    const int b = find_sequence(p.offsets, p.B, t, lane);
    if (lane == 0) {
      const int first = p.offsets[b];
      row_of[r] = first >= 0 && first <= t && t < p.offsets[b + 1] ? pool_row(p, b, t, first, err) : kLeft;
    }
  }
  __syncthreads();
  constexpr int kBytes = KIND == PA_KV_BF16 ? 32 : KIND == PA_KV_FP8_E4M3 ? 16 : 8;   // of 16 channels
  constexpr int kPieces = D / 16, kBatch = 4;
  const int per_row = p.Hkv * kPieces;
  const int total = n * per_row;
  const uint8_t *pool = which ? p.pool[1] : p.pool[0];
  const float *scales = which ? p.scale[1] : p.scale[0];
  uint16_t *out = (which ? p.out[1] : p.out[0]) + t0 * per_row * 16;
  for (int c0 = tid; c0 < total; c0 += kBatch * kThreads) {
    uint32_t o[kBatch][8];
    bool keep[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int c = c0 + i * kThreads;
      const int row = c < total ? row_of[c / per_row] : kLeft;
      keep[i] = row != kLeft;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[i][e] = 0u;
      if (row < 0) continue;
      const int piece = c % per_row;
      float scale = 1.f;
      if constexpr (KIND != PA_KV_BF16)
        scale = __ldg(scales + static_cast<int64_t>(row / p.bs) * p.Hkv + piece / kPieces);
      restore16<KIND>(pool + (static_cast<int64_t>(row) * per_row + piece) * kBytes, scale, o[i]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (!keep[i]) continue;
      uint16_t *dst = out + static_cast<int64_t>(c0 + i * kThreads) * 16;
      if (p.wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[i][0]),
                     "r"(o[i][1]), "r"(o[i][2]), "r"(o[i][3]), "r"(o[i][4]), "r"(o[i][5]), "r"(o[i][6]),
                     "r"(o[i][7])
                     : "memory");
      } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(o[i][4], o[i][5], o[i][6], o[i][7]);
      }
    }
  }
}

}  // namespace

pa_status run_read_cache(const pa_shape &s, void *k_out, void *v_out, const void *k_pool,
                         const void *v_pool, const float *k_scale, const float *v_scale,
                         const int32_t *bt, const int32_t *sl, const int32_t *offsets, int T,
                         const int32_t *starts, int32_t *err, cudaStream_t stream) {
  ReadParams p{};
  int tensors = 0;
  auto add = [&](void *out, const void *pool, const float *scale) {
    if (!out) return;
    p.out[tensors] = static_cast<uint16_t *>(out);
    p.pool[tensors] = static_cast<const uint8_t *>(pool);
    p.scale[tensors++] = scale;
  };
  add(k_out, k_pool, k_scale);
  add(v_out, v_pool, v_scale);
  p.offsets = offsets;
  p.starts = starts;
  p.seq_lens = sl;
  p.block_tables = bt;
  p.err = err;
  p.B = s.B;
  p.Hkv = s.Hkv;
  p.T = T;
  p.bs = s.block_size;
  p.max_blocks = s.max_blocks;
  p.nblocks = s.nblocks;
  p.wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  // four pieces a thread
  const int per_row = s.Hkv * s.D / 16;
  p.rows = std::max(1, std::min(kMaxRows, 4 * kThreads / per_row));
  const dim3 grid((T + p.rows - 1) / p.rows, tensors);
  cudaError_t e;
  if (s.kv_dtype == PA_KV_FP8_E4M3)
    e = launch_pdl(read_kernel<PA_KV_FP8_E4M3, 128>, grid, dim3(kThreads), 0, stream, p);
  else if (s.kv_dtype == PA_KV_INT4)
    e = launch_pdl(read_kernel<PA_KV_INT4, 128>, grid, dim3(kThreads), 0, stream, p);
  else if (s.D == 128)
    e = launch_pdl(read_kernel<PA_KV_BF16, 128>, grid, dim3(kThreads), 0, stream, p);
  else
    e = launch_pdl(read_kernel<PA_KV_BF16, 64>, grid, dim3(kThreads), 0, stream, p);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
