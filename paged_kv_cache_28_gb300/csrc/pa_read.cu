// pa_read.cu -- cached rows as dense bf16 tensors (pa_read_cache).
//
//     out[offsets[b] + i][h][:] = bf16(code * scale[block][h]),   block of position starts[b] + i
//
// (bf16 pools: the row itself.)  One pass, each byte read once and written once, so HBM bounds it;
// a CTA takes consecutive rows, whose places it finds first (a warp looks through the offsets 32 at a
// time), and then every thread has the same 16 channels of four rows on their way at once.
#include <algorithm>

#include "pa_common.cuh"
#include "pa_extend.h"
#include "pa_internal.h"

namespace pa {
namespace {

struct ReadParams {
  uint16_t *out[2];                     // K's and V's, or one of them
  const uint8_t *pool[2];
  const float *scale[2];
  int tensors;
  const int32_t *offsets, *starts, *seq_lens, *block_tables;
  int32_t *err;
  int B, Hkv, T, bs, bs_log2, max_blocks, nblocks;
  int rows;                             // output rows of a CTA, at most kMaxRows
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
  const int block = p.block_tables[static_cast<int64_t>(b) * p.max_blocks + (pos >> p.bs_log2)];
  if (block < 0 || block >= p.nblocks) {
    set_err(err, PA_DEVERR_BLOCK_ID);
    return kZeros;
  }
  return block * p.bs + static_cast<int>(pos & (p.bs - 1));
}

// Whether row t is sequence b's, whose offsets neither fall nor leave the rows.
__device__ __forceinline__ bool has_row(const ReadParams &p, int b, int t) {
  const int q0 = p.offsets[b], q1 = p.offsets[b + 1];
  return q0 >= 0 && q0 <= t && t < q1 && q1 <= p.T;
}

// The last sequence whose first row is at most t (a warp, all lanes), where no offset falls: the bound
// moves by 32 looks at a time, so that 16,384 sequences take three loads.
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

// 16 channels as the pool holds them.
template <int KIND>
struct Raw {
  static constexpr int kBytes = KIND == PA_KV_BF16 ? 32 : KIND == PA_KV_FP8_E4M3 ? 16 : 8;
  uint32_t w[kBytes / 4];
  __device__ __forceinline__ void load(const uint8_t *src) {
    if constexpr (KIND == PA_KV_INT4) {
      *reinterpret_cast<uint2 *>(w) = __ldcs(reinterpret_cast<const uint2 *>(src));
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(w)[i] = __ldcs(reinterpret_cast<const uint4 *>(src) + i);
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (uint32_t &x : w) x = KIND == PA_KV_INT4 ? 0x88888888u : 0u;       // codes of 0
  }
  __device__ __forceinline__ void restore(float scale, uint32_t (&o)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if constexpr (KIND == PA_KV_BF16) {
        o[i] = w[i];
      } else if constexpr (KIND == PA_KV_FP8_E4M3) {
        const float2 v = e4m3x2_to_float2(w[i >> 1] >> (16 * (i & 1)));
        o[i] = pack_bf16(__fmul_rn(v.x, scale), __fmul_rn(v.y, scale));
      } else {
        const uint32_t c = w[i >> 2] >> (8 * (i & 3));
        o[i] = pack_bf16(__fmul_rn(static_cast<float>(static_cast<int>(c & 15u) - 8), scale),
                         __fmul_rn(static_cast<float>(static_cast<int>(c >> 4 & 15u) - 8), scale));
      }
    }
  }
};

template <int KIND, int D>
__global__ void __launch_bounds__(kThreads) read_kernel(const ReadParams p) {
  __shared__ int row_of[kMaxRows];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * p.rows;
  const int n = static_cast<int>(min(static_cast<int64_t>(p.rows), p.T - t0));
  if (blockIdx.x == 0)                                   // offsets that fall or leave the rows
    for (int b = tid; b < p.B; b += kThreads) {
      const int q0 = p.offsets[b], q1 = p.offsets[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > p.T) set_err(p.err, PA_DEVERR_QUERY);
    }
  bool lost = false;
  for (int r = warp; r < n; r += kThreads / 32) {
    const int t = static_cast<int>(t0) + r;
    const int b = find_sequence(p.offsets, p.B, t, lane);
    const bool mine = has_row(p, b, t);
    lost |= !mine;
    if (lane == 0) row_of[r] = mine ? pool_row(p, b, t, p.offsets[b], p.err) : kLeft;
  }
  if (__syncthreads_or(lost)) {                          // a row of no sequence, or the search was misled
    int falls = 0;
    for (int b = tid; b < p.B; b += kThreads) falls |= p.offsets[b + 1] < p.offsets[b];
    if (__syncthreads_or(falls)) {
      for (int r = warp; r < n; r += kThreads / 32) {
        if (row_of[r] != kLeft) continue;
        const int t = static_cast<int>(t0) + r;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
          const uint32_t found = __ballot_sync(0xffffffffu, b0 + lane < p.B && has_row(p, b0 + lane, t));
          if (!found) continue;
          const int b = b0 + __ffs(found) - 1;
          if (lane == 0) row_of[r] = pool_row(p, b, t, p.offsets[b], p.err);
          break;
        }
      }
      __syncthreads();
    }
  }
  constexpr int kPieces = D / 16, kBatch = 4;
  const int per_row = p.Hkv * kPieces;
  // a thread keeps to its piece of a row: piece, piece + kThreads, ... of wide rows
  const int step = max(1, kThreads / per_row);           // rows at a time
  const int r0 = tid / per_row;
  if (r0 >= step) return;
  for (int piece = tid - r0 * per_row; piece < per_row; piece += kThreads) {
    const int head = piece / kPieces;
    for (int rr = r0; rr < n; rr += kBatch * step) {
      // four rows of K and of V on their way at once
      Raw<KIND> raw[2][kBatch];
      float scale[2][kBatch];
      int row[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = rr + i * step;
        row[i] = r < n ? row_of[r] : kLeft;
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x >= p.tensors) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          scale[x][i] = 0.f;
          if (row[i] >= 0) {
            if constexpr (KIND != PA_KV_BF16)
              scale[x][i] = __ldg(p.scale[x] + static_cast<int64_t>(row[i] >> p.bs_log2) * p.Hkv + head);
            raw[x][i].load(p.pool[x] + (static_cast<int64_t>(row[i]) * per_row + piece) * Raw<KIND>::kBytes);
          } else {
            raw[x][i].clear();
          }
        }
      }
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (x >= p.tensors) break;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (row[i] == kLeft) continue;
          uint32_t o[8];
          raw[x][i].restore(scale[x][i], o);
          uint16_t *dst = p.out[x] + ((t0 + rr + i * step) * per_row + piece) * 16;
          if (p.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(o[0]),
                         "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7])
                         : "memory");
          } else {
            __stcs(reinterpret_cast<uint4 *>(dst), make_uint4(o[0], o[1], o[2], o[3]));
            __stcs(reinterpret_cast<uint4 *>(dst) + 1, make_uint4(o[4], o[5], o[6], o[7]));
          }
        }
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
  auto add = [&](void *out, const void *pool, const float *scale) {
    if (!out) return;
    p.out[p.tensors] = static_cast<uint16_t *>(out);
    p.pool[p.tensors] = static_cast<const uint8_t *>(pool);
    p.scale[p.tensors++] = scale;
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
  p.bs_log2 = s.block_size == 16 ? 4 : 5;
  p.max_blocks = s.max_blocks;
  p.nblocks = s.nblocks;
  p.wide = ((reinterpret_cast<uintptr_t>(k_out) | reinterpret_cast<uintptr_t>(v_out)) & 31u) == 0;
  // four rows a thread; fewer in small calls, so that there are about two CTAs an SM
  const int per_row = s.Hkv * s.D / 16, step = std::max(1, kThreads / per_row);
  p.rows = std::max(1, std::min({kMaxRows, 4 * step, T / 304}));
  const dim3 grid((T - 1) / p.rows + 1);
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
