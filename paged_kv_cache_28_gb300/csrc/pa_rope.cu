// pa_rope.cu -- the position rotation of a call's queries and keys, and the slot-mapped write
// of the rotated keys and the values (pa_rope_and_cache, pa_rope_axes_and_cache), in one pass.
//
// Pair j of a head's first `rotary_dim` channels turns by the angle whose cosine and sine the
// caller's table holds for the token's position:
//     a' = a cos - b sin,   b' = b cos + a sin
// in fp32 with each product and sum rounded (no fused multiply-add, so that the bits are those
// of the written formula), rounded once to bf16.  The rotated keys and the values then go to
// the cache as pa_reshape_and_cache writes them.
//
// Nothing here is reused but the table row of a token, so the bf16 kernel is bound by HBM: each
// vector is read once and written once.  16,384 tokens of 64 query and 8 KV heads take 109 us, 92 %
// of the measured copy bandwidth (119 us before the first vectors' loads went ahead of the token's
// slot and angles).  9,485 tokens into an E4M3 cache take 111 us, 50 % of it: the writers alone take
// 74, the queries (by the bf16 kernel, with four KV heads) 60, and beside each other they hide
// little.  What bounds the writers by themselves has not been measured.
// 261 us -> 155 with quotients by the reciprocal and the block index by a shift, 118 with the
// tokens of a job in a loop and the writers' CTAs among the queries', 111 with a CTA's eight tokens
// looked at by a warp each.
#include <algorithm>
#include <type_traits>

#include "pa_codec.cuh"
#include "pa_common.cuh"
#include "pa_extend.h"
#include "pa_internal.h"

namespace pa {
namespace {

struct RopeParams {
  const float *cos_sin;
  const int32_t *positions;
  const int64_t *slots;
  uint16_t *q_out;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  uint8_t *k_pool, *v_pool;
  float *k_scale, *v_scale;
  int32_t *err;
  int T, Hq, Hkv, r, num_positions, bs, nblocks;
  int num_axes;            // several axes: positions [num_axes, T], and pair j's axis in bits 2 j ..
  uint32_t axes[4];
};

// How many axes the positions have, and whether pairs 4 i .. 4 i + 3 share theirs, so that their
// angles lie side by side in the table: a kernel for each.  8,726 tokens into an E4M3 cache take 102 us
// with one axis, 115 with three in fours, 130 with three in turn.  The bf16 kernels, which load
// each angle for several heads, take them pair by pair (16,384 tokens: 104 us with one axis, 109 to
// 113 with three either way).
constexpr int kOneAxis = 0, kInFours = 1, kAnyPair = 2;

// The rows of the table that a token's pairs turn by: one, or one for each axis.
struct AxisRows {
  int pos[PA_MAX_AXES];
};
template <int kAxes>
using Place = std::conditional_t<kAxes != kOneAxis, AxisRows, int>;

template <int kAxes>
__device__ __forceinline__ Place<kAxes> load_place(const RopeParams &p, int t) {
  if constexpr (kAxes != kOneAxis) {
    AxisRows x;
#pragma unroll
    for (int a = 0; a < PA_MAX_AXES; ++a)
      x.pos[a] = p.positions[static_cast<int64_t>(a < p.num_axes ? a : 0) * p.T + t];
    return x;
  } else {
    return p.positions[t];
  }
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int pair) {
  return (p.axes[pair >> 4] >> (2 * (pair & 15))) & 3;
}

// (a, b) turned by (c, s)
__device__ __forceinline__ float2 turn(float a, float b, float c, float s) {
  return make_float2(__fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s)),
                     __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s)));
}

// Whether a token is written: a slot in the pool and its positions in the table.
__device__ __forceinline__ bool in_table(const RopeParams &p, int pos) {
  return pos >= 0 && pos < p.num_positions;
}
__device__ __forceinline__ bool in_table(const RopeParams &p, const AxisRows &at) {
  bool in = true;
#pragma unroll
  for (int pos : at.pos) in = in && in_table(p, pos);
  return in;
}
template <class At>
__device__ __forceinline__ bool token_ok(const RopeParams &p, int64_t slot, const At &at, bool report) {
  if (slot < 0) return false;                            // padding
  int bits = 0;
  if (slot >= static_cast<int64_t>(p.nblocks) * p.bs) bits |= PA_DEVERR_SLOT;
  if (!in_table(p, at)) bits |= PA_DEVERR_POSITION;
  if (bits && report) set_err(p.err, bits);
  return bits == 0;
}

// One thread's share of a head: 16 channels as two 16-byte chunks that hold eight whole pairs
// (channels j and j + r / 2, or neighbours), and their angles.
struct Item {
  bool rotates;
  float cos[8], sin[8];
};

template <int kAxes>
__device__ __forceinline__ void load_item(const RopeParams &p, int item, int pos, Item &x) {
  x.rotates = item < p.r / 16;
  if (!x.rotates) return;
  const float4 *row =
      reinterpret_cast<const float4 *>(p.cos_sin + static_cast<int64_t>(pos) * p.r + 8 * item);
  const float4 *sin_row = row + p.r / 8;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    *reinterpret_cast<float4 *>(x.cos + 4 * i) = __ldg(row + i);
    *reinterpret_cast<float4 *>(x.sin + 4 * i) = __ldg(sin_row + i);
  }
}
// The table row of axis a.
__device__ __forceinline__ int row_of(const AxisRows &at, int a) {
  int pos = at.pos[0];
#pragma unroll
  for (int i = 1; i < PA_MAX_AXES; ++i) pos = a == i ? at.pos[i] : pos;
  return pos;
}
template <int kAxes>
__device__ __forceinline__ void load_item(const RopeParams &p, int item, const AxisRows &at, Item &x) {
  x.rotates = item < p.r / 16;
  if (!x.rotates) return;
  const uint32_t axes = p.axes[item >> 1] >> (16 * (item & 1));        // of the eight pairs, two bits each
  constexpr int N = kAxes == kInFours ? 4 : 1;
#pragma unroll
  for (int e = 0; e < 8; e += N) {
    const float *row = p.cos_sin + static_cast<int64_t>(row_of(at, axes >> (2 * e) & 3)) * p.r + 8 * item + e;
    if constexpr (N == 4) {
      *reinterpret_cast<float4 *>(x.cos + e) = __ldg(reinterpret_cast<const float4 *>(row));
      *reinterpret_cast<float4 *>(x.sin + e) = __ldg(reinterpret_cast<const float4 *>(row + p.r / 2));
    } else {
      x.cos[e] = __ldg(row);
      x.sin[e] = __ldg(row + p.r / 2);
    }
  }
}

template <bool kInterleaved>
__device__ __forceinline__ void rotate_item(const Item &x, uint4 &a, uint4 &b) {
  uint32_t *u = reinterpret_cast<uint32_t *>(&a), *w = reinterpret_cast<uint32_t *>(&b);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      const float2 y = turn(bf16_lo(u[i]), bf16_hi(u[i]), x.cos[i], x.sin[i]);
      const float2 z = turn(bf16_lo(w[i]), bf16_hi(w[i]), x.cos[4 + i], x.sin[4 + i]);
      u[i] = pack_bf16(y.x, y.y);
      w[i] = pack_bf16(z.x, z.y);
    } else {
      const float2 y = turn(bf16_lo(u[i]), bf16_lo(w[i]), x.cos[2 * i], x.sin[2 * i]);
      const float2 z = turn(bf16_hi(u[i]), bf16_hi(w[i]), x.cos[2 * i + 1], x.sin[2 * i + 1]);
      u[i] = pack_bf16(y.x, z.x);
      w[i] = pack_bf16(y.y, z.y);
    }
  }
}

// Heads first, first + step, ... < last of token t, counted through the queries, then (bf16
// pools) the keys and the values; this thread's item of each.  Four heads' loads are in flight
// at once, the first four's before the token's slot, position and angles are there.
template <int D, bool kInterleaved, int kAxes>
__device__ __forceinline__ void rope_heads(const RopeParams &p, int t, int item, int first, int step,
                                           int last, bool report) {
  constexpr int U = 4;
  const bool split = !kInterleaved && item < p.r / 16;
  const int c0 = split ? 8 * item : 16 * item, c1 = split ? p.r / 2 + 8 * item : 16 * item + 8;
  uint4 a[U], b[U];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * step;
      if (h >= last) break;
      const uint16_t *src = h < p.Hq ? p.q + t * p.q_stride + h * D
                            : h < p.Hq + p.Hkv ? p.k + t * p.k_stride + (h - p.Hq) * D
                                               : p.v + t * p.v_stride + (h - p.Hq - p.Hkv) * D;
      a[i] = *reinterpret_cast<const uint4 *>(src + c0);
      b[i] = *reinterpret_cast<const uint4 *>(src + c1);
    }
  };
  load(first);
  const int64_t slot = p.slots[t];
  const Place<kAxes> at = load_place<kAxes>(p, t);
  if (!token_ok(p, slot, at, report)) return;
  Item x;
  load_item<kAxes>(p, item, at, x);
  for (int h0 = first; h0 < last; h0 += step * U) {
    if (h0 > first) load(h0);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * step;
      if (h >= last) break;
      if (x.rotates && h < p.Hq + p.Hkv) rotate_item<kInterleaved>(x, a[i], b[i]);
      uint16_t *dst =
          h < p.Hq ? p.q_out + (static_cast<int64_t>(t) * p.Hq + h) * D
          : h < p.Hq + p.Hkv
              ? reinterpret_cast<uint16_t *>(p.k_pool) + (slot * p.Hkv + h - p.Hq) * D
              : reinterpret_cast<uint16_t *>(p.v_pool) + (slot * p.Hkv + h - p.Hq - p.Hkv) * D;
      *reinterpret_cast<uint4 *>(dst + c0) = a[i];
      *reinterpret_cast<uint4 *>(dst + c1) = b[i];
    }
  }
}

// The queries alone: heads first, first + step, ... of token t (D = 128), two at a time.
template <bool kInterleaved, int kAxes>
__device__ __forceinline__ void rope_queries(const RopeParams &p, int t, int item, int first, int step) {
  constexpr int D = 128, U = 2;
  const bool split = !kInterleaved && item < p.r / 16;
  const int c0 = split ? 8 * item : 16 * item, c1 = split ? p.r / 2 + 8 * item : 16 * item + 8;
  const uint16_t *src = p.q + t * p.q_stride + first * D + c0;
  uint16_t *dst = p.q_out + (static_cast<int64_t>(t) * p.Hq + first) * D + c0;
  const int other = c1 - c0;
  uint4 a[U], b[U];
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i * step < p.Hq) {
        a[i] = *reinterpret_cast<const uint4 *>(src + i * step * D);
        b[i] = *reinterpret_cast<const uint4 *>(src + i * step * D + other);
      }
  };
  load(first);
  const int64_t slot = p.slots[t];
  const Place<kAxes> at = load_place<kAxes>(p, t);
  if (!token_ok(p, slot, at, false)) return;
  Item x;
  load_item<kAxes>(p, item, at, x);
#pragma unroll 1
  for (int h = first; h < p.Hq; h += U * step) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (h + i * step < p.Hq) {
        if (x.rotates) rotate_item<kInterleaved>(x, a[i], b[i]);
        *reinterpret_cast<uint4 *>(dst + i * step * D) = a[i];
        *reinterpret_cast<uint4 *>(dst + i * step * D + other) = b[i];
      }
    src += U * step * D;
    dst += U * step * D;
    if (h + U * step < p.Hq) load(h + U * step);
  }
}

// BF16 pools: blockIdx.x is the token; blockIdx.y a share of its heads.  Six CTAs an SM (80 registers)
// keep the memory busiest: 112, 111, 109, 136 us for 16,384 tokens with 95 registers, 5, 6 and 8 CTAs.
template <int D, bool kInterleaved, int kAxes>
__global__ void __launch_bounds__(128, 6) rope_bf16_kernel(const RopeParams p) {
  pdl_trigger();
  pdl_wait();
  constexpr int kItems = D / 16, kHeads = 128 / kItems;
  rope_heads<D, kInterleaved, kAxes>(p, blockIdx.x, threadIdx.x % kItems,
                                     (p.q ? 0 : p.Hq) + blockIdx.y * kHeads + threadIdx.x / kItems,
                                     gridDim.y * kHeads, p.Hq + 2 * p.Hkv,
                                     threadIdx.x == 0 && blockIdx.y == 0);
}

// Quantised pools (D = 128).  `cache_ctas` CTAs write the cache, a share of `tokens` tokens each; as in
// pa_reshape_and_cache, the first token of the call in a block (its leader) stands for every
// token of the call in that block, applied in token order.  A warp takes (KV head, K or V) jobs,
// a lane four consecutive channels.  The codes of a job's rows stay in shared memory while its
// tokens are applied, so a token that raises the scale costs no trip to the pool, and each row
// is written once.  The other CTAs rotate the queries of a token each.
//
// The scale is absmax times the fp32 reciprocal of the largest code (pa_reshape_and_cache
// divides: the two differ by one unit in the last place at most); codes are x / scale, rounded,
// in both.
template <class Codec, bool kInterleaved, int kAxes>
__global__ void __launch_bounds__(256, 3) rope_quant_kernel(const RopeParams p, int cache_ctas, int tokens,
                                                            int shares) {
  using Word = typename Codec::Word;
  constexpr int D = 128, kWarps = 8, kBatch = 8;
  extern __shared__ uint32_t smem[];                     // [kWarps][bs][32] words: a job's rows
  __shared__ int members[256];      // this chunk's tokens of the block, in token order
  __shared__ int member_off[256];
  __shared__ int warp_count[kWarps];
  __shared__ uint2 vectors[kWarps][kBatch][32];
  __shared__ uint32_t offsets_seen;
  __shared__ bool first_of_run[kWarps];
  pdl_trigger();
  pdl_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // the two kinds of CTA alternate, so that the writers' arithmetic runs beside the queries' traffic
  const int period = gridDim.x / cache_ctas, writer = blockIdx.x / period;
  if (blockIdx.x % period != 0 || writer >= cache_ctas) {
    const int t = blockIdx.x - min(writer + 1, cache_ctas);
    rope_queries<kInterleaved, kAxes>(p, t, tid % 8, tid / 8, 32);
    return;
  }
  const int nth = writer / shares, share = writer % shares;
  Word *codes = reinterpret_cast<Word *>(smem) + warp * p.bs * 32 + lane;    // row r: codes[32 r]
  // A token right after another of its block (a prompt's tokens fill their blocks in order) has
  // nothing to do; a warp looks at each of the CTA's.  The others look through the call: an earlier
  // token of the block leads it, and without a later one past the first 256 tokens one look is enough.
  auto same_block = [&](int u, int64_t o, int64_t blk0) {
    return o >= blk0 && o < blk0 + p.bs && token_ok(p, o, load_place<kAxes>(p, u), false);
  };
  if (warp < tokens && lane == 0) {
    const int t = nth * tokens + warp;
    bool first = false;
    if (t < p.T) {
      const int64_t slot = p.slots[t], before = t > 0 ? p.slots[t - 1] : -1;
      first = token_ok(p, slot, load_place<kAxes>(p, t), true) &&
              !(t > 0 && same_block(t - 1, before, slot & ~static_cast<int64_t>(p.bs - 1)));
    }
    first_of_run[warp] = first;
  }
  __syncthreads();
  for (int c = 0; c < tokens; ++c) {
    if (!first_of_run[c]) continue;
    const int t = nth * tokens + c;
    const int64_t slot = p.slots[t];
    const int64_t blk = slot >> (p.bs == 16 ? 4 : 5), blk0 = blk * p.bs;
    auto in_block = [&](int u, int64_t o) { return same_block(u, o, blk0); };
    int earlier = 0, later = 0;
    bool look = true;
    if constexpr (kAxes != kOneAxis) {
      // (a token of the block by its slot alone; with several positions each the look at them would
      // be most of the loop)
      int any = 0;
#pragma unroll 8
      for (int u = tid; u < p.T; u += 256) {
        const int64_t o = p.slots[u];
        any |= o >= blk0 && o < blk0 + p.bs && (u < t - 1 || u >= t + 256);
      }
      look = __syncthreads_or(any);
    }
    if (look) {
#pragma unroll 8
      for (int u = tid; u < t - 1; u += 256) earlier |= in_block(u, p.slots[u]);
#pragma unroll 8
      for (int u = t + 256 + tid; u < p.T; u += 256) later |= in_block(u, p.slots[u]);
    }
    const int others = __syncthreads_or(earlier | later);
    if (others && __syncthreads_or(earlier)) continue;
    const int end = others ? p.T : min(p.T, t + 256);
    if (tid == 0) offsets_seen = 0u;
    for (int c0 = t; c0 < end; c0 += 256) {
      // the chunk's tokens of this block, in token order (ballot compaction)
      const int u = c0 + tid;
      const int64_t o = u < p.T ? p.slots[u] : -1;
      const bool mine = u < p.T && in_block(u, o);
      const uint32_t ballot = __ballot_sync(0xffffffffu, mine);
      if (lane == 0) warp_count[warp] = __popc(ballot);
      __syncthreads();
      int before = 0, n = 0;
      for (int w = 0; w < kWarps; ++w) {
        before += w < warp ? warp_count[w] : 0;
        n += warp_count[w];
      }
      if (mine) {
        const int i = before + __popc(ballot & ((1u << lane) - 1u));
        const int off = static_cast<int>(o - blk0);
        members[i] = u;
        member_off[i] = off;
        // a second token for one slot: applied after the first, and reported
        if (atomicOr(&offsets_seen, 1u << off) & (1u << off)) set_err(p.err, PA_DEVERR_FP8_CONFLICT);
      }
      __syncthreads();
      for (int job = share * kWarps + warp; job < 2 * p.Hkv; job += shares * kWarps) {
        const int h = job >> 1;
        const bool is_v = job & 1;
        uint8_t *pool = is_v ? p.v_pool : p.k_pool;
        float *scale = (is_v ? p.v_scale : p.k_scale) + blk * p.Hkv + h;
        const uint16_t *src = (is_v ? p.v : p.k) + h * D + lane * 4;
        const int64_t stride = is_v ? p.v_stride : p.k_stride;
        Word *const rows = reinterpret_cast<Word *>(
            pool + (blk0 * p.Hkv + h) * int64_t(Codec::kRowBytes) + lane * sizeof(Word));
        const int pitch = p.Hkv * (Codec::kRowBytes / int(sizeof(Word)));     // words to the next row
        // the lane's own angles: its four channels' pairs lie r / 8 lanes away, or it has two pairs
        const bool turns = !is_v && lane * 4 < p.r;
        const bool upper = !kInterleaved && lane * 4 >= p.r / 2;
        const int j = kInterleaved ? lane * 2 : lane * 4 - (upper ? p.r / 2 : 0);
        const int peer = (upper ? lane - p.r / 8 : lane + p.r / 8) & 31;
        // the positions of the lane's first pair
        const int32_t *positions = p.positions;
        if constexpr (kAxes != kOneAxis)
          if (turns) positions += static_cast<int64_t>(axis_of(p, j)) * p.T;
        float s = *scale;
        ByReciprocal over(1.f);
        uint32_t held = 0;                               // rows whose codes are in shared memory
        for (int i0 = 0; i0 < n; i0 += kBatch) {
          // a batch's vectors, rotated and rounded as the cache takes them, and their maxima
          uint2 x[kBatch];
          float amax[kBatch];
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (i0 + i < n) x[i] = *reinterpret_cast<const uint2 *>(src + members[i0 + i] * stride);
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (i0 + i >= n) break;
            if (!is_v) {
              const float v[4] = {bf16_lo(x[i].x), bf16_hi(x[i].x), bf16_lo(x[i].y), bf16_hi(x[i].y)};
              const float *row = p.cos_sin + static_cast<int64_t>(positions[members[i0 + i]]) * p.r + j;
              // the same for pair j + e, where pairs have axes of their own
              [[maybe_unused]] auto other_row = [&](int e) {
                const int64_t axis = axis_of(p, j + e);
                return p.cos_sin + static_cast<int64_t>(p.positions[axis * p.T + members[i0 + i]]) * p.r + j + e;
              };
              if constexpr (kInterleaved) {
                if (turns) {
                  float2 c, sn;
                  if constexpr (kAxes != kAnyPair) {
                    c = __ldg(reinterpret_cast<const float2 *>(row));
                    sn = __ldg(reinterpret_cast<const float2 *>(row + p.r / 2));
                  } else {
                    const float *next = other_row(1);
                    c = make_float2(__ldg(row), __ldg(next));
                    sn = make_float2(__ldg(row + p.r / 2), __ldg(next + p.r / 2));
                  }
                  const float2 y = turn(v[0], v[1], c.x, sn.x), z = turn(v[2], v[3], c.y, sn.y);
                  x[i] = make_uint2(pack_bf16(y.x, y.y), pack_bf16(z.x, z.y));
                }
              } else {
                const uint32_t w0 = __shfl_sync(0xffffffffu, x[i].x, peer);
                const uint32_t w1 = __shfl_sync(0xffffffffu, x[i].y, peer);
                const float w[4] = {bf16_lo(w0), bf16_hi(w0), bf16_lo(w1), bf16_hi(w1)};
                if (turns) {
                  alignas(16) float cc[4], ss[4];
                  if constexpr (kAxes != kAnyPair) {
                    const float4 c = __ldg(reinterpret_cast<const float4 *>(row));
                    const float4 sn = __ldg(reinterpret_cast<const float4 *>(row + p.r / 2));
                    cc[0] = c.x, cc[1] = c.y, cc[2] = c.z, cc[3] = c.w;
                    ss[0] = sn.x, ss[1] = sn.y, ss[2] = sn.z, ss[3] = sn.w;
                  } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                      const float *own = other_row(e);
                      cc[e] = __ldg(own);
                      ss[e] = __ldg(own + p.r / 2);
                    }
                  }
                  float y[4];                            // a cos - b sin, or b cos + a sin
#pragma unroll
                  for (int e = 0; e < 4; ++e)
                    y[e] = __fadd_rn(__fmul_rn(v[e], cc[e]), __fmul_rn(w[e], upper ? ss[e] : -ss[e]));
                  x[i] = make_uint2(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]));
                }
              }
            }
            // The largest magnitude by integers, which order alike.  A NaN is left out, as by fmaxf in
            // pa_reshape_and_cache: it costs its own channel, not its block's scale.  A vector of
            // nothing but NaN has -1 as its largest, a NaN's bits.
            const float most = fmaxf(fmaxf(fabsf(bf16_lo(x[i].x)), fabsf(bf16_hi(x[i].x))),
                                     fmaxf(fabsf(bf16_lo(x[i].y)), fabsf(bf16_hi(x[i].y))));
            const int key = isnan(most) ? -1 : __float_as_int(most);
            amax[i] = __int_as_float(__reduce_max_sync(0xffffffffu, key));
          }
          // lane i: the scale that the batch's token i asks for.  The vectors wait in shared memory,
          // so that the tokens can be taken in a loop: unrolled, this part overflows the
          // instruction cache (155 us for 9,485 tokens, against 118 when it was made a loop).
          float want = 0.f;
#pragma unroll
          for (int i = 0; i < kBatch; ++i) {
            if (lane == i) want = __fmul_rn(amax[i], Codec::kPerCode);
            if (i0 + i < n) vectors[warp][i][lane] = x[i];
          }
#pragma unroll 1
          for (int i = 0; i < kBatch && i0 + i < n; ++i) {
            const int off = member_off[i0 + i];
            const float cand = __shfl_sync(0xffffffffu, want, i);
            const float s_new = (off == 0 || cand > s) ? cand : s;
            if (s_new != s || i0 + i == 0) over = ByReciprocal(s_new);
            const bool fits = over.fits();
            if (off > 0 && s_new > s) {
              const uint32_t below = (1u << off) - 1u;
              if ((held & below) != below)
                for (int r = 0; r < off; ++r)
                  if (!(held >> r & 1)) codes[32 * r] = rows[r * pitch];
              held |= below;
              if (fits) {
#pragma unroll 2
                for (int r = 0; r < off; ++r) codes[32 * r] = Codec::reencode_over(codes[32 * r], s, over);
              } else {
#pragma unroll 1
                for (int r = 0; r < off; ++r) codes[32 * r] = Codec::reencode(codes[32 * r], s, s_new);
              }
            }
            const uint2 y = vectors[warp][i][lane];
            const float v[4] = {bf16_lo(y.x), bf16_hi(y.x), bf16_lo(y.y), bf16_hi(y.y)};
            codes[32 * off] = fits ? Codec::encode_over(v, over) : Codec::encode(v, s_new);
            held |= 1u << off;
            s = s_new;
          }
        }
        for (uint32_t left = held; left; left &= left - 1) {
          const int r = __ffs(left) - 1;
          rows[r * pitch] = codes[32 * r];
        }
        if (lane == 0) *scale = s;
      }
      __syncthreads();   // the member lists and the scales are reused by the next chunk
    }
  }
}

template <int D, bool I, int A>
cudaError_t launch_bf16(const RopeParams &p, cudaStream_t stream) {
  // few tokens: their heads go over several CTAs, about two per SM
  constexpr int kHeads = 128 / (D / 16);
  const int heads = p.Hq + 2 * p.Hkv;
  const int shares = std::max(1, std::min((heads + kHeads - 1) / kHeads, 304 / p.T));
  return launch_pdl(rope_bf16_kernel<D, I, A>, dim3(p.T, shares), dim3(128), 0, stream, p);
}

template <class Codec, bool I, int A>
cudaError_t launch_quant(const RopeParams &p, cudaStream_t stream) {
  // a prompt's tokens mostly leave at once, so a CTA looks at several; a batch's stay
  const int tokens = p.T >= 2048 ? 8 : 1;
  // few tokens: their jobs go over several CTAs, each of which finds its block's tokens
  const int shares = p.T >= 1024 ? 1 : (2 * p.Hkv + 7) / 8;
  const int cache_ctas = (p.T + tokens - 1) / tokens * shares;
  const size_t smem = 8 * 32 * sizeof(typename Codec::Word) * p.bs;
  const cudaError_t e = cudaFuncSetAttribute(rope_quant_kernel<Codec, I, A>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, 32 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_quant_kernel<Codec, I, A>, dim3(cache_ctas + (p.q ? p.T : 0)), dim3(256), smem,
                    stream, p, cache_ctas, tokens, shares);
}

template <bool I, int A>
cudaError_t launch_kind(const pa_shape &s, const RopeParams &p, cudaStream_t stream) {
  if (s.kv_dtype == PA_KV_FP8_E4M3) return launch_quant<Fp8Codec, I, A>(p, stream);
  if (s.kv_dtype == PA_KV_INT4) return launch_quant<Int4Codec, I, A>(p, stream);
  constexpr int B = A == kOneAxis ? kOneAxis : kAnyPair;
  return s.D == 128 ? launch_bf16<128, I, B>(p, stream) : launch_bf16<64, I, B>(p, stream);
}

}  // namespace

pa_status run_rope_and_cache(const pa_shape &s, const pa_rope &rope, const pa_rope_axes *axes,
                             const float *cos_sin,
                             const int32_t *positions, void *q_out, const void *q,
                             const void *k_new, const void *v_new, void *k_pool, void *v_pool,
                             float *k_scale, float *v_scale, const int64_t *slot_mapping,
                             int32_t *err, cudaStream_t stream) {
  RopeParams p{};
  p.cos_sin = cos_sin;
  p.positions = positions;
  p.slots = slot_mapping;
  p.q_out = static_cast<uint16_t *>(q_out);
  p.q = static_cast<const uint16_t *>(q);
  p.k = static_cast<const uint16_t *>(k_new);
  p.v = static_cast<const uint16_t *>(v_new);
  p.q_stride = rope.q_stride ? rope.q_stride : static_cast<int64_t>(s.Hq) * s.D;
  p.k_stride = rope.k_stride ? rope.k_stride : static_cast<int64_t>(s.Hkv) * s.D;
  p.v_stride = rope.v_stride ? rope.v_stride : static_cast<int64_t>(s.Hkv) * s.D;
  p.k_pool = static_cast<uint8_t *>(k_pool);
  p.v_pool = static_cast<uint8_t *>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = err;
  p.T = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.r = rope.rotary_dim;
  p.num_positions = rope.num_positions;
  p.bs = s.block_size;
  p.nblocks = s.nblocks;
  const bool i = rope.interleaved;
  cudaError_t e;
  if (axes) {
    bool in_fours = true;
    p.num_axes = axes->num_axes;
    for (int j = 0; j < rope.rotary_dim / 2; ++j) {
      p.axes[j / 16] |= static_cast<uint32_t>(axes->pair_axis[j]) << (2 * (j % 16));
      in_fours = in_fours && axes->pair_axis[j] == axes->pair_axis[j & ~3];
    }
    if (in_fours)
      e = i ? launch_kind<true, kInFours>(s, p, stream) : launch_kind<false, kInFours>(s, p, stream);
    else
      e = i ? launch_kind<true, kAnyPair>(s, p, stream) : launch_kind<false, kAnyPair>(s, p, stream);
  } else {
    e = i ? launch_kind<true, kOneAxis>(s, p, stream) : launch_kind<false, kOneAxis>(s, p, stream);
  }
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

}  // namespace pa
