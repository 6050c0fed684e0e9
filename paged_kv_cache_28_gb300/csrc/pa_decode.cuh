// pa_decode.cuh -- the paged decode's tile engine, its split (segment) kernel and merge, and the
// host helpers that launch them: for pa_decode.cu (the plain decodes) and pa_decode_scored.cu.
#pragma once

#include <cudaTypedefs.h>

#include <type_traits>

#include "pa_common.cuh"
#include "pa_internal.h"
#include "pa_score.cuh"

namespace pa {

// ----------------------------------------------------------------------------
// configuration
// ----------------------------------------------------------------------------

// Cached element kinds.
constexpr int kKindBf16 = 0;
constexpr int kKindFp8 = 1;   // E4M3 codes, one per byte
constexpr int kKindInt4 = 2;  // 4-bit codes, two per byte (offset binary)
// 4-bit codes with two adjacent KV heads per unit: their 64-byte rows sit side by
// side in the pool, so one 128-byte box per token feeds both and every fetched
// byte is used (a lone 64-byte row costs a 128-byte DRAM fetch); n-tile h serves
// the group of KV head 2 u + h.
constexpr int kKindInt4x2 = 3;
// E4M3 units of two adjacent KV heads, in the split decode: a token row holds both heads'
// 128-byte rows (two TMA boxes); n-tile h serves the group of KV head 2 u + h.  Per byte
// of codes, the tile bookkeeping (records, barrier waits, copy issue) is shared by two
// heads and each warp keeps twice the bytes in flight.  pa_decode without a workspace
// keeps one E4M3 head per unit: there the paired form's three CTAs per SM (against
// four) measured slower.
constexpr int kKindFp8x2 = 4;

// SCORED_: scores changed before their softmax, and a bf16 output (pa_decode_scored).
template <int D_, int NT_, int KIND_, bool SCORED_ = false>
struct Cfg {
  static constexpr int D = D_;
  static constexpr int NT = NT_;            // 8-head n-tiles (G <= 8 * NT)
  static constexpr int KIND = KIND_;
  static constexpr bool SCORED = SCORED_;
  static constexpr bool FP8 = KIND == kKindFp8 || KIND == kKindFp8x2;
  static constexpr bool INT4 = KIND == kKindInt4 || KIND == kKindInt4x2;
  static constexpr bool PAIRED = KIND == kKindInt4x2 || KIND == kKindFp8x2;
  static constexpr int HEADS = PAIRED ? 2 : 1;      // KV heads per unit
  static constexpr bool QUANT = KIND != kKindBf16;   // codes x per-(block, head) scale
  static constexpr int KS = D / 16;         // QK k-steps of 16 elements
  static constexpr int DT = D / 16;         // PV 16-row output tiles
  static constexpr int ROW = HEADS * (INT4 ? D / 2 : (FP8 ? D : 2 * D));  // bytes of a unit's row
  static constexpr int BOX_BYTES = ROW < 128 ? ROW : 128;        // TMA box width (swizzle span)
  static constexpr int BOXES = ROW / BOX_BYTES;                  // boxes per tile row
  static constexpr int BOX_X = BOX_BYTES / (KIND == kKindBf16 ? 2 : 1);  // box width in elements
  static constexpr int KV_BYTES = kTile * ROW;
  // Paired 4-bit units read a piece's query rows straight from global memory and keep
  // the Q^T fragments in a per-warp shared-memory area: no Q slot in the stages (a
  // quarter less shared memory) and 32 registers freed for the tile loop, which made
  // pa_decode on these pools 8 % faster.  Other kinds carry the query rows in the
  // stage that starts a piece and hold the fragments in registers.
  static constexpr bool QSMEM = PAIRED;
  static constexpr int Q_BYTES = QSMEM ? 0 : 8 * NT * D * 2;
  static constexpr int QF_BYTES = QSMEM ? NT * KS * 32 * 8 : 0;   // per warp: uint2 per lane
  static constexpr int STAGE_BYTES = 2 * KV_BYTES + Q_BYTES;
  static constexpr int STAGES = PAIRED ? 2 : (INT4 ? 4 : 2);
  static constexpr int WARPS = 4;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int META_BYTES = 32;     // int4 unit + k/v scale
  static constexpr int SMEM = 1024 + WARPS * (STAGES * (STAGE_BYTES + 8 + META_BYTES) + QF_BYTES);
  // CTAs per SM that shared memory allows (227 KB usable, 1 KB reserved per CTA, 4 KB
  // left for the split kernel's length scan); the register budget is held to it.
  // Paired 4-bit units stop at three: four would fit in shared memory, but their
  // 128-register budget spills and measured slower than three CTAs at up to 168.
  static constexpr int MIN_BLOCKS_RAW = (227 * 1024) / (SMEM + 1024 + 4096);
  static constexpr int MIN_BLOCKS =
      QSMEM ? 3 : (MIN_BLOCKS_RAW < 1 ? 1 : (MIN_BLOCKS_RAW > 4 ? 4 : MIN_BLOCKS_RAW));
  static_assert(STAGE_BYTES % 1024 == 0, "stages must keep 1024-byte alignment");
  static_assert(!PAIRED || (NT == 2 && D == 128), "paired heads: one n-tile per KV head");
  static_assert(KV_BYTES % 1024 == 0, "swizzled tiles must be 1024-byte aligned");
  static_assert(!QSMEM || PAIRED, "query rows from global memory: paired units only");
  // pa_decode's CTA merges its warps' accumulators in the stage area; their m and l go
  // after every per-warp area (mbarrier memory is never reused)
  static_assert(WARPS * 8 * NT * D * 4 <= WARPS * STAGES * STAGE_BYTES, "pair merge must fit");
  // after them: the CTA's folded m and l (cluster launches) and one cluster mbarrier
  static constexpr int PAIR_SMEM = SMEM + (2 * WARPS + 2) * 8 * NT * 4 + 16;
};

struct Params {
  float *out;
  const uint16_t *q;
  const float *k_scale;
  const float *v_scale;
  const int32_t *block_tables;
  const int32_t *seq_lens;
  const int32_t *shared_prefix_lens;   // optional L2 hint per sequence
  int window;                          // > 0: attend over the last `window` positions only
  int topk;                            // > 0: attend over the pages listed in sel only
  const int32_t *sel;                  // [B, Hkv, topk] chosen 16-token pages (ascending)
  const int32_t *casc_tiles;           // [B] shared tiles done by the cascade kernel, or null
  uint64_t casc_ws;                    // the cascade workspace address (0: none), for the merge
  int32_t *err;
  int B, Hq, Hkv, G, bs, nblocks, max_blocks;
  float sl2;  // sm_scale * log2(e); with a cap: sm_scale / cap
  float cap2; // scored: cap * log2(e), or 0
  const float *slopes;   // scored: [query heads], or null
  // split-KV
  int32_t *prefix_out;   // workspace copy of the tile prefix, read by the merge
  float *o_part;
  float *lse_part;
  int num_splits;        // segments (split workers)
  // pa_decode_splitkv: every piece goes to caller arrays parts_o [B, Hq, S, D] and
  // parts_lse [B, Hq, S] (S = parts_S slots per query head, unused slots -inf);
  // parts_S = 0: workspace mode (units finished in one segment go straight to out)
  int parts_S;
  float *parts_o;
  float *parts_lse;
};

// ----------------------------------------------------------------------------
// per-warp softmax state
// ----------------------------------------------------------------------------

// What changes the scores of a piece (scored): the cap, each head's slope and how far behind the
// query the tile's first token lies.
template <bool SCORED, int NT>
struct ScoreState {};
template <int NT>
struct ScoreState<true, NT> {
  float cap2, slope[NT][2];     // in the log2 domain
  int behind;
};

template <class C>
struct State : ScoreState<C::SCORED, C::NT> {
  float acc[C::NT][C::DT][4];   // O^T fragments (d x heads)
  float m[C::NT][2];            // running max, log2 domain, heads 2q, 2q+1 of each n-tile
  float l[C::NT][2];            // this thread's share of the running sum
  uint32_t qf[C::QSMEM ? 1 : C::NT][C::QSMEM ? 1 : C::KS][2]; // Q^T B-fragments (else in smem)
  float qshift;                 // quantised: 2^-k undoing the power-of-two scaling of q
  float vref[C::NT];            // quantised: V scale each n-tile's accumulator is expressed in
  float vinv[C::NT];            // 1 / vref, or 0 before the piece's first nonzero V scale

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][dt][i] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
      vref[nt] = 1.f;
      vinv[nt] = 0.f;
    }
    qshift = 1.f;
  }
};

// Output row (d) of accumulator element i of d-tile dt for this lane.
template <class C>
__device__ __forceinline__ int acc_d(int dt, int i, int lane) {
  if constexpr (C::INT4)   // d-tile (chunk c = dt/2, half dt%2): rows 4r + 2 half + {0, 1}
    return (dt >> 1) * 32 + 4 * (lane >> 2) + 2 * (dt & 1) + (i >> 1);
  else if constexpr (C::FP8)
    return dt * 16 + 2 * (lane >> 2) + (i >> 1);
  else
    return dt * 16 + (lane >> 2) + (i >> 1) * 8;
}

// Load the group's Q^T fragments from the stage's Q slot ([8*NT rows][D] bf16), or,
// with C::QSMEM, from the query rows in global memory into the warp's fragment area
// qfs (lane-private: each lane reads back only what it wrote).
template <class C>
__device__ __forceinline__ void load_q(State<C> &st, uint32_t qslot, const uint16_t *qslot_ptr,
                                       uint4 *qfs, int G, int lane) {
  if constexpr (!C::QUANT) {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < C::KS; ks += 2) {
        uint32_t r[4];
        const int g = nt * 8 + (lane & 7);
        const int chunk = ks * 2 + (lane >> 3);
        ldsm_x4(r, qslot + g * (C::D * 2) + chunk * 16);
        st.qf[nt][ks][0] = r[0];
        st.qf[nt][ks][1] = r[1];
        st.qf[nt][ks + 1][0] = r[2];
        st.qf[nt][ks + 1][1] = r[3];
      }
  } else {
    // K codes arrive in a permuted order (see process_tile).  FP8: k-step ks, lane
    // (r, q) pairs Q[g=r][16ks + 4q + {0,1}] and Q[g=r][16ks + 4q + {2,3}].  4-bit:
    // k-step ks = 2c + u pairs Q[r][b + 2u + {0,4}] and Q[r][b + 2u + {1,5}] with
    // b = 32c + 8q.  q is scaled by 2^k so that its largest magnitude sits just
    // below 2^15 (exact in f16).
    const int r = lane >> 2, qd = lane & 3;
    uint2 raw[C::NT][C::KS];
    float amax = 0.f;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        // 4-bit: the eight values b..b+7 of chunk c arrive as two uint2 (u = 0, 1)
        const int off = C::INT4 ? (ks >> 1) * 32 + qd * 8 + (ks & 1) * 4 : ks * 16 + qd * 4;
        const uint2 *src = reinterpret_cast<const uint2 *>(qslot_ptr + (nt * 8 + r) * C::D + off);
        if constexpr (C::QSMEM)   // global memory: rows past the group read as zeros
          raw[nt][ks] = nt * 8 + r < G ? __ldg(src) : make_uint2(0u, 0u);
        else
          raw[nt][ks] = *src;
        amax = fmaxf(amax, fmaxf(fmaxf(fabsf(bf16_lo(raw[nt][ks].x)), fabsf(bf16_hi(raw[nt][ks].x))),
                                 fmaxf(fabsf(bf16_lo(raw[nt][ks].y)), fabsf(bf16_hi(raw[nt][ks].y)))));
      }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    int k = 0;
    if (amax > 0.f) {
      const int e = ((__float_as_uint(amax) >> 23) & 0xFF) - 126;   // amax < 2^e
      k = min(max(15 - e, -100), 100);
    }
    const float up = __uint_as_float(static_cast<uint32_t>(127 + k) << 23);
    st.qshift = __uint_as_float(static_cast<uint32_t>(127 - k) << 23);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int ks = 0; ks < C::KS; ++ks) {
        if constexpr (C::INT4) {
          // ks = 2c + u: values b + 2u + {0,1,2,3} sit in raw[.][2c] (u = 0: 0..3 of b)
          // and raw[.][2c + 1] (4..7 of b); pair (2u, 2u + 4) and (2u + 1, 2u + 5)
          const uint2 lo4 = raw[nt][ks & ~1], hi4 = raw[nt][ks | 1];
          const uint32_t e = (ks & 1) ? lo4.y : lo4.x;   // values b+2u, b+2u+1
          const uint32_t f = (ks & 1) ? hi4.y : hi4.x;   // values b+2u+4, b+2u+5
          const uint32_t f0 = pack_f16(bf16_lo(e) * up, bf16_lo(f) * up);
          const uint32_t f1 = pack_f16(bf16_hi(e) * up, bf16_hi(f) * up);
          if constexpr (C::QSMEM) {   // k-steps 2j and 2j + 1 share one 16-byte entry
            uint4 &q4 = qfs[(nt * (C::KS / 2) + (ks >> 1)) * 32 + lane];
            if (ks & 1) {
              q4.z = f0;
              q4.w = f1;
            } else {
              q4.x = f0;
              q4.y = f1;
            }
          } else {
            st.qf[nt][ks][0] = f0;
            st.qf[nt][ks][1] = f1;
          }
        } else {
          const uint2 v = raw[nt][ks];
          const uint32_t f0 = pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up);
          const uint32_t f1 = pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up);
          if constexpr (C::QSMEM) {   // k-steps 2j and 2j + 1 share one 16-byte entry
            uint4 &q4 = qfs[(nt * (C::KS / 2) + (ks >> 1)) * 32 + lane];
            if (ks & 1) {
              q4.z = f0;
              q4.w = f1;
            } else {
              q4.x = f0;
              q4.y = f1;
            }
          } else {
            st.qf[nt][ks][0] = f0;
            st.qf[nt][ks][1] = f1;
          }
        }
      }
  }
}

// The 16-token tiles a sequence of L cached tokens is attended over: with a window
// ("KV Cache Engineering for LLM Serving", section 3) only positions
// [max(0, L - window), L) count, so whole tiles before that are skipped and the
// first kept tile may start part-way.
struct SeqTiles {
  int first;       // absolute index of the first tile
  int count;       // tiles attended
  int last_valid;  // valid tokens in the last tile (1..16)
  int first_skip;  // tokens before the window in the first tile (0..15)
};

__device__ __forceinline__ SeqTiles seq_tiles(int L, int window, int cascade_tiles = 0) {
  int start = (window > 0 && L > window) ? L - window : 0;
  // tiles of a shared prefix that the cascade kernel attends over are skipped here
  start = max(start, min(cascade_tiles * kTile, L));
  const int end_tiles = (L + kTile - 1) / kTile;
  SeqTiles t;
  t.first = start / kTile;
  t.count = end_tiles - t.first;
  t.last_valid = L - (end_tiles - 1) * kTile;
  t.first_skip = start - t.first * kTile;
  return t;
}

constexpr int kLoShift = 16;   // unit info bits 16..19: first valid token of the tile
constexpr int kKvhShift = 20;  // unit info bits 20..30: the unit's KV head (of the unit view)
constexpr int kKvhMask = 0x7FF;

// A head's reference maximum (log2 domain) moves only when a score exceeds it by more
// than this, so every p stays <= 2^8.
constexpr float kMaxSlack = 8.f;
// Quantised caches: largest restored |V| of a tile (V scale x largest code) for which P
// enters the PV product as one f16 term; the term's rounding then adds at most
// 2^-12 * 16 < 4e-3 to an output, a fifth of the quantised tolerance 2e-2.
constexpr float kOneTermV = 16.f;

// Tiles attended per (sequence, KV head): the window's tiles, the chosen pages, or
// the tiles after a cascaded shared prefix.
__device__ __forceinline__ int pair_tile_count(int L, int window, int topk,
                                               int cascade_tiles = 0) {
  if (topk > 0) return min(topk, (L + kTile - 1) / kTile);
  return seq_tiles(L, window, cascade_tiles).count;
}

// One 16-token tile: scores, online-softmax update, P V accumulation.
// sscale[nt]: factor from raw mma scores to log2-domain scores; vs[nt]: V scale of a
// quantised tile; vzero[h]: the tile's V scale of the unit's KV head h is zero, so
// its V rows count as zeros.  The accumulator stays in units of the piece's first
// nonzero V scale: a tile with another scale enters through P scaled by the ratio.
template <class C, bool LO>
__device__ __forceinline__ void process_tile(State<C> &st, const uint4 *qfs, uint32_t ktile,
                                             uint32_t vtile, int lo, int nvalid,
                                             const float (&sscale)[C::NT],
                                             const float (&vs)[C::NT],
                                             const bool (&vzero)[C::HEADS], int lane) {
  // tokens lo <= t < nvalid of the tile are attended
  const int r = lane >> 2, qd = lane & 3;
  float s[C::NT][4];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;

  // ---- S^T = K Q^T
  if constexpr (!C::QUANT) {
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int ks = 0; ks < C::KS; ++ks) {
      const int c = ((ks & 3) << 1) + (lane >> 4);
      uint32_t a[4];
      ldsm_x4(a, ktile + (ks >> 2) * (kTile * 128) + row * 128 + ((c ^ (row & 7)) << 4));
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) mma_bf16(s[nt], a, st.qf[nt][ks][0], st.qf[nt][ks][1]);
    }
  } else if constexpr (C::INT4) {
    // 64-byte head rows: lane (r, q) receives nibbles b..b+7 (b = 32c + 8q) of row r;
    // int4_pair_f16 yields the pairs (b+i, b+i+4) that load_q mirrors.  One head: a
    // 64-byte-swizzled box; paired heads: head h is chunks 4h..4h+3 of a 128-byte-
    // swizzled row and feeds n-tile h only.
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int h = 0; h < C::HEADS; ++h)
#pragma unroll
      for (int cc = 0; cc < C::D / 64; ++cc) {
        const int c = 2 * cc + (lane >> 4);
        uint32_t R[4];
        if constexpr (C::PAIRED)
          ldsm_x4(R, ktile + row * 128 + (((4 * h + c) ^ (row & 7)) << 4));
        else
          ldsm_x4(R, ktile + row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
#pragma unroll
        for (int half = 0; half < 2; ++half) {  // chunk 2cc + half: R[2 half] rows r, R[2 half + 1] rows r + 8
          uint4 q4 = make_uint4(0u, 0u, 0u, 0u);
          if constexpr (C::QSMEM) q4 = qfs[(h * (C::KS / 2) + 2 * cc + half) * 32 + lane];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a[4] = {int4_pair_f16(R[2 * half], 2 * u),
                                   int4_pair_f16(R[2 * half + 1], 2 * u),
                                   int4_pair_f16(R[2 * half], 2 * u + 1),
                                   int4_pair_f16(R[2 * half + 1], 2 * u + 1)};
            const int ks = (2 * cc + half) * 2 + u;
            if constexpr (C::QSMEM) {
              mma_f16(s[h], a, u ? q4.z : q4.x, u ? q4.w : q4.y);
            } else if constexpr (C::PAIRED) {
              mma_f16(s[h], a, st.qf[h][ks][0], st.qf[h][ks][1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < C::NT; ++nt)
                mma_f16(s[nt], a, st.qf[nt][ks][0], st.qf[nt][ks][1]);
            }
          }
        }
      }
  } else {
    // ldmatrix on byte pairs: lane (r, q) receives codes 4q..4q+3 of a 16-code chunk;
    // the mma's k order is permuted accordingly (load_q applies the same order to q).
    // Paired heads: head h is box h of the tile and feeds n-tile h only.
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int h = 0; h < C::HEADS; ++h)
#pragma unroll
      for (int kk = 0; kk < C::D / 32; ++kk) {
        const int c = 2 * kk + (lane >> 4);
        uint32_t R[4];
        ldsm_x4(R, ktile + h * (kTile * 128) + row * 128 + ((c ^ (row & 7)) << 4));
        const uint32_t a0[4] = {e4m3x2_to_f16x2(R[0]), e4m3x2_to_f16x2(R[1]),
                                e4m3x2_hi_to_f16x2(R[0]), e4m3x2_hi_to_f16x2(R[1])};
        const uint32_t a1[4] = {e4m3x2_to_f16x2(R[2]), e4m3x2_to_f16x2(R[3]),
                                e4m3x2_hi_to_f16x2(R[2]), e4m3x2_hi_to_f16x2(R[3])};
        if constexpr (C::PAIRED) {
          const uint4 q4 = qfs[(h * (C::KS / 2) + kk) * 32 + lane];
          mma_f16(s[h], a0, q4.x, q4.y);
          mma_f16(s[h], a1, q4.z, q4.w);
        } else {
#pragma unroll
          for (int nt = 0; nt < C::NT; ++nt) {
            mma_f16(s[nt], a0, st.qf[nt][2 * kk][0], st.qf[nt][2 * kk][1]);
            mma_f16(s[nt], a1, st.qf[nt][2 * kk + 1][0], st.qf[nt][2 * kk + 1][1]);
          }
        }
      }
  }

  // ---- V scale of a quantised tile relative to the accumulator's unit (warp-uniform).
  // The piece starts with vinv = 0, so its first nonzero scale takes the rare branch
  // that (re)expresses the accumulator in the tile's own scale.
  float rat[C::NT];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt) {
    rat[nt] = 1.f;
    if constexpr (C::QUANT) {
      rat[nt] = vs[nt] * st.vinv[nt];
      if (!vzero[C::PAIRED ? nt : 0] && !(rat[nt] <= kRatMax && rat[nt] >= kRatMin)) {
        const float f = st.vref[nt] / vs[nt];
#pragma unroll
        for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.acc[nt][dt][i] *= f;
        st.vref[nt] = vs[nt];
        st.vinv[nt] = 1.f / vs[nt];
        rat[nt] = 1.f;
      }
    }
  }

  // ---- online softmax (log2 domain); element i: token r + 8*(i>>1), head 2q + (i&1).
  // Each head's reference maximum st.m moves only when a score exceeds it by more than
  // kMaxSlack, so p <= 2^kMaxSlack; the result is the same (o and l share the
  // reference).  A tile that moves no reference needs no reduction across lanes and
  // no rescaling of the accumulator: one compare per score and a warp vote.
  const bool ragged = nvalid < kTile || lo > 0;   // warp-uniform
  float x[C::NT][4];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) x[nt][i] = s[nt][i] * sscale[nt];
  if constexpr (C::SCORED) {
    // capped: x is the score over the cap so far.  Scores seldom pass the cap, so a tile of them
    // takes the short form and one vote.
    if (st.cap2 > 0.f) {
      bool far = false;
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) far |= fabsf(x[nt][i]) > 1.f;
      const bool any = __any_sync(0xffffffffu, far);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[nt][i] = st.cap2 * (any ? tanh_any(x[nt][i]) : tanh_within_1(x[nt][i]));
    }
    const float d0 = static_cast<float>(r - st.behind), d1 = static_cast<float>(r + 8 - st.behind);
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(st.slope[nt][i & 1], (i >> 1) ? d1 : d0, x[nt][i]);
  }
  if (ragged) {
    const bool in0 = r >= lo && r < nvalid, in1 = r + 8 >= lo && r + 8 < nvalid;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!((i >> 1) ? in1 : in0)) x[nt][i] = -INFINITY;
  }
  bool over = false;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) over |= x[nt][i] > st.m[nt][i & 1] + kMaxSlack;
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      float alpha[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float mx = fmaxf(x[nt][j], x[nt][j + 2]);
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
        const float mnew = fmaxf(st.m[nt][j], mx);
        alpha[j] = ex2(st.m[nt][j] - mnew);
        st.l[nt][j] *= alpha[j];
        st.m[nt][j] = mnew;
      }
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.acc[nt][dt][i] *= alpha[i & 1];
    }
  }
  float p[C::NT][4];
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p[nt][j] = ex2(x[nt][j] - st.m[nt][j]);
      p[nt][j + 2] = ex2(x[nt][j + 2] - st.m[nt][j]);
      st.l[nt][j] += p[nt][j] + p[nt][j + 2];
    }

  // ---- P^T fragments, transposed in registers.  bf16 caches split p into two bf16
  // terms, hi + lo (16 significant bits).  Quantised caches feed p times the tile's
  // V-scale ratio as one f16 term (relative rounding <= 2^-12).  With LO (tiles whose
  // restored V values exceed kOneTermV, chosen by the caller) the f16 remainder follows
  // as a second term, 22 significant bits in all: its fragments are parked in the tile's
  // K area (free once S is computed) and the same PV code runs a second time with them,
  // so this rare instantiation needs no more registers than the common one.
  uint32_t bh[C::NT][2], bl[C::NT][2];
  if constexpr (C::QUANT && LO) __syncwarp();   // every lane is done reading the K tile
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (!C::QUANT) {
        const float p0 = p[nt][2 * h], p1 = p[nt][2 * h + 1];
        const uint32_t hi = pack_bf16(p0, p1);
        bh[nt][h] = movmatrix_trans(hi);
        bl[nt][h] = movmatrix_trans(pack_bf16(p0 - bf16_lo(hi), p1 - bf16_hi(hi)));
      } else {
        const float p0 = p[nt][2 * h] * rat[nt], p1 = p[nt][2 * h + 1] * rat[nt];
        const uint32_t hi = pack_f16(p0, p1);
        bh[nt][h] = movmatrix_trans(hi);
        if constexpr (LO) {
          const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
          sts_u32(ktile + ((nt * 2 + h) * 32 + lane) * 4,
                  movmatrix_trans(pack_f16(p0 - hf.x, p1 - hf.y)));
        }
      }
    }
  // the second pass of a quantised LO tile: the parked remainders become the P fragments
  auto take_lo = [&]() {
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) bh[nt][h] = lds_u32(ktile + ((nt * 2 + h) * 32 + lane) * 4);
  };

  // ---- O^T += V^T P^T.  A masked token has p = 0 exactly, but stale bf16 or E4M3 rows
  // may hold non-finite values (0 * NaN = NaN), so for those caches the V rows of a
  // ragged tile (and of a tile whose V scale is zero) are zeroed in registers under
  // one warp-uniform branch; full tiles skip it.  Every 4-bit code converts to a finite
  // value and a zero V scale already makes P zero (rat = 0), so 4-bit tiles need no
  // mask.
  if constexpr (!C::QUANT) {
    auto pv = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t m01 = 0xFFFFFFFFu, m23 = 0xFFFFFFFFu;
      if constexpr (MASK) {
        auto in = [&](int t) { return t >= lo && t < nvalid; };
        m01 = (in(2 * qd) ? 0x0000FFFFu : 0u) | (in(2 * qd + 1) ? 0xFFFF0000u : 0u);
        m23 = (in(2 * qd + 8) ? 0x0000FFFFu : 0u) | (in(2 * qd + 9) ? 0xFFFF0000u : 0u);
      }
      const int t = (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt) {
        const int c = ((dt & 3) << 1) + ((lane >> 3) & 1);
        uint32_t a[4];
        ldsm_x4_trans(a, vtile + (dt >> 2) * (kTile * 128) + t * 128 + ((c ^ (t & 7)) << 4));
        if constexpr (MASK) {
          a[0] &= m01;
          a[1] &= m01;
          a[2] &= m23;
          a[3] &= m23;
        }
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt) {
          mma_bf16(st.acc[nt][dt], a, bh[nt][0], bh[nt][1]);
          mma_bf16(st.acc[nt][dt], a, bl[nt][0], bl[nt][1]);
        }
      }
    };
    if (ragged) pv(std::true_type{}); else pv(std::false_type{});
  } else if constexpr (C::INT4) {
    // ldmatrix.trans on the byte-pair view gives lane (r, q) the nibbles d = 32c + 4r
    // .. +3 of tokens 2q (low half) and 2q + 1 (high half): int4_pair_f16(., i) is
    // V^T row d = 32c + 4r + i over tokens (2q, 2q + 1).  Paired heads as for K.
    const int t = (lane & 7) + (((lane >> 3) & 1) << 3);
    auto pv = [&]() {
#pragma unroll
      for (int h = 0; h < C::HEADS; ++h) {
#pragma unroll
        for (int cc = 0; cc < C::D / 64; ++cc) {
          const int c = 2 * cc + (lane >> 4);
          uint32_t R[4];
          if constexpr (C::PAIRED)
            ldsm_x4_trans(R, vtile + t * 128 + (((4 * h + c) ^ (t & 7)) << 4));
          else
            ldsm_x4_trans(R, vtile + t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
#pragma unroll
          for (int half = 0; half < 2; ++half)    // chunk 2cc + half
#pragma unroll
            for (int mt = 0; mt < 2; ++mt) {      // rows 4r + 2mt + {0, 1}
              const uint32_t a[4] = {int4_pair_f16(R[2 * half], 2 * mt),
                                     int4_pair_f16(R[2 * half], 2 * mt + 1),
                                     int4_pair_f16(R[2 * half + 1], 2 * mt),
                                     int4_pair_f16(R[2 * half + 1], 2 * mt + 1)};
              const int dt = (2 * cc + half) * 2 + mt;
              if constexpr (C::PAIRED) {
                mma_f16(st.acc[h][dt], a, bh[h][0], bh[h][1]);
              } else {
#pragma unroll
                for (int nt = 0; nt < C::NT; ++nt) mma_f16(st.acc[nt][dt], a, bh[nt][0], bh[nt][1]);
              }
            }
        }
      }
    };
    pv();
    if constexpr (LO) {
      take_lo();
      pv();
    }
  } else {
    // ldmatrix.trans on byte pairs gives lane (r, q): bytes (t=2q: d=2r, 2r+1) and
    // (t=2q+1: d=2r, 2r+1); regrouping by d yields V^T rows d = 2r (even) and 2r+1
    // (odd) -- the tile's 16 output rows in the order (2r, 2r+1).
    // Paired heads: head h is box h of the tile and feeds n-tile h only.
    auto pv = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      uint32_t m01[C::HEADS], m23[C::HEADS];
#pragma unroll
      for (int h = 0; h < C::HEADS; ++h) {
        m01[h] = m23[h] = 0xFFFFFFFFu;
        if constexpr (MASK) {
          if (vzero[h]) {
            m01[h] = m23[h] = 0u;
          } else {
            auto in = [&](int t) { return t >= lo && t < nvalid; };
            m01[h] = (in(2 * qd) ? 0x0000FFFFu : 0u) | (in(2 * qd + 1) ? 0xFFFF0000u : 0u);
            m23[h] = (in(2 * qd + 8) ? 0x0000FFFFu : 0u) | (in(2 * qd + 9) ? 0xFFFF0000u : 0u);
          }
        }
      }
      const int t = (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
      for (int h = 0; h < C::HEADS; ++h)
#pragma unroll
        for (int cc = 0; cc < C::D / 32; ++cc) {
          const int c = 2 * cc + (lane >> 4);
          uint32_t R[4];
          ldsm_x4_trans(R, vtile + h * (kTile * 128) + t * 128 + ((c ^ (t & 7)) << 4));
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            // one permute per register: (t0 d0, t0 d1, t1 d0, t1 d1) -> (t0 d0, t1 d0,
            // t0 d1, t1 d1); its low half is row 2r, its high half row 2r + 1
            const uint32_t lo8 = __byte_perm(R[2 * hh], 0, 0x3120);
            const uint32_t hi8 = __byte_perm(R[2 * hh + 1], 0, 0x3120);
            uint32_t a[4] = {e4m3x2_to_f16x2(lo8), e4m3x2_hi_to_f16x2(lo8),
                             e4m3x2_to_f16x2(hi8), e4m3x2_hi_to_f16x2(hi8)};
            if constexpr (MASK) {
              a[0] &= m01[h];
              a[1] &= m01[h];
              a[2] &= m23[h];
              a[3] &= m23[h];
            }
            if constexpr (C::PAIRED) {
              mma_f16(st.acc[h][2 * cc + hh], a, bh[h][0], bh[h][1]);
            } else {
#pragma unroll
              for (int nt = 0; nt < C::NT; ++nt)
                mma_f16(st.acc[nt][2 * cc + hh], a, bh[nt][0], bh[nt][1]);
            }
          }
        }
    };
    bool zmask = false;
#pragma unroll
    for (int h = 0; h < C::HEADS; ++h) zmask |= vzero[h];
    if (ragged || zmask) pv(std::true_type{}); else pv(std::false_type{});
    if constexpr (LO) {
      take_lo();
      if (ragged || zmask) pv(std::true_type{}); else pv(std::false_type{});
    }
  }
}

// Sum l over the 8 lanes that share a head pair; returns the per-head total.
template <class C>
__device__ __forceinline__ void reduce_l(const State<C> &st, float (&ltot)[C::NT][2]) {
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v = st.l[nt][j];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      ltot[nt][j] = v;
    }
}

// Write o = acc / l (normalised) for heads g < G to dst[g * hstride + d]; and, if
// requested, lse to lse_dst[g * lstride].
__device__ __forceinline__ void put(float *dst, float v) { *dst = v; }
__device__ __forceinline__ void put(uint16_t *dst, float v) {
  *dst = static_cast<uint16_t>(pack_bf16(v, 0.f));
}

template <class C, class Out>
__device__ __forceinline__ void write_normalised(const State<C> &st, Out *dst, float *lse_dst,
                                                 int G, int lane, size_t hstride = C::D,
                                                 size_t lstride = 1) {
  float ltot[C::NT][2];
  reduce_l<C>(st, ltot);
  const int qd = lane & 3;
#pragma unroll
  for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = nt * 8 + 2 * qd + j;
      if (g >= G) continue;
      const float f = (C::QUANT ? st.vref[nt] : 1.f) / ltot[nt][j];
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt) {
        put(dst + g * hstride + acc_d<C>(dt, j, lane), st.acc[nt][dt][j] * f);
        put(dst + g * hstride + acc_d<C>(dt, j + 2, lane), st.acc[nt][dt][j + 2] * f);
      }
      if (lse_dst && (lane >> 2) == 0)
        lse_dst[g * lstride] = (st.m[nt][j] + __log2f(ltot[nt][j])) * kLn2;
    }
}

// The cascade partials of sequence b, KV head kvh: lse [pieces][G] and o
// [pieces][G][D] in the cascade workspace at `cws` (0: none).  Returns the pieces.
__device__ __forceinline__ int cascade_partials(uint64_t cws, int B, int Hq, int Hkv, int G,
                                                int D, int b, int kvh, const float *&clse,
                                                const float *&co) {
  if (!cws) return 0;
  const CascadeLayout cl = cascade_layout(B, Hq, D);
  const uint8_t *cw = reinterpret_cast<const uint8_t *>(cws);
  const int m = reinterpret_cast<const int32_t *>(cw + cl.member)[b];
  if (m < 0) return 0;
  const size_t c0 = (static_cast<size_t>(m) * Hkv + kvh) * kCascadePieces * G;
  clse = reinterpret_cast<const float *>(cw + cl.lse) + c0;
  co = reinterpret_cast<const float *>(cw + cl.o) + c0 * D;
  return reinterpret_cast<const int32_t *>(cw + cl.pieces)[b];
}

// ----------------------------------------------------------------------------
// unit sources: which tiles a warp processes, in order
// ----------------------------------------------------------------------------

// Tiles w, w + NW, ... of one (b, kvh) pair's attended tiles, read straight from
// the block table.
// The copy record of one tile, built lane-parallel when a source loads 32 tiles:
// (row of the tile's first token in the pools' 2-D view, unit, scale index
// phys * Hkv + kvh of the unit view or -1 for a bad block, info bits).  A bad block
// reads the rows past the pool, which the copy fills with zeros.
__device__ __forceinline__ int4 tile_record(int phys, int tile, int unit, int kvh, int hkv,
                                            int bs, int nblocks, int info) {
  if (phys == kInvalidPhys) return make_int4(nblocks * bs, unit, -1, info);
  // block_size is 16 or 32: the tile's first row in its block is a mask away
  return make_int4(phys * bs + ((tile * kTile) & (bs - 1)), unit, phys * hkv + kvh, info);
}

struct PairSource {
  const int32_t *row;
  const int32_t *sel;   // this pair's chosen pages, or null
  int32_t *err;
  int pair, kvh, hkv, w, nw, bs, nblocks;
  SeqTiles geo;         // with a selection: count = pages chosen, first = 0
  int npages;           // 16-token pages of the sequence
  int shared_len;       // L2 hint: leading tokens in shared blocks, or -1 (no hint)
  int base;
  int4 cur, nxt;

  __device__ __forceinline__ int count() const {
    return geo.count > w ? (geo.count - w + nw - 1) / nw : 0;
  }
  __device__ __forceinline__ int4 load(int i) const {
    const int j = w + i * nw;
    if (j >= geo.count) return make_int4(0, 0, -1, 0);   // never issued
    int tile = geo.first + j, last_tile = geo.first + geo.count - 1;
    if (sel) {
      tile = __ldg(sel + j);
      last_tile = npages - 1;
    }
    const bool bad_page = sel && (tile < 0 || tile >= npages);
    if (bad_page) {
      set_err(err, PA_DEVERR_BLOCK_ID);
      tile = 0;
    }
    int phys = bad_page ? kInvalidPhys : __ldg(row + (tile * kTile) / bs);
    if (phys < 0 || phys >= nblocks) {
      set_err(err, PA_DEVERR_BLOCK_ID);
      phys = kInvalidPhys;
    }
    int info = (tile == last_tile) ? geo.last_valid : kTile;
    if (j == 0) info |= kFirstOfPair | (sel ? 0 : geo.first_skip << kLoShift);
    if (j == geo.count - 1) info |= kLastOfPair;
    if (i == 0) info |= kPieceStart;
    if (j + nw >= geo.count) info |= kPieceEnd;
    if (shared_len >= 0) info |= ((tile + 1) * kTile <= shared_len) ? kHintShared : kHintPrivate;
    return tile_record(phys, tile, pair, kvh, hkv, bs, nblocks, info | (kvh << kKvhShift));
  }
  __device__ __forceinline__ void init(int lane) {
    base = 0;
    cur = load(lane);
    nxt = load(32 + lane);
  }
  __device__ __forceinline__ int4 get(int i, int lane) {
    while (i >= base + 32) {
      cur = nxt;
      base += 32;
      nxt = load(base + 32 + lane);
    }
    return shfl_int4(cur, i - base);
  }
};

// A contiguous segment [begin, end) of the tile stream: position f belongs to the
// sequence b with prefix[b] <= f < prefix[b + 1] (binary search in shared memory),
// then to KV head (f - prefix[b]) / count(b) and attended tile (f - prefix[b]) % count(b).
struct SegmentSource {
  const int32_t *prefix;     // shared: [B + 1]
  const int32_t *seq_lens;
  const int32_t *block_tables;
  const int32_t *shared_prefix_lens;   // may be null
  const int32_t *sel;                  // [B, Hkv, topk] chosen pages, or null
  const int32_t *casc_tiles;           // [B] cascaded shared tiles, or null
  int32_t *err;
  int B, Hkv, bs, nblocks, max_blocks, window, topk;
  int begin, end;
  int base;
  int4 cur, nxt;

  __device__ __forceinline__ int count() const { return end - begin; }
  // Positions from the first token of tile i of the segment, which is of sequence b's unit kvh, to
  // the sequence's last token.
  __device__ __forceinline__ int behind(int i, int b, int kvh) const {
    const int start = prefix[b], nt = (prefix[b + 1] - start) / Hkv;
    const int L = min(max(__ldg(seq_lens + b), 0), max_blocks * bs);
    return L - 1 - (seq_tiles(L, window).first + begin + i - start - kvh * nt) * kTile;
  }
  __device__ __forceinline__ int4 load(int i) const {
    const int f = begin + i;
    if (f >= end) return make_int4(0, 0, -1, 0);   // never issued
    int lo = 0, hi = B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= f) lo = mid; else hi = mid - 1;
    }
    const int b = lo, start = prefix[b];
    const int nt = (prefix[b + 1] - start) / Hkv;
    const int r = f - start;
    const int kvh = r / nt, j = r - kvh * nt;
    const int L = min(max(__ldg(seq_lens + b), 0), max_blocks * bs);
    const int ct = casc_tiles ? casc_tiles[b] : 0;
    const SeqTiles geo = seq_tiles(L, window, ct);
    int tile = geo.first + j, last_tile = geo.first + geo.count - 1;
    bool bad_page = false;
    if (sel) {
      const int npages = (L + kTile - 1) / kTile;
      tile = __ldg(sel + (static_cast<size_t>(b) * Hkv + kvh) * topk + j);
      last_tile = npages - 1;
      bad_page = tile < 0 || tile >= npages;
      if (bad_page) {
        set_err(err, PA_DEVERR_BLOCK_ID);
        tile = 0;
      }
    }
    int phys = bad_page ? kInvalidPhys
                        : __ldg(block_tables + static_cast<size_t>(b) * max_blocks + (tile * kTile) / bs);
    if (phys < 0 || phys >= nblocks) {
      set_err(err, PA_DEVERR_BLOCK_ID);
      phys = kInvalidPhys;
    }
    int info = (tile == last_tile) ? geo.last_valid : kTile;
    if (j == 0) info |= kFirstOfPair | kPieceStart | (sel ? 0 : geo.first_skip << kLoShift);
    if (j == nt - 1) info |= kLastOfPair | kPieceEnd;
    if (i == 0) info |= kPieceStart;
    if (f == end - 1) info |= kPieceEnd;
    if (shared_prefix_lens)
      info |= ((tile + 1) * kTile <= __ldg(shared_prefix_lens + b)) ? kHintShared : kHintPrivate;
    if (ct > 0) info |= kCascade;
    return tile_record(phys, tile, b * Hkv + kvh, kvh, Hkv, bs, nblocks,
                       info | (kvh << kKvhShift));
  }
  __device__ __forceinline__ void init(int lane) {
    base = 0;
    cur = load(lane);
    nxt = load(32 + lane);
  }
  __device__ __forceinline__ int4 get(int i, int lane) {
    while (i >= base + 32) {
      cur = nxt;
      base += 32;
      nxt = load(base + 32 + lane);
    }
    return shfl_int4(cur, i - base);
  }
};

// ----------------------------------------------------------------------------
// the per-warp pipeline
// ----------------------------------------------------------------------------

struct WarpSmem {
  uint8_t *stage;     // STAGES * STAGE_BYTES, 1024-aligned
  uint64_t *bar;      // STAGES mbarriers
  int4 *meta;         // STAGES * 2 int4: unit, then the unit's k scales and v scales
  uint4 *qf;          // Q^T fragments when they live in shared memory, else null
};

template <class C>
__device__ __forceinline__ void issue(const WarpSmem &ws, int s, int4 u, const Params &p,
                                      const CUtensorMap *tmK, const CUtensorMap *tmV, int lane) {
  if (lane != 0) return;
  uint8_t *stage = ws.stage + s * C::STAGE_BYTES;
  const uint32_t bar = smem_u32(&ws.bar[s]);
  const int y = u.x, sidx = u.z;
  const int kvh = (u.w >> kKvhShift) & kKvhMask;
  ws.meta[2 * s] = u;
  if constexpr (C::QUANT) {
    // the k scales of the unit's KV heads (kvh, or 2 kvh and 2 kvh + 1), then their
    // v scales
    float *sc = reinterpret_cast<float *>(&ws.meta[2 * s + 1]);
    if (sidx >= 0) {
      const size_t i = static_cast<size_t>(sidx) * C::HEADS;
      if constexpr (C::PAIRED) {
        cp_async_8(smem_u32(sc), p.k_scale + i);
        cp_async_8(smem_u32(sc + 2), p.v_scale + i);
      } else {
        cp_async_4(smem_u32(sc), p.k_scale + i);
        cp_async_4(smem_u32(sc + 2), p.v_scale + i);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 4; ++h) sc[h] = 0.f;
    }
    cp_async_arrive(bar);
  }
  const bool with_q = !C::QSMEM && (u.w & kPieceStart) != 0;
  const uint32_t bytes = 2 * C::KV_BYTES + (with_q ? p.G * C::D * 2 : 0);
  const uint32_t dst = smem_u32(stage);
  fence_proxy_async();
  mbar_arrive_expect_tx(bar, bytes);
  // the row of KV head kvh starts at element kvh * (ROW / element bytes)
  const int x0 = kvh * C::BOXES * C::BOX_X;
  if (u.w & (kHintShared | kHintPrivate)) {
    const uint64_t pol = (u.w & kHintShared) ? l2_policy_evict_last() : l2_policy_evict_first();
#pragma unroll
    for (int h = 0; h < C::BOXES; ++h) {
      const int x = x0 + h * C::BOX_X;
      tma_load_2d_hint(dst + h * (kTile * C::BOX_BYTES), tmK, x, y, bar, pol);
      tma_load_2d_hint(dst + C::KV_BYTES + h * (kTile * C::BOX_BYTES), tmV, x, y, bar, pol);
    }
  } else {
#pragma unroll
    for (int h = 0; h < C::BOXES; ++h) {
      const int x = x0 + h * C::BOX_X;
      tma_load_2d(dst + h * (kTile * C::BOX_BYTES), tmK, x, y, bar);
      tma_load_2d(dst + C::KV_BYTES + h * (kTile * C::BOX_BYTES), tmV, x, y, bar);
    }
  }
  if (with_q) {                                  // a piece starts: the group's query rows
    const int b = u.y / p.Hkv;
    bulk_load(dst + 2 * C::KV_BYTES, p.q + (static_cast<size_t>(b) * p.Hq + kvh * p.G) * C::D,
              p.G * C::D * 2, bar);
  }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  const bool ok = mbar_wait(bar, parity);
  return __all_sync(0xffffffffu, ok);
}

// Runs all units of `src` (already init()ed) through the warp's ring.
// on_piece_end(u, piece_has_pair_start, st) is called after the last tile of every
// piece.  Returns false after a wait timeout.
template <class C, class Src, class OnEnd>
__device__ __forceinline__ bool run_warp(Src &src, const WarpSmem &ws, State<C> &st,
                                         const Params &p, const CUtensorMap *tmK,
                                         const CUtensorMap *tmV, OnEnd &&on_piece_end,
                                         int lane) {
  const int n = src.count();
#pragma unroll
  for (int s = 0; s < C::STAGES; ++s)
    if (s < n) issue<C>(ws, s, src.get(s, lane), p, tmK, tmV, lane);
  bool piece_first = false;
  for (int i = 0; i < n; ++i) {
    const int s = i % C::STAGES;
    const uint32_t bar = smem_u32(&ws.bar[s]);
    if (!warp_wait(bar, (i / C::STAGES) & 1)) {
      set_err(lane == 0 ? p.err : nullptr, PA_DEVERR_TIMEOUT);
      for (int j = i; j < n && j < i + C::STAGES; ++j)
        mbar_wait(smem_u32(&ws.bar[j % C::STAGES]), (j / C::STAGES) & 1);
      return false;
    }
    const int4 u = ws.meta[2 * s];
    uint8_t *stage = ws.stage + s * C::STAGE_BYTES;
    const uint32_t ktile = smem_u32(stage);
    float sscale[C::NT], vs[C::NT];
    bool vzero[C::HEADS];
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt) {
      sscale[nt] = p.sl2;
      vs[nt] = 1.f;
    }
#pragma unroll
    for (int h = 0; h < C::HEADS; ++h) vzero[h] = false;
    if (u.w & kPieceStart) {
      st.reset();
      if constexpr (C::QSMEM) {   // the group's query rows, straight from global memory
        const int b = u.y / p.Hkv, kvh = (u.w >> kKvhShift) & kKvhMask;
        load_q<C>(st, 0u, p.q + (static_cast<size_t>(b) * p.Hq + kvh * p.G) * C::D, ws.qf,
                  p.G, lane);
      } else {
        load_q<C>(st, ktile + 2 * C::KV_BYTES,
                  reinterpret_cast<const uint16_t *>(stage + 2 * C::KV_BYTES), nullptr, p.G,
                  lane);
      }
      piece_first = (u.w & kFirstOfPair) != 0;
      if constexpr (C::SCORED) {
        const int b = u.y / p.Hkv, kvh = u.y - b * p.Hkv;
        st.cap2 = p.cap2;
        st.behind = src.behind(i, b, kvh);
#pragma unroll
        for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int g = nt * 8 + 2 * (lane & 3) + j;
            st.slope[nt][j] = p.slopes && g < p.G ? slope_log2(__ldg(p.slopes + kvh * p.G + g)) : 0.f;
          }
      }
    }
    if constexpr (C::QUANT) {
      // n-tile nt reads KV head nt of the unit (paired) or the unit's one head; a zero
      // V scale zeroes the tile's V rows
      const float4 sc = *reinterpret_cast<const float4 *>(&ws.meta[2 * s + 1]);
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) {
        const int h = C::PAIRED ? nt : 0;
        const float ks = h ? sc.y : sc.x, v = h ? sc.w : sc.z;
        sscale[nt] = p.sl2 * ks * st.qshift;
        vzero[h] = !(v > 0.f);
        vs[nt] = v;
      }
    }
    // quantised tiles whose restored V values exceed kOneTermV take the two-term weights
    bool lo = false;
    if constexpr (C::QUANT) {
#pragma unroll
      for (int nt = 0; nt < C::NT; ++nt) lo |= vs[nt] * (C::FP8 ? 448.f : 7.f) > kOneTermV;
    }
    if (lo)
      process_tile<C, true>(st, ws.qf, ktile, ktile + C::KV_BYTES, (u.w >> kLoShift) & 0xF,
                            u.w & 0xFF, sscale, vs, vzero, lane);
    else
      process_tile<C, false>(st, ws.qf, ktile, ktile + C::KV_BYTES, (u.w >> kLoShift) & 0xF,
                             u.w & 0xFF, sscale, vs, vzero, lane);
    if constexpr (C::SCORED) st.behind -= kTile;
    if (u.w & kPieceEnd) on_piece_end(u, piece_first, st);
    __syncwarp();
    if (i + C::STAGES < n) issue<C>(ws, s, src.get(i + C::STAGES, lane), p, tmK, tmV, lane);
  }
  return true;
}

template <class C>
__device__ __forceinline__ WarpSmem setup_smem(uint8_t *raw, int warp, int G, int lane) {
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  WarpSmem ws;
  ws.stage = base + warp * C::STAGES * C::STAGE_BYTES;
  uint8_t *tail = base + C::WARPS * C::STAGES * C::STAGE_BYTES;
  ws.bar = reinterpret_cast<uint64_t *>(tail) + warp * C::STAGES;
  ws.meta = reinterpret_cast<int4 *>(tail + C::WARPS * C::STAGES * 8) + warp * C::STAGES * 2;
  ws.qf = nullptr;
  if constexpr (C::QSMEM)
    ws.qf = reinterpret_cast<uint4 *>(tail + C::WARPS * C::STAGES * (8 + C::META_BYTES) +
                                      warp * C::QF_BYTES);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) mbar_init(smem_u32(&ws.bar[s]), C::QUANT ? 2 : 1);
    fence_mbar_init();
  }
  // query rows G..8*NT-1 of every Q slot stay zero (the bulk copy writes G rows)
  if constexpr (!C::QSMEM) {
    const int pad = (8 * C::NT - G) * C::D * 2;
    for (int s = 0; s < C::STAGES; ++s) {
      uint8_t *qs = ws.stage + s * C::STAGE_BYTES + 2 * C::KV_BYTES + G * C::D * 2;
      for (int o = lane * 16; o < pad; o += 32 * 16)
        *reinterpret_cast<uint4 *>(qs + o) = make_uint4(0, 0, 0, 0);
    }
  }
  __syncwarp();
  return ws;
}

// First byte after the per-warp stages, barriers, metadata and Q^T fragment areas
// (16-byte aligned).
template <class C>
__device__ __forceinline__ uint8_t *split_tail(uint8_t *raw) {
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  return base + C::WARPS * (C::STAGES * (C::STAGE_BYTES + 8 + C::META_BYTES) + C::QF_BYTES);
}

// Dynamic shared memory of the split kernel: stages plus the length scan.
template <class C>
__host__ __device__ constexpr int split_smem(int B) {
  return C::SMEM + ((B + 1) * 4 + 15) / 16 * 16;
}

// ----------------------------------------------------------------------------
// pa_decode_splitkv: plan (scan + unit list), segmented decode, merge
// ----------------------------------------------------------------------------

__device__ __forceinline__ int clamp_len(int L, int cap) { return min(max(L, 0), cap); }

// Block-wide scan of the sequence lengths into shared memory:
//   prefix[b] = Hkv * sum_{b' < b} count(b'),  prefix[B] = total tiles,
// where count(b) is the number of 16-token tiles sequence b attends over.
// Out-of-range lengths are clamped (and reported once, by CTA 0).  Returns the
// largest count (the longest unit).
template <int THREADS>
__device__ int scan_lengths(const Params &p, int32_t *prefix) {
  __shared__ int warp_sums[THREADS / 32];
  __shared__ int carry_s, nmax_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = p.max_blocks * p.bs;
  if (tid == 0) carry_s = nmax_s = 0;
  __syncthreads();
  for (int base = 0; base < p.B; base += THREADS) {
    const int i = base + tid;
    int v = 0;
    if (i < p.B) {
      const int L0 = p.seq_lens[i];
      const int ct = p.casc_tiles ? p.casc_tiles[i] : 0;
      if ((L0 < 0 || L0 > cap || L0 < ct * kTile) && blockIdx.x == 0)
        set_err(p.err, PA_DEVERR_SEQ_LEN);
      const int c = pair_tile_count(clamp_len(L0, cap), p.window, p.topk, ct);
      if (c > 0) atomicMax(&nmax_s, c);
      v = p.Hkv * c;
    }
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sums[warp] = x;
    __syncthreads();
    int before = carry_s;
    for (int w = 0; w < warp; ++w) before += warp_sums[w];
    if (i < p.B) prefix[i] = before + x - v;
    __syncthreads();
    if (tid == THREADS - 1) carry_s = before + x;
    __syncthreads();
  }
  if (tid == 0) prefix[p.B] = carry_s;
  __syncthreads();
  return nmax_s;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, C::MIN_BLOCKS)
    decode_segment_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  WarpSmem ws = setup_smem<C>(smem_raw, warp, p.G, lane);
  int32_t *prefix = reinterpret_cast<int32_t *>(split_tail<C>(smem_raw));
  if (p.casc_tiles) pdl_wait();   // the cascaded tiles are written by the cascade kernel
  const int nmax = scan_lengths<C::THREADS>(p, prefix);
  const int seg = blockIdx.x * C::WARPS + warp;
  const int total = prefix[p.B];
  int W = max(1, (total + p.num_splits - 1) / p.num_splits);
  // pa_decode_splitkv: a unit of n tiles is cut into at most ceil((n - 1) / W) + 1
  // pieces, so W >= (nmax - 1) / (S - 1) keeps every unit within its S slots; with
  // S = 1 the segment bounds move to the next unit start, so no unit is cut
  const int S = p.parts_S;
  if (S >= 2) W = max(W, (nmax - 1 + S - 2) / (S - 1));
  SegmentSource src;
  src.prefix = prefix;
  src.seq_lens = p.seq_lens;
  src.block_tables = p.block_tables;
  src.shared_prefix_lens = p.shared_prefix_lens;
  src.err = p.err;
  src.B = p.B;
  src.Hkv = p.Hkv;
  src.bs = p.bs;
  src.nblocks = p.nblocks;
  src.max_blocks = p.max_blocks;
  src.window = p.window;
  src.sel = p.sel;
  src.topk = p.topk;
  src.casc_tiles = p.casc_tiles;
  src.begin = min(seg * W, total);
  src.end = (seg < p.num_splits) ? min(src.begin + W, total) : src.begin;
  if (S == 1) {
    auto unit_start_at_or_after = [&](int f) {   // f <= total
      if (f >= total) return total;
      int lo = 0, hi = p.B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (prefix[mid] <= f) lo = mid; else hi = mid - 1;
      }
      const int nt = (prefix[lo + 1] - prefix[lo]) / p.Hkv;
      const int us = prefix[lo] + (f - prefix[lo]) / nt * nt;
      return us < f ? us + nt : us;
    };
    src.begin = unit_start_at_or_after(src.begin);
    src.end = unit_start_at_or_after(src.end);
  }
  // the chosen pages are written by the selection launched just before
  if (p.sel) pdl_wait();
  src.init(lane);
  // without a selection everything above reads only caller inputs (lengths, block
  // tables); the pools (written by the cache write) and the workspace (read by the
  // previous merge) are touched only after the previous grid has finished
  pdl_wait();
  if (S > 0) {
    // sequences with no tile to attend have no piece: all their slots are empty
    for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
      if (prefix[b + 1] != prefix[b]) continue;
      float *l = p.parts_lse + static_cast<size_t>(b) * p.Hq * S;
      const size_t n = static_cast<size_t>(p.Hq) * S;
      for (size_t i = threadIdx.x; i < n; i += C::THREADS) l[i] = -INFINITY;
    }
  } else if (blockIdx.x == 0) {
    for (int i = threadIdx.x; i <= p.B; i += C::THREADS) p.prefix_out[i] = prefix[i];
    if (threadIdx.x == 0) {                 // for the merge: KV heads per unit, cascade
      p.prefix_out[p.B + 1] = C::HEADS;
      p.prefix_out[p.B + 2] = static_cast<int32_t>(static_cast<uint32_t>(p.casc_ws));
      p.prefix_out[p.B + 3] = static_cast<int32_t>(static_cast<uint32_t>(p.casc_ws >> 32));
    }
  }
  State<C> st;
  st.reset();
  run_warp<C>(
      src, ws, st, p, &tmK, &tmV,
      [&](int4 u, bool piece_first, State<C> &s) {
        const int b = u.y / p.Hkv, kvh = u.y - b * p.Hkv;
        const size_t row = static_cast<size_t>(b) * p.Hq + kvh * p.G;
        if (S > 0) {
          // piece k of the unit: the segments before this one that hold its tiles
          const int nt = (prefix[b + 1] - prefix[b]) / p.Hkv;
          const int k = S == 1 ? 0 : seg - (prefix[b] + kvh * nt) / W;
          write_normalised<C>(s, p.parts_o + (row * S + k) * C::D, p.parts_lse + row * S + k,
                              p.G, lane, static_cast<size_t>(S) * C::D, S);
          if (u.w & kLastOfPair) {              // the unit's last piece: later slots are empty
            const int rest = S - 1 - k;
            for (int i = lane; i < p.G * rest; i += 32) {
              const int g = i / rest;
              p.parts_lse[(row + g) * S + k + 1 + (i - g * rest)] = -INFINITY;
            }
          }
        } else if (piece_first && (u.w & kLastOfPair)) {   // the whole unit is in this segment
          if (u.w & kCascade) {                     // joined with its shared prefix by the merge
            const CascadeLayout cl = cascade_layout(p.B, p.Hq, C::D);
            uint8_t *cw = reinterpret_cast<uint8_t *>(p.casc_ws);
            write_normalised<C>(s, reinterpret_cast<float *>(cw + cl.uo) + row * C::D,
                                reinterpret_cast<float *>(cw + cl.ulse) + row, p.G, lane);
          } else {
            using Out = std::conditional_t<C::SCORED, uint16_t, float>;
            write_normalised<C>(s, reinterpret_cast<Out *>(p.out) + row * C::D, nullptr, p.G, lane);
          }
        } else {
          const size_t slot = static_cast<size_t>(seg) * 2 + (piece_first ? 1 : 0);
          write_normalised<C>(s, p.o_part + slot * p.G * C::D, p.lse_part + slot * p.G, p.G,
                              lane);
        }
      },
      lane);
}

// ----------------------------------------------------------------------------
// host side of the split decode
// ----------------------------------------------------------------------------

// Opt the kernel in to the dynamic shared memory it needs (per call: cheap, and
// correct whichever device is current).
template <class K>
static cudaError_t prep_kernel(K kernel, int smem) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
  return e;
}

static Params make_params(const pa_shape &s, float *out, const void *q, const float *k_scale,
                          const float *v_scale, const int32_t *bt, const int32_t *sl,
                          const pa_decode_opts *opts, float sm_scale, int32_t *err) {
  Params p{};
  p.window = opts ? opts->window : 0;
  p.topk = (opts && opts->selected_pages) ? opts->topk : 0;
  p.sel = p.topk > 0 ? opts->selected_pages : nullptr;
  p.out = out;
  p.q = static_cast<const uint16_t *>(q);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.block_tables = bt;
  p.seq_lens = sl;
  p.err = err;
  p.B = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.G = s.Hq / s.Hkv;
  p.bs = s.block_size;
  p.nblocks = s.nblocks;
  p.max_blocks = s.max_blocks;
  p.sl2 = sm_scale * kLog2e;
  return p;
}

template <class C>
static pa_status launch_segments(const Params &p, const CUtensorMap &mk, const CUtensorMap &mv,
                                 cudaStream_t stream) {
  const int smem = split_smem<C>(p.B);
  if (prep_kernel(decode_segment_kernel<C>, smem) != cudaSuccess) return PA_ERR_CUDA;
  const int grid = (p.num_splits + C::WARPS - 1) / C::WARPS;
  return launch_pdl(decode_segment_kernel<C>, dim3(grid), dim3(C::THREADS), smem, stream, mk, mv,
                    p) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

// Dispatch on (D, n-tiles, dtype), and on the file's constant kScored.
#define PA_DISPATCH(D_, NT_, KIND_, FN, ...)                                  \
  if (s.D == D_ && nt == NT_ && kind == KIND_) return FN<Cfg<D_, NT_, KIND_, kScored>>(__VA_ARGS__);

// 4-bit pools whose KV heads can be served two at a time: an even number of heads,
// groups of 8 query heads (one n-tile each), D = 128.  A Quest selection is per KV
// head, and the cascade stacks one KV head's query rows, so a decode with either
// serves the heads singly.
static bool int4_pairable(const pa_shape &s) {
  return s.kv_dtype == PA_KV_INT4 && s.D == 128 && s.Hkv % 2 == 0 && s.Hq == 8 * s.Hkv;
}
// E4M3 pools on the same rule.
static bool fp8_pairable(const pa_shape &s) {
  return s.kv_dtype == PA_KV_FP8_E4M3 && s.D == 128 && s.Hkv % 2 == 0 && s.Hq == 8 * s.Hkv;
}
static bool pairable(const pa_shape &s) { return int4_pairable(s) || fp8_pairable(s); }

// cascade: the decode runs the cascade (only pa_decode given a workspace does);
// cta_per_unit: pa_decode without a workspace (it pairs 4-bit heads, not E4M3 ones).
static int heads_per_unit(const pa_shape &s, const pa_decode_opts *opts, bool cascade = false,
                          bool cta_per_unit = false) {
  const bool per_head = (opts && opts->topk > 0 && opts->selected_pages) || cascade;
  const bool pair = int4_pairable(s) || (fp8_pairable(s) && !cta_per_unit);
  return (pair && !per_head) ? 2 : 1;
}

// The decode's view of the shape: units of `heads` adjacent KV heads.
static pa_shape unit_view(const pa_shape &s, int heads) {
  pa_shape v = s;
  v.Hkv = s.Hkv / heads;
  return v;
}

static int kind_of(const pa_shape &s, int heads) {
  if (s.kv_dtype == PA_KV_INT4) return heads == 2 ? kKindInt4x2 : kKindInt4;
  if (s.kv_dtype == PA_KV_FP8_E4M3) return heads == 2 ? kKindFp8x2 : kKindFp8;
  return kKindBf16;
}

#define PA_DISPATCH_ALL(FN, ...)                      \
  PA_DISPATCH(128, 1, kKindBf16, FN, __VA_ARGS__)     \
  PA_DISPATCH(128, 2, kKindBf16, FN, __VA_ARGS__)     \
  PA_DISPATCH(64, 1, kKindBf16, FN, __VA_ARGS__)      \
  PA_DISPATCH(64, 2, kKindBf16, FN, __VA_ARGS__)      \
  PA_DISPATCH(128, 1, kKindFp8, FN, __VA_ARGS__)      \
  PA_DISPATCH(128, 2, kKindFp8, FN, __VA_ARGS__)      \
  PA_DISPATCH(128, 1, kKindInt4, FN, __VA_ARGS__)     \
  PA_DISPATCH(128, 2, kKindInt4, FN, __VA_ARGS__)     \
  PA_DISPATCH(128, 2, kKindInt4x2, FN, __VA_ARGS__)   \
  PA_DISPATCH(128, 2, kKindFp8x2, FN, __VA_ARGS__)

}  // namespace pa
