// pa_attend.cu -- attention of ragged query tokens over the paged cache on tcgen05
// (pa_extend: causal, with an optional window; pa_cross_attend: every cached token).
//
//     out[i][h] = sum_j w_ij V[j] / sum_j w_ij,   w_ij = 2^(c s_ij - c m_i),
//     s_ij = <q[i][h], K[j]>,  c = sm_scale log2(e),  m_i a reference maximum of row i,
//
// j over the keys that token i sees.  The query heads of one KV head share its keys, so a
// tile's 128 rows are (token, head of the group) pairs: tok = floor(128 / G) tokens.
//
// Work.  A unit is (sequence, KV head, up to S tokens); its keys are the aligned 128-token
// tiles that any of its tokens sees (at least one tile, so that a row without keys is written
// too).  The tiles of all units, in (sequence, head, unit, key) order, are cut into equal
// segments, one per worker, as in the split decode: no length mix leaves a worker idle.  A
// unit inside one segment is written straight to `out`; a unit cut by segment bounds leaves
// (o, m, l) per piece in the workspace, joined by attend_merge_kernel in key order, so that
// the result does not depend on timing.
//
// Two forms.  Shared (long query runs): one worker per CTA, S = 2 tok, the CTA's two row
// tiles read the same keys.  Separate (few tokens per sequence): the CTA's two row tiles
// belong to two workers with S = tok, each with its own keys, so that one's loads, products
// and exponentials fill the other's waits.
//
// One CTA per SM: Q, K and V tiles in 128-byte-swizzled shared memory (TMA, one box per 16
// tokens of a page), S and O in TMEM (128 + D columns per row tile), P written over S as
// bf16 and read from TMEM by the second product.  Warps 0-3 and 4-7: the softmax of row
// tiles 0 and 1, one thread per row; one warp issues the products, one the loads.
#include <algorithm>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kKeys = 128;              // keys per tile
constexpr int kRows = 128;              // rows per tile
constexpr float kMaxJump = 8.f;         // the reference maximum moves only past this many octaves

struct AttendParams {
  uint16_t *out;
  const int32_t *offsets, *seq_lens, *block_tables;
  const float *k_scale, *v_scale;
  int32_t *err;
  float *part_o;                        // [2 workers][rows][D]
  float2 *part_ml;                      // [2 workers][rows]: (reference maximum times c, l)
  int4 *cut;                            // [workers]: the unit a worker leaves unfinished
  int B, Hq, Hkv, G, T, bs, max_blocks, nblocks, window, causal, tok, workers, rows;
  float c;                              // |sm_scale| log2(e)
  uint32_t negate;                      // sm_scale < 0: the products take -Q
};

// ------------------------------------------------------------------ units of work

struct Seq {
  int q0, n, L;      // first query row, query tokens, cached tokens (0: no token sees a key)
  int base;          // position of the first query token (causal)
  int lo;            // first position that any query token sees
};

__device__ __forceinline__ Seq load_seq(const AttendParams &p, int b, int32_t *err) {
  Seq s;
  const int q0 = p.offsets[b], q1 = p.offsets[b + 1];
  s.L = p.seq_lens[b];
  int bits = 0;
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= p.T;
  if (!ok) bits |= PA_DEVERR_QUERY;
  s.q0 = ok ? q0 : 0;
  s.n = ok ? q1 - q0 : 0;
  const int64_t most = static_cast<int64_t>(p.max_blocks) * p.bs;
  if (s.L < 0 || s.L > most) {
    bits |= PA_DEVERR_SEQ_LEN;
    s.L = s.L < 0 ? 0 : static_cast<int>(most);
  }
  if (p.causal && s.n > s.L) {
    bits |= PA_DEVERR_SEQ_LEN;
    s.L = 0;
  }
  s.base = p.causal && s.L > 0 ? s.L - s.n : 0;
  s.lo = p.causal && p.window > 0 && s.base >= p.window ? s.base - p.window + 1 : 0;
  if (bits && err) atomicOr(err, bits);
  return s;
}

// Key tiles of unit u (tokens [u S, (u + 1) S) of the sequence): first tile and count.
__device__ __forceinline__ void unit_tiles(const AttendParams &p, const Seq &s, int u, int S,
                                           int &t0, int &count) {
  int hi = s.L, lo = 0;
  if (p.causal && s.L > 0) {
    hi = s.base + min(s.n, (u + 1) * S);
    if (p.window > 0) lo = max(0, s.base + u * S - p.window + 1);
  }
  t0 = lo / kKeys;
  count = max(1, (hi + kKeys - 1) / kKeys - t0);
}

// sum over i < n of floor((a i + b) / 128) for a > 0, b >= 0: (the sum of a i + b, less the sum
// of its residues mod 128) / 128.  The residues run with period P = 128 / g, g = gcd(a, 128),
// through every value that is b mod g.
__device__ __forceinline__ int64_t floor_sum(int64_t n, int a, int64_t b) {
  const int lg = min(__ffs(a) - 1, 7), g = 1 << lg, P = kKeys >> lg;
  int64_t rest = (n >> (7 - lg)) * (static_cast<int64_t>(P) * (b & (g - 1)) + kKeys * (P - 1) / 2);
  for (int i = static_cast<int>(n & (P - 1)) - 1; i >= 0; --i) rest += (a * i + b) & (kKeys - 1);
  return (a * (n * (n - 1) / 2) + n * b - rest) >> 7;
}

// Key tiles of the first u units of one KV head of a sequence.
__device__ int64_t tiles_before(const AttendParams &p, const Seq &s, int u, int S) {
  if (u == 0) return 0;
  int t0, count;
  if (!p.causal || s.L == 0) {
    unit_tiles(p, s, 0, S, t0, count);
    return static_cast<int64_t>(u) * count;
  }
  int64_t sum = floor_sum(u, S, static_cast<int64_t>(s.base) + S + kKeys - 1);
  const int64_t end = s.base + static_cast<int64_t>(u) * S;
  if (end > s.L) sum += (s.L + kKeys - 1) / kKeys - (end + kKeys - 1) / kKeys;   // a short last unit
  if (p.window > 0) {
    const int gap = p.window - 1 - s.base;               // unit v's window starts at v S - gap
    const int v0 = gap > 0 ? (gap - 1) / S + 1 : 0;
    if (u > v0) sum -= floor_sum(u - v0, S, static_cast<int64_t>(v0) * S - gap);
  }
  return sum;
}

__device__ __forceinline__ int64_t shfl64(int64_t v, int src) {
  return __shfl_sync(0xffffffffu, v, src);
}

__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {   // inclusive
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// ceil(a / w), w < 2^15, by digits of 16 bits (a 64-bit division is a call, which would
// spill the softmax warps' registers)
__device__ __forceinline__ int64_t div_up(int64_t a, int w) {
  a += w - 1;
  int64_t q = 0;
  uint32_t r = 0;
#pragma unroll
  for (int sh = 48; sh >= 0; sh -= 16) {
    const uint32_t d = (r << 16) | (static_cast<uint32_t>(a >> sh) & 0xFFFFu);
    q = (q << 16) | (d / w);
    r = d % w;
  }
  return q;
}

__device__ __forceinline__ int64_t seq_tiles_total(const AttendParams &p, const Seq &s, int S) {
  return s.n > 0 ? p.Hkv * tiles_before(p, s, (s.n + S - 1) / S, S) : 0;
}

// A piece of a unit: key tiles [tile, tile + n) of unit tokens [row, row + ntok).
struct Piece {
  int seq, h, row, ntok, pos;  // pos: position of the first token (causal)
  int tile, n;                 // n = 0: no more pieces
  int L, lo;                   // the sequence's keys lie in [lo, L)
  int starts, ends;            // holds the unit's first / last key tile
};

// The pieces of one worker, in order.
struct Walker {
  int b, h, u, off, U;
  int remaining;
  Seq s;

  // [start, end) of the tile stream; sums: tiles of each group of 32 sequences
  __device__ void init(const AttendParams &p, const int64_t *sums, int64_t start, int64_t end,
                       int S, int lane) {
    remaining = static_cast<int>(max(static_cast<int64_t>(0), end - start));
    b = h = u = off = U = 0;
    s = Seq{};
    if (remaining == 0) return;
    const int groups = (p.B + 31) / 32;
    int g = 0;
    int64_t before = 0;
    for (int g0 = 0; g0 < groups; g0 += 32) {
      const int64_t v = scan64(g0 + lane < groups ? sums[g0 + lane] : 0, lane);
      const uint32_t past = __ballot_sync(0xffffffffu, before + v > start);
      const int first = past ? __ffs(past) - 1 : 32;
      if (first > 0) before += shfl64(v, first - 1);
      g = g0 + first;
      if (past) break;
    }
    const int mine = g * 32 + lane;
    Seq t{};
    int64_t total = 0;
    if (mine < p.B) {
      t = load_seq(p, mine, nullptr);
      total = seq_tiles_total(p, t, S);
    }
    const int64_t v = scan64(total, lane);
    const uint32_t past = __ballot_sync(0xffffffffu, before + v > start);
    const int l = past ? __ffs(past) - 1 : 31;
    const int64_t upto = shfl64(v - total, l);
    b = g * 32 + l;
    s = load_seq(p, b, nullptr);
    U = (s.n + S - 1) / S;
    const int64_t rem = start - before - upto;
    const int64_t per_head = tiles_before(p, s, U, S);
    for (int bit = 1 << 11; bit > 0; bit >>= 1)          // the last head with h per_head <= rem
      if ((h + bit) * per_head <= rem) h += bit;
    const int64_t r = rem - h * per_head;
    int lo = 0, hi = U;                       // the last unit with tiles_before <= r
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int cand = lo + lane * step;
      const uint32_t ok =
          __ballot_sync(0xffffffffu, cand < hi && tiles_before(p, s, cand, S) <= r);
      lo += (31 - __clz(ok)) * step;          // lane 0 always holds
      hi = min(hi, lo + step);
    }
    u = lo;
    off = static_cast<int>(r - tiles_before(p, s, u, S));
  }

  // rest: tiles of the unit after this piece
  __device__ __forceinline__ bool next(const AttendParams &p, int S, Piece &x, int &rest) {
    x.n = 0;
    if (remaining == 0) return false;
    while (U == 0) {                          // sequences without query tokens
      s = load_seq(p, ++b, nullptr);
      U = (s.n + S - 1) / S;
    }
    int t0, count;
    unit_tiles(p, s, u, S, t0, count);
    x.seq = b;
    x.h = h;
    x.row = s.q0 + u * S;
    x.ntok = min(S, s.n - u * S);
    x.pos = s.base + u * S;
    x.tile = t0 + off;
    x.n = min(count - off, remaining);
    x.L = s.L;
    x.lo = s.lo;
    x.starts = off == 0;
    off += x.n;
    remaining -= x.n;
    rest = count - off;
    x.ends = rest == 0;
    if (x.ends) {
      off = 0;
      if (++u == U) {
        u = 0;
        if (++h == p.Hkv) {
          h = 0;
          U = 0;                              // the next sequence is read when it is wanted
        }
      }
    }
    return true;
  }
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Matrix products of one thread are complete when `bar` has been arrived at.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}

// D[128 x N] (+)= A B, one 16-deep step; A in shared memory / in TMEM.
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t add) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(add)
      : "memory");
}

// Shared-memory operand in 128-byte swizzle: 8 rows x 128 bytes per atom, `sbo` bytes from
// one group of 8 rows to the next; `lbo` bytes between 64-element column chunks of an
// operand whose columns, not its depth, run along the rows.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) |
         (static_cast<uint64_t>(sbo >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// bf16 x bf16 -> fp32, M = 128; b_cols: B's columns run along its rows in memory.
constexpr uint32_t mma_desc(int N, bool b_cols) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (b_cols ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(kRows >> 4) << 24);
}
constexpr uint32_t kNegateA = 1u << 13;

#define PA_R8(r, o) "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), \
                    "=r"(r[o + 5]), "=r"(r[o + 6]), "=r"(r[o + 7])
#define PA_I8(r, o) "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), \
                    "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])

// 32 columns of this thread's TMEM lane
__device__ __forceinline__ void tc_ld32(uint32_t *r, uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : PA_R8(r, 0), PA_R8(r, 8), PA_R8(r, 16), PA_R8(r, 24)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::PA_I8(r, 0),
      PA_I8(r, 8), PA_I8(r, 16), PA_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,"
      "%13,%14,%15};" ::PA_I8(r, 0),
      PA_I8(r, 8), "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *map, int x, int y,
                                            int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}

// two fp32 operations in one instruction
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)),
        "l"(reinterpret_cast<uint64_t &>(c)));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(reinterpret_cast<uint64_t &>(d))
      : "l"(reinterpret_cast<uint64_t &>(a)), "l"(reinterpret_cast<uint64_t &>(b)));
  return d;
}

// ------------------------------------------------------------------ codes to bf16

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Two E4M3 codes (bytes 2 i and 2 i + 1 of w), exact: exponent and mantissa moved to bf16's
// places are the value times 2^-120 (the difference of the exponent biases, 127 - 7).
__device__ __forceinline__ uint32_t e4m3_pair_bf16(uint32_t w, int i) {
  const uint32_t x = __byte_perm(w, 0u, i == 0 ? 0x1404 : 0x3424);       // codes in the high bytes
  return bf16x2_mul((x & 0x80008000u) | ((x >> 4) & 0x07F007F0u), 0x7B807B80u);
}

// The two 4-bit codes of byte i of w, given w and w >> 4, exact: 128 + u is a bf16 with u in its
// lowest bits; less 136 it is the code u - 8.
__device__ __forceinline__ uint32_t int4_pair_bf16(uint32_t w, uint32_t w4, int i) {
  const uint32_t x = __byte_perm(w, w4, 0x4400 + i * 0x1111);
  return bf16x2_sub((x & 0x000F000Fu) | 0x43004300u, 0x43084308u);
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// A tile's codes (as TMA swizzled them) to a bf16 tile (128-byte swizzle), by four warps.
// Neighbouring lanes write both 64-column halves of a row at once; the order of a lane's stores
// keeps the two halves off each other's banks.
template <int KIND>
__device__ __forceinline__ void restore_tile(uint32_t raw, uint32_t dst, int w, int lane) {
  constexpr int kBatch = 4;
  if constexpr (KIND == PA_KV_FP8_E4M3) {
    const int c = lane & 7;                              // 16 codes: columns [16 c, 16 c + 16)
    for (int i0 = 0; i0 < 8; i0 += kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = (i0 + i) * 16 + w * 4 + (lane >> 3);
        v[i] = lds128(raw + r * 128 + ((c ^ (r & 7)) << 4));
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int r = (i0 + i) * 16 + w * 4 + (lane >> 3);
        const uint4 lo = make_uint4(e4m3_pair_bf16(v[i].x, 0), e4m3_pair_bf16(v[i].x, 1),
                                    e4m3_pair_bf16(v[i].y, 0), e4m3_pair_bf16(v[i].y, 1));
        const uint4 hi = make_uint4(e4m3_pair_bf16(v[i].z, 0), e4m3_pair_bf16(v[i].z, 1),
                                    e4m3_pair_bf16(v[i].w, 0), e4m3_pair_bf16(v[i].w, 1));
        const uint32_t row = dst + (c >> 2) * (kKeys * 128) + r * 128;
        const int c8 = 2 * (c & 3), odd = c >> 2;
        sts128(row + (((c8 + odd) ^ (r & 7)) << 4), odd ? hi : lo);
        sts128(row + (((c8 + 1 - odd) ^ (r & 7)) << 4), odd ? lo : hi);
      }
    }
  } else {
    const int c = lane & 3;                              // 32 codes: columns [32 c, 32 c + 32)
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + w * 8 + (lane >> 2);
      v[i] = lds128(raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 32 + w * 8 + (lane >> 2);
      const uint32_t row = dst + (c >> 1) * (kKeys * 128) + r * 128;
      const bool swap = c >= 2;
      if (swap) v[i] = make_uint4(v[i].z, v[i].w, v[i].x, v[i].y);
      const uint32_t words[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {                      // chunk j, or j ^ 2 of the other half
        const uint32_t x = words[j], x4 = x >> 4;
        const int c8 = 4 * (c & 1) + (swap ? j ^ 2 : j);
        sts128(row + ((c8 ^ (r & 7)) << 4),
               make_uint4(int4_pair_bf16(x, x4, 0), int4_pair_bf16(x, x4, 1),
                          int4_pair_bf16(x, x4, 2), int4_pair_bf16(x, x4, 3)));
      }
    }
  }
}

// ------------------------------------------------------------------ the kernel

// kKind: the pools' pa_kv_dtype.  Codes (D = 128) are restored to bf16 tiles, without their scale,
// by four warps of their own: K's scale multiplies the scores of a page, V's its weights.
template <int kD, int kKind, bool kShared>
struct AttendCfg {
  static constexpr int D = kD, KIND = kKind;
  static constexpr bool SHARED = kShared, QUANT = kKind != PA_KV_BF16;
  static constexpr int HALVES = D / 64;                 // 128-byte column chunks of a bf16 row
  static constexpr int TILE = kKeys * D * 2;            // bytes of a Q, K or V tile
  static constexpr int CODE_ROW = KIND == PA_KV_INT4 ? 64 : 128;
  static constexpr int RAW_TILE = kKeys * CODE_ROW;
  // the ring of K and V tiles; code pools: as many code tiles wait before it (224 KB with Q)
  static constexpr int STAGES = D == 64 ? 12 : KIND == PA_KV_BF16 ? 5 : KIND == PA_KV_FP8_E4M3 ? 3 : 4;
  static constexpr int RAW = QUANT ? 4 : 1;
  static constexpr int RING = 2 * TILE;                 // after the two Q tiles
  static constexpr int RAW_RING = RING + STAGES * TILE;
  static constexpr int SMEM = RAW_RING + (QUANT ? RAW * RAW_TILE : 0) + 1024;
  // Warps 0-7 softmax, then (code pools) four that restore codes, then one each for the
  // products, the loads and the pieces of each stream.  Registers are dealt out by groups of four
  // warps: 384 threads start with 168, 64,512 in all, dealt anew as 256 x 208 + 128 x 88 (512
  // with 128: 256 x 184 + 256 x 72): a softmax thread holds its row's 128 scores.
  static constexpr int THREADS = QUANT ? 512 : 384;
  static constexpr int CODE_WARP = 8;
  static constexpr int MMA_WARP = QUANT ? 12 : 8, LOAD_WARP = MMA_WARP + 1, PIECE_WARP = MMA_WARP + 2;
  static constexpr int SOFTMAX_REGS = QUANT ? 184 : 208, OTHER_REGS = QUANT ? 72 : 88;
  static constexpr int STREAMS = SHARED ? 1 : 2;        // key streams of a CTA
  static constexpr int PIECES = 8;                      // pieces known ahead per stream
  static constexpr int SCALES = 5;                      // tiles whose scales are held per stream
  // the scales of tile j + SCALES are stored before its K is issued; by then the copies have
  // come 2 (SCALES - 1) past V of tile j, which must be further than both rings hold
  static_assert(!QUANT || 2 * (SCALES - 1) >= RAW + STAGES, "scales overwritten too early");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kPieceBars = 2 * C::STAGES + 9, kRawBars = kPieceBars + 2 * C::STREAMS * C::PIECES;
  constexpr int kBars = kRawBars + (C::QUANT ? 2 * C::RAW + C::STREAMS * C::SCALES : 0);
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ Piece pieces[C::STREAMS][C::PIECES];
  __shared__ uint32_t tmem_slot;
  // scales of the tiles on their way: K's pages (16 tokens each), then V's
  __shared__ float4 scales[C::STREAMS][C::QUANT ? C::SCALES : 1][4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  auto kv_full = [&](int i) { return bar0 + 8 * i; };
  auto kv_empty = [&](int i) { return bar0 + 8 * (C::STAGES + i); };
  auto q_full = [&](int t) { return bar0 + 8 * (2 * C::STAGES + t); };
  auto s_full = [&](int t) { return bar0 + 8 * (2 * C::STAGES + 2 + t); };
  auto p_ready = [&](int t) { return bar0 + 8 * (2 * C::STAGES + 4 + t); };
  auto o_full = [&](int t) { return bar0 + 8 * (2 * C::STAGES + 6 + t); };
  const uint32_t done_bar = bar0 + 8 * (2 * C::STAGES + 8);
  // piece k of a stream is known / no longer needed
  auto pc_full = [&](int st, uint32_t k) {
    return bar0 + 8 * (kPieceBars + st * C::PIECES + k % C::PIECES);
  };
  auto pc_empty = [&](int st, uint32_t k) {
    return bar0 + 8 * (kPieceBars + (C::STREAMS + st) * C::PIECES + k % C::PIECES);
  };
  // code pools: code tiles landed / restored, scales of a stream's tile n stored
  auto raw_full = [&](int i) { return bar0 + 8 * (kRawBars + i); };
  auto raw_empty = [&](int i) { return bar0 + 8 * (kRawBars + C::RAW + i); };
  auto sc_full = [&](int st, uint32_t n) {
    return bar0 + 8 * (kRawBars + 2 * C::RAW + st * C::SCALES + n % C::SCALES);
  };
  auto sc_parity = [](uint32_t n) { return (n / C::SCALES) & 1; };
  auto pc_parity = [](uint32_t k) { return (k / C::PIECES) & 1; };
  const int S = C::SHARED ? 2 * p.tok : p.tok;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(kv_full(i), C::QUANT ? 4 : 1);           // the restoring warps, or the copies
      mbar_init(kv_empty(i), 1);
    }
    if constexpr (C::QUANT) {
      for (int i = 0; i < C::RAW; ++i) {
        mbar_init(raw_full(i), 1);
        mbar_init(raw_empty(i), 4);
      }
      for (int st = 0; st < C::STREAMS; ++st)
        for (int n = 0; n < C::SCALES; ++n) mbar_init(sc_full(st, n), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_ready(t), 4);
      mbar_init(o_full(t), 1);
    }
    mbar_init(done_bar, 1);
    for (int st = 0; st < C::STREAMS; ++st)
      for (int k = 0; k < C::PIECES; ++k) {
        mbar_init(pc_full(st, k), 1);
        mbar_init(pc_empty(st, k), 2 + (C::SHARED ? 8 : 4) + (C::QUANT ? 4 : 0));   // every reader
      }
    fence_mbar_init();
  }
  if (warp == C::MMA_WARP) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(&tmem_slot))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_trigger();
  pdl_wait();

  // every CTA counts the tiles: one sum per group of 32 sequences, in the space of the last
  // stage of the ring (which the loads wait for the piece warps to be done with)
  int64_t *sums = reinterpret_cast<int64_t *>(smem_raw + (sm - smem_u32(smem_raw)) + C::RING +
                                              (C::STAGES - 1) * C::TILE);
  const int groups = (p.B + 31) / 32;
  for (int g = warp; g < groups; g += C::THREADS / 32) {
    const int b = g * 32 + lane;
    int64_t t = 0;
    if (b < p.B) t = seq_tiles_total(p, load_seq(p, b, blockIdx.x == 0 ? p.err : nullptr), S);
    t = scan64(t, lane);
    if (lane == 31) sums[g] = t;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  bool ok = true;
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    // ---------------------------------------------------------------- softmax, one thread per row
    const int t = warp >> 2, st = C::SHARED ? 0 : t;
    const int row = tid & 127;
    const uint32_t tS = tmem + ((tid & 96) << 16) + t * kKeys;
    const uint32_t tO = tmem + ((tid & 96) << 16) + 256 + t * 128;
    const int my_tok = row / p.G;
    const int tok0 = C::SHARED ? t * p.tok : 0;          // first token of this row tile in a unit
    bool q_sent = false;                                 // Q of the next piece is on its way
    uint32_t q_loads = 0, q_used = 0, s_phase = 0, o_phase = 0;
    uint32_t tiles = 0;                                  // key tiles of the stream so far
    auto load_q = [&](const Piece &x) {                  // by one thread
      mbar_arrive_expect_tx(q_full(t), C::HALVES * p.tok * p.G * 128);
#pragma unroll
      for (int half = 0; half < C::HALVES; ++half)
        tma_load_3d(sm + t * C::TILE + half * (kKeys * 128), &tmQ, half * 64, x.h * p.G,
                    x.row + tok0, q_full(t));
      ++q_loads;
    };
    for (uint32_t k = 0;; ++k) {
      ok = mbar_wait(pc_full(st, k), pc_parity(k));
      if (!ok) break;
      const Piece x = pieces[st][k % C::PIECES];
      __syncwarp();
      if (lane == 0) mbar_arrive(pc_empty(st, k));
      if (x.n == 0) break;
      const uint32_t tile0 = tiles;
      tiles += x.n;
      const int ntok = min(p.tok, x.ntok - tok0);        // tokens of this tile
      if (ntok <= 0) continue;
      if (row == 0 && !q_sent) load_q(x);
      __syncwarp();
      q_sent = false;
      ++q_used;
      const bool live = my_tok < ntok;                   // else: a row of nobody
      const bool warp_live = (tid & 96) / p.G < ntok;
      // this row sees keys [lo, hi); every row of the tile sees [all_lo, all_hi)
      const int pos = x.pos + tok0 + my_tok;
      const int hi = p.causal ? min(pos + 1, x.L) : x.L;
      const int lo = p.causal && p.window > 0 ? max(0, pos - p.window + 1) : 0;
      const int all_hi = p.causal ? min(x.pos + tok0 + 1, x.L) : x.L;
      const int all_lo = p.causal && p.window > 0 ? x.pos + tok0 + ntok - p.window : 0;
      float m = -INFINITY;                               // reference maximum, times c
      float l = 0.f;
      for (int i = 0; i < x.n; ++i) {
        const int key0 = (x.tile + i) * kKeys;
        ok = mbar_wait(s_full(t), s_phase);
        if (!ok) break;
        s_phase ^= 1;
        if (i == x.n - 1 && row == 0) {
          // the products with this Q tile are done: the next piece's may come, if that piece is
          // known (it is, but for a piece that this row tile has no part in)
          const uint32_t k1 = k + 1;
          if (mbar_wait(pc_full(st, k1), pc_parity(k1))) {
            const Piece &y = pieces[st][k1 % C::PIECES];
            if (y.n > 0 && y.ntok > tok0) {
              load_q(y);
              q_sent = true;
            }
          }
        }
        __syncwarp();
        tc_fence_after();
        if (warp_live) {
          uint32_t s[kKeys];
#pragma unroll
          for (int j = 0; j < kKeys; j += 32) tc_ld32(s + j, tS + j);
          tc_wait_ld();
          const float *sc = nullptr;                     // 8 K scales, 8 V scales
          if constexpr (C::QUANT) {
            const uint32_t n = tile0 + i;
            ok = mbar_wait(sc_full(st, n), sc_parity(n));
            sc = reinterpret_cast<const float *>(scales[st][n % C::SCALES]);
#pragma unroll
            for (int j = 0; j < kKeys; j += 2) {
              const float f = sc[j / 16] * p.c;
              const float2 y = mul2(make_float2(__uint_as_float(s[j]), __uint_as_float(s[j + 1])),
                                    make_float2(f, f));
              s[j] = __float_as_uint(y.x);
              s[j + 1] = __float_as_uint(y.y);
            }
          }
          if (key0 < all_lo || key0 + kKeys > all_hi) {
            const int a = lo - key0;
            const unsigned n = static_cast<unsigned>(max(0, hi - lo));
#pragma unroll
            for (int j = 0; j < kKeys; ++j)
              if (static_cast<unsigned>(j - a) >= n) s[j] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int j = 0; j < kKeys; j += 8)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mx[e] = fmaxf(mx[e], fmaxf(__uint_as_float(s[j + e]), __uint_as_float(s[j + 4 + e])));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (C::QUANT ? 1.f : p.c);
          if (m == -INFINITY) m = top;                   // O and l are zero so far
          // the reference moves only past kMaxJump octaves: weights stay below 2^8, far
          // inside bf16 and fp32, and O is seldom rescaled
          const bool jump = live && l > 0.f && top > m + kMaxJump;
          if (__any_sync(0xffffffffu, jump)) {
            const float f = jump ? ex2(m - top) : 1.f;
            if (jump) m = top;
            l *= f;
#pragma unroll
            for (int j = 0; j < C::D; j += 32) {
              uint32_t o[32];
              tc_ld32(o, tO + j);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc_st32(tO + j, o);
            }
            tc_wait_st();
          }
          const float2 c2 = make_float2(p.c, p.c);
          const float neg = m == -INFINITY ? 0.f : -m;
          const float2 n2 = make_float2(neg, neg);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int j = 0; j < kKeys; j += 32) {
            uint32_t packed[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float2 y = make_float2(__uint_as_float(s[j + 2 * e]), __uint_as_float(s[j + 2 * e + 1]));
              y = C::QUANT ? add2(y, n2) : fma2(y, c2, n2);
              y.x = ex2(y.x);
              y.y = ex2(y.y);
              sum[e & 1] = add2(sum[e & 1], y);
              if constexpr (C::QUANT) {
                const float f = sc[8 + (j + 2 * e) / 16];
                y = mul2(y, make_float2(f, f));
              }
              packed[e] = pack_bf16(y.x, y.y);
            }
            tc_st16(tS + j / 2, packed);
          }
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
          tc_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready(t));
      }
      if (!ok) break;
      ok = mbar_wait(o_full(t), o_phase);
      if (!ok) break;
      o_phase ^= 1;
      tc_fence_after();
      if (warp_live) {
        if (x.starts && x.ends) {
          const float inv = l > 0.f ? 1.f / l : 0.f;
          uint16_t *dst = p.out + (static_cast<int64_t>(x.row + tok0 + my_tok) * p.Hq +
                                   x.h * p.G + (row - my_tok * p.G)) * C::D;
#pragma unroll
          for (int j = 0; j < C::D; j += 32) {
            uint32_t o[32];
            tc_ld32(o, tO + j);
            tc_wait_ld();
            if (live) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                uint4 v;
                uint32_t *u = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  u[i] = l > 0.f ? pack_bf16(__uint_as_float(o[8 * e + 2 * i]) * inv,
                                             __uint_as_float(o[8 * e + 2 * i + 1]) * inv)
                                 : 0u;
                reinterpret_cast<uint4 *>(dst + j)[e] = v;
              }
            }
          }
        } else {
          const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x * C::STREAMS + st) + x.starts;
          const int64_t r = slot * p.rows + (C::SHARED ? t * kRows : 0) + row;
          if (live) p.part_ml[r] = make_float2(m, l);
          float *dst = p.part_o + r * C::D;
#pragma unroll
          for (int j = 0; j < C::D; j += 32) {
            uint32_t o[32];
            tc_ld32(o, tO + j);
            tc_wait_ld();
            if (live) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                reinterpret_cast<uint4 *>(dst + j)[e] =
                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          }
        }
      }
      tc_fence_before();
    }
    // after a wait that gave up, a Q tile may still be arriving
    if (!ok && row == 0)
      for (uint32_t k = q_used > 0 ? q_used - 1 : 0; k < q_loads; ++k) mbar_wait(q_full(t), k & 1);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp >= C::PIECE_WARP) {
      // ---------------------------------------------------------------- the pieces of a stream
      const int st = warp - C::PIECE_WARP;
      if (st < C::STREAMS) {
        const int worker = blockIdx.x * C::STREAMS + st;
        int64_t total = 0;
        for (int g = lane; g < groups; g += 32) total += sums[g];
        total = shfl64(scan64(total, lane), 31);
        const int64_t width = div_up(total, p.workers);
        const int64_t first = min(total, worker * width);
        Walker walk;
        walk.init(p, sums, first, min(total, first + width), S, lane);
        fence_proxy_async();               // the sums' space is the ring's from here
        __syncwarp();
        int4 cut = make_int4(0, 0, 0, 0);
        for (uint32_t k = 0;; ++k) {
          Piece x;
          int rest = 0;
          const bool more = walk.next(p, S, x, rest);
          ok = mbar_wait(pc_empty(st, k), pc_parity(k) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            pieces[st][k % C::PIECES] = x;
            mbar_arrive(pc_full(st, k));
          }
          if (!more) break;
          if (x.starts && !x.ends)
            cut = make_int4(x.row, x.ntok, x.h, (rest - 1) / static_cast<int>(width) + 1);
        }
        if (lane == 0) p.cut[worker] = cut;
      }
    } else if (warp == C::LOAD_WARP) {
      // ---------------------------------------------------------------- K and V tiles
      // lane (half, page): one box of 16 tokens x 64 columns; code pools: x a whole row, by lanes
      // 0-7, while lanes 0-7 and 8-15 fetch the pages' K and V scales
      const int page = lane & 7, half = C::QUANT ? 0 : lane >> 3;
      const bool loads = lane < 8 * (C::QUANT ? 1 : C::HALVES);
      constexpr int kRing = C::QUANT ? C::RAW : C::STAGES;
      auto ring_full = [&](int i) { return C::QUANT ? raw_full(i) : kv_full(i); };
      auto ring_empty = [&](int i) { return C::QUANT ? raw_empty(i) : kv_empty(i); };
      struct Tile {
        bool ok;
        int h, boxes, blk, g;                              // blk < 0: this lane loads nothing
        float scale;
      };
      Piece pc[C::STREAMS] = {};
      int at[C::STREAMS] = {};
      uint32_t seen[C::STREAMS] = {};
      bool over[C::STREAMS] = {};
      Tile cur[C::STREAMS] = {}, prev[C::STREAMS] = {};
      auto fetch = [&](int st) {
        Tile t{};
        if (over[st]) return t;
        Piece &x = pc[st];
        if (at[st] == x.n) {
          const uint32_t k = seen[st]++;
          ok = ok && mbar_wait(pc_full(st, k), pc_parity(k));
          if (!ok) return t;
          x = pieces[st][k % C::PIECES];
          __syncwarp();
          if (lane == 0) mbar_arrive(pc_empty(st, k));
          at[st] = 0;
          over[st] = x.n == 0;
          if (over[st]) return t;
        }
        const int first = (x.tile + at[st]) * kKeys;
        ++at[st];
        t.ok = true;
        t.h = x.h;
        const int hi = min(x.L, first + kKeys), lo = max(x.lo, first);
        t.boxes = hi > lo ? (hi + 15) / 16 - lo / 16 : 0;
        t.g = first + 16 * page;
        t.blk = -1;
        if (t.g < hi && t.g + 16 > lo)
          t.blk = p.block_tables[static_cast<int64_t>(x.seq) * p.max_blocks + t.g / p.bs] & 0x7fffffff;
        return t;
      };
      uint32_t count = 0;
      auto issue = [&](const CUtensorMap *map, const Tile &t) {
        const int stage = count % kRing;
        ok = ok && mbar_wait(ring_empty(stage), ((count / kRing) & 1) ^ 1);
        if (!ok) return;
        ++count;
        constexpr int kBox = C::QUANT ? 16 * C::CODE_ROW : 16 * 128;
        if (lane == 0)
          mbar_arrive_expect_tx(ring_full(stage), t.boxes * kBox * (C::QUANT ? 1 : C::HALVES));
        __syncwarp();
        if (loads && t.blk >= 0) {
          int row = p.nblocks * p.bs;                      // outside the pool: reads zeros
          if (t.blk < p.nblocks)
            row = t.blk * p.bs + t.g % p.bs;
          else
            set_err(p.err, PA_DEVERR_BLOCK_ID);
          if constexpr (C::QUANT)
            tma_load_2d(sm + C::RAW_RING + stage * C::RAW_TILE + page * kBox, map, t.h * C::CODE_ROW,
                        row, ring_full(stage));
          else
            tma_load_2d(sm + C::RING + stage * C::TILE + half * (kKeys * 128) + page * kBox, map,
                        t.h * C::D + half * 64, row, ring_full(stage));
        }
      };
      // A tile's block ids are fetched two tiles ahead of its copy and its scales one ahead.
      uint32_t tiles[C::STREAMS] = {};
      Tile nxt[C::STREAMS] = {};
      auto fetch_scale = [&](Tile &t) {
        t.scale = 0.f;
        if (C::QUANT && t.ok && lane < 16 && t.blk >= 0 && t.blk < p.nblocks)
          t.scale = (lane < 8 ? p.k_scale : p.v_scale)[static_cast<int64_t>(t.blk) * p.Hkv + t.h];
      };
#pragma unroll
      for (int st = 0; st < C::STREAMS; ++st) {
        cur[st] = fetch(st);
        fetch_scale(cur[st]);
        if (cur[st].ok) nxt[st] = fetch(st);
      }
      for (bool more = true; more && ok;) {
        more = false;
#pragma unroll
        for (int st = 0; st < C::STREAMS; ++st) {
          if (!ok || !(prev[st].ok || cur[st].ok)) continue;
          more = true;
          fetch_scale(nxt[st]);
          const Tile far = nxt[st].ok ? fetch(st) : Tile{};
          if (prev[st].ok) issue(&tmV, prev[st]);
          if (cur[st].ok) {
            if constexpr (C::QUANT) {
              const uint32_t n = tiles[st]++;
              if (lane < 16) reinterpret_cast<float *>(scales[st][n % C::SCALES])[lane] = cur[st].scale;
              __syncwarp();
              if (lane == 0) mbar_arrive(sc_full(st, n));
            }
            issue(&tmK, cur[st]);
          }
          prev[st] = cur[st];
          cur[st] = nxt[st];
          nxt[st] = far;
        }
      }
      if (!ok) {
        // the copies in flight land in this CTA's memory: wait for them before leaving
        for (uint32_t k = count > kRing ? count - kRing : 0; k < count; ++k)
          mbar_wait(ring_full(k % kRing), (k / kRing) & 1);
      }
    } else if (C::QUANT && warp < C::MMA_WARP) {
      // ---------------------------------------------------------------- codes to bf16 tiles
      // in the order of the ring, until the pieces' tiles are all done
      uint32_t todo[C::STREAMS] = {}, next_piece[C::STREAMS] = {}, count = 0;
      bool over[C::STREAMS] = {};
      bool v_due[C::STREAMS] = {};
      auto one = [&] {
        const int from = count % C::RAW, to = count % C::STAGES;
        ok = ok && mbar_wait(raw_full(from), (count / C::RAW) & 1) &&
             mbar_wait(kv_empty(to), ((count / C::STAGES) & 1) ^ 1);
        if (!ok) return;
        ++count;
        restore_tile<C::KIND>(sm + C::RAW_RING + from * C::RAW_TILE, sm + C::RING + to * C::TILE,
                              warp - C::CODE_WARP, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(from));
          mbar_arrive(kv_full(to));
        }
      };
      for (bool more = true; more && ok;) {
        more = false;
#pragma unroll
        for (int st = 0; st < C::STREAMS; ++st) {
          if (todo[st] == 0 && !over[st]) {
            const uint32_t k = next_piece[st]++;
            ok = ok && mbar_wait(pc_full(st, k), pc_parity(k));
            if (!ok) break;
            todo[st] = pieces[st][k % C::PIECES].n;
            __syncwarp();
            if (lane == 0) mbar_arrive(pc_empty(st, k));
            over[st] = todo[st] == 0;
          }
          if (v_due[st]) one();                          // V of the tile before
          v_due[st] = todo[st] > 0;
          if (v_due[st]) {
            --todo[st];
            one();                                       // K
            more = true;
          }
        }
      }
    } else if (warp == C::MMA_WARP) {
      // ---------------------------------------------------------------- matrix products
      const uint32_t idS = mma_desc(kKeys, false) | (p.negate ? kNegateA : 0u);
      constexpr uint32_t idO = mma_desc(C::D, true);
      struct Tile {
        bool ok, first, last, two;
        int tile, lo, L;
      };
      Piece pc[C::STREAMS] = {};
      int at[C::STREAMS] = {};
      uint32_t seen[C::STREAMS] = {};
      bool over[C::STREAMS] = {};
      Tile cur[C::STREAMS] = {}, prev[C::STREAMS] = {};
      auto fetch = [&](int st) {
        Tile t{};
        if (over[st]) return t;
        if (at[st] == pc[st].n) {
          const uint32_t k = seen[st]++;
          ok = ok && mbar_wait(pc_full(st, k), pc_parity(k));
          if (!ok) return t;
          pc[st] = pieces[st][k % C::PIECES];
          __syncwarp();
          if (lane == 0) mbar_arrive(pc_empty(st, k));
          at[st] = 0;
          over[st] = pc[st].n == 0;
          if (over[st]) return t;
        }
        t.ok = true;
        t.first = at[st] == 0;
        t.two = C::SHARED && pc[st].ntok > p.tok;
        t.tile = pc[st].tile + at[st];
        t.lo = pc[st].lo;
        t.L = pc[st].L;
        t.last = ++at[st] == pc[st].n;
        return t;
      };
      uint32_t count = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
      // rows of a V tile that no token sees may hold anything: they become zeros, since
      // 0 * NaN would reach the sum
      auto clear_unseen = [&](const Tile &t, int stage) {
        const int a = t.lo - t.tile * kKeys, z = t.L - t.tile * kKeys;     // seen rows [a, z)
        if (a <= 0 && z >= kKeys) return;
        const uint32_t base = sm + C::RING + stage * C::TILE;
        for (int r = 0; r < kKeys; ++r) {
          if (r >= a && r < z) continue;
          if (lane < 8 * C::HALVES)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             base + (lane >> 3) * (kKeys * 128) + r * 128 + (lane & 7) * 16),
                         "r"(0u)
                         : "memory");
        }
        fence_proxy_async();
        __syncwarp();
      };
      auto mma_s = [&](int t, int stage) {                 // S_t = Q_t K^T
        if (lane == 0) {
          const uint64_t a = smem_desc(sm + t * C::TILE, 16, 1024);
          const uint64_t b = smem_desc(sm + C::RING + stage * C::TILE, 16, 1024);
  #pragma unroll
          for (int k = 0; k < C::D / 16; ++k) {
            const uint32_t o = ((k >> 2) * (kKeys * 128) + (k & 3) * 32) >> 4;
            tc_mma_ss(tmem + t * kKeys, a + o, b + o, idS, k > 0);
          }
          tc_commit(s_full(t));
        }
        __syncwarp();
      };
      auto mma_o = [&](int t, int stage, const Tile &x) {  // O_t += P_t V
        if (lane == 0) {
          const uint64_t b = smem_desc(sm + C::RING + stage * C::TILE, kKeys * 128, 1024);
  #pragma unroll
          for (int k = 0; k < kKeys / 16; ++k)
            tc_mma_ts(tmem + 256 + t * 128, tmem + t * kKeys + k * 8, b + ((k * 16 * 128) >> 4), idO,
                      !x.first || k > 0);
          if (x.last) tc_commit(o_full(t));
        }
        __syncwarp();
      };
      auto full = [&](uint32_t k) {
        ok = ok && mbar_wait(kv_full(k % C::STAGES), (k / C::STAGES) & 1);
      };
      auto release = [&](uint32_t k) {
        if (ok && lane == 0) tc_commit(kv_empty(k % C::STAGES));
      };
  #pragma unroll
      for (int st = 0; st < C::STREAMS; ++st) cur[st] = fetch(st);
      for (bool more = true; more && ok;) {
        more = false;
  #pragma unroll
        for (int st = 0; st < C::STREAMS; ++st) {
          const bool v = prev[st].ok, k = cur[st].ok;
          if (!ok || !(v || k)) continue;
          more = true;
          const uint32_t vk = count, kk = count + (v ? 1 : 0);
          count = kk + (k ? 1 : 0);
  #pragma unroll
          for (int i = 0; i < (C::SHARED ? 2 : 1); ++i) {
            const int t = C::SHARED ? i : st;
            if (v && (i == 0 || prev[st].two)) {
              if (i == 0) {
                full(vk);
                if (ok) clear_unseen(prev[st], vk % C::STAGES);
              }
              ok = ok && mbar_wait(p_ready(t), p_phase[t]);
              p_phase[t] ^= 1;
              if (ok) {
                tc_fence_after();
                mma_o(t, vk % C::STAGES, prev[st]);
              }
            }
            if (v && i == (C::SHARED ? 1 : 0)) release(vk);
            if (k && (i == 0 || cur[st].two)) {
              if (i == 0) full(kk);
              if (cur[st].first) {
                ok = ok && mbar_wait(q_full(t), q_phase[t]);
                q_phase[t] ^= 1;
              }
              if (ok) mma_s(t, kk % C::STAGES);
            }
          }
          if (k) release(kk);
          prev[st] = cur[st];
          if (k) cur[st] = fetch(st);
        }
      }
      // nothing of this CTA's products is in flight when its memory goes
      if (lane == 0) tc_commit(done_bar);
      __syncwarp();
      ok = mbar_wait(done_bar, 0) && ok;
    }
  }
  if (!ok && lane == 0) set_err(p.err, PA_DEVERR_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// Joins the pieces of the unit that worker blockIdx.x left unfinished: its own (the unit's
// first keys), then those that the next workers began with, in key order.
//     out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i,   M = max_i m_i
template <int D>
__global__ void __launch_bounds__(256) attend_merge_kernel(const AttendParams p) {

  pdl_trigger();
  pdl_wait();
  const int4 cut = p.cut[blockIdx.x];
  if (cut.w == 0) return;
  const int lane = threadIdx.x & 31;
  constexpr int E = D / 32;                              // channels per lane
  for (int r = blockIdx.y * 8 + (threadIdx.x >> 5); r < p.rows; r += gridDim.y * 8) {
    const int t = r / kRows, rr = r - t * kRows;
    const int in_tile = rr / p.G, tok = t * p.tok + in_tile;
    if (in_tile >= p.tok || tok >= cut.y) continue;
    auto slot = [&](int i) {
      const int64_t s = i == 0 ? 2 * static_cast<int64_t>(blockIdx.x) + 1
                               : 2 * (static_cast<int64_t>(blockIdx.x) + i);
      return s * p.rows + r;
    };
    float M = -INFINITY;
    for (int i = lane; i <= cut.w; i += 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float l = 0.f, o[E] = {};
    for (int i = 0; i <= cut.w; ++i) {
      const float2 ml = p.part_ml[slot(i)];
      if (!(ml.y > 0.f)) continue;
      const float f = ex2(ml.x - M);
      l += f * ml.y;
      const float *src = p.part_o + slot(i) * D + lane * E;
      if constexpr (E == 4) {
        const float4 v = *reinterpret_cast<const float4 *>(src);
        o[0] += f * v.x;
        o[1] += f * v.y;
        o[2] += f * v.z;
        o[3] += f * v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2 *>(src);
        o[0] += f * v.x;
        o[1] += f * v.y;
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    uint16_t *dst = p.out + (static_cast<int64_t>(cut.x + tok) * p.Hq + cut.z * p.G +
                             (rr - in_tile * p.G)) * D + lane * E;
    if constexpr (E == 4)
      *reinterpret_cast<uint2 *>(dst) =
          make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
    else
      *reinterpret_cast<uint32_t *>(dst) = pack_bf16(o[0] * inv, o[1] * inv);
  }
}

// ------------------------------------------------------------------ host side

// Separate key streams while a sequence has at most one row tile of tokens on average.
struct Plan {
  bool shared;
  int tok, workers, rows;
  size_t ml, o, total;         // byte offsets in the workspace (`cut` is at 0), and its size
};

Plan make_plan(const pa_shape &s, int T, int sms) {
  Plan x;
  const int G = s.Hq / s.Hkv;
  x.tok = kRows / G;
  x.shared = T > static_cast<int64_t>(s.B) * x.tok;
  x.workers = x.shared ? sms : 2 * sms;
  x.rows = x.shared ? 2 * kRows : static_cast<int>(std::min(static_cast<int64_t>(kRows), static_cast<int64_t>(T) * G));
  auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
  const size_t rows = 2 * static_cast<size_t>(x.workers) * x.rows;
  x.ml = up(x.workers * sizeof(int4));
  x.o = x.ml + up(rows * sizeof(float2));
  x.total = x.o + up(rows * s.D * sizeof(float));
  return x;
}

template <class C>
pa_status launch(const AttendParams &p, const CUtensorMap &mq, const CUtensorMap &mk,
                 const CUtensorMap &mv, cudaStream_t stream) {
  auto kernel = attend_kernel<C>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  if (launch_pdl(kernel, dim3(p.workers / C::STREAMS), dim3(C::THREADS), C::SMEM, stream, mq, mk, mv, p) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  const dim3 grid(p.workers, C::SHARED ? 8 : 4);
  return launch_pdl(attend_merge_kernel<C::D>, grid, dim3(256), 0, stream, p) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

size_t attend_workspace_bytes(const pa_shape &s, int T, int sms) { return make_plan(s, T, sms).total; }

pa_status run_attend(const pa_shape &s, void *out, const void *q, const int32_t *offsets, int T,
                     const void *k_pool, const void *v_pool, const float *k_scale,
                     const float *v_scale, const int32_t *bt, const int32_t *sl, bool causal,
                     int window, float sm_scale, void *workspace, int sms, int32_t *err,
                     cudaStream_t stream) {
  const Plan plan = make_plan(s, T, sms);
  AttendParams p{};
  p.out = static_cast<uint16_t *>(out);
  p.offsets = offsets;
  p.seq_lens = sl;
  p.block_tables = bt;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.err = err;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.cut = reinterpret_cast<int4 *>(ws);
  p.part_ml = reinterpret_cast<float2 *>(ws + plan.ml);
  p.part_o = reinterpret_cast<float *>(ws + plan.o);
  p.B = s.B;
  p.Hq = s.Hq;
  p.Hkv = s.Hkv;
  p.G = s.Hq / s.Hkv;
  p.T = T;
  p.bs = s.block_size;
  p.max_blocks = s.max_blocks;
  p.nblocks = s.nblocks;
  p.window = window;
  p.causal = causal;
  p.tok = plan.tok;
  p.workers = plan.workers;
  p.rows = plan.rows;
  // c > 0 keeps a masked score's c s at -inf; 1e-30 scores every key alike, as 0 does
  const float c = sm_scale * kLog2e;
  p.c = fmaxf(fabsf(c), 1e-30f);
  p.negate = c < 0.f;
  CUtensorMap mq, mk, mv;
  if (!make_query_map(&mq, q, s, T, plan.tok) || !make_pool_map(&mk, k_pool, s, 1) ||
      !make_pool_map(&mv, v_pool, s, 1))
    return PA_ERR_CUDA;
#define PA_ATTEND(D, KIND)                                                      \
  (plan.shared ? launch<AttendCfg<D, KIND, true>>(p, mq, mk, mv, stream)        \
               : launch<AttendCfg<D, KIND, false>>(p, mq, mk, mv, stream))
  if (s.kv_dtype == PA_KV_FP8_E4M3) return PA_ATTEND(128, PA_KV_FP8_E4M3);
  if (s.kv_dtype == PA_KV_INT4) return PA_ATTEND(128, PA_KV_INT4);
  return s.D == 128 ? PA_ATTEND(128, PA_KV_BF16) : PA_ATTEND(64, PA_KV_BF16);
#undef PA_ATTEND
}

}  // namespace pa
