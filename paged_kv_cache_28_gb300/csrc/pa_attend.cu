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
// bf16 and read from TMEM by the second product.  Each role has its own warps (AttendCfg), and
// they meet at mbarriers only.
//
// What bounds it (D = 128, measured on a GB300):
//   Shared form: a 128 x 128 x 128 product takes the tensor core 512 cycles, so a key tile costs
//   four of them, 2,048; a row tile's softmax takes 870 cycles alone (its 128 exponentials a row
//   at 5.1 cycles a warp) and about 2,000 beside the other's and the products, which read and
//   write the same TMEM.  A key tile takes about 3,300 cycles: the chain S -> softmax -> P V of
//   each row tile, half of it behind the other's.  2,048 tokens after 15,952 cached ones, 64
//   query and 8 KV heads: 0.80-0.82 ms, 1,390-1,431 TFLOP/s, 73-75 % of the measured cuBLAS peak.
//   Separate form: the loads.  32 tokens after 257,000 cached ones: 0.178 ms, 5.9 TB/s, 87 %
//   of the measured copy bandwidth.
//   Code pools: restoring the codes takes issue slots and shared memory from the softmax; a
//   windowed layer over 4-bit pages runs at 950 TFLOP/s.
//
// What made it fast, with the time of the 2,048-token chunk: one warp issuing both row tiles'
// products, 981 us; a warp each, taking turns, 872; P announced at half of the keys instead of at
// three quarters, 835; a piece left in shared memory instead of in the softmax's registers and
// loads issued in a short loop, 800.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>

#include "pa_common.cuh"
#include "pa_extend.h"
#include "pa_internal.h"

namespace pa {
namespace {

constexpr int kKeys = 128;              // keys per tile
constexpr int kRows = 128;              // rows per tile
constexpr int kEarly = 64;              // keys whose weights are announced ahead of the rest
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
  int unit_cost;                        // what a unit costs besides its tiles, in tiles
  uint64_t over_workers;                // 2^64 / workers, rounded up
  float c;                              // |sm_scale| log2(e)
  uint32_t negate;                      // sm_scale < 0: the products take -Q
  bool wide;                            // `out` is 32-byte aligned
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

// Key tiles of unit u (tokens [u S, (u + 1) S) of the sequence): first tile and count.  In the
// stream that is cut into segments a unit is `unit_cost` tiles longer: its start and end take about
// as long as that, and so batches of short and long units balance.
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

// Length of the first u units of one KV head of a sequence in the stream.
__device__ int64_t tiles_before(const AttendParams &p, const Seq &s, int u, int S) {
  if (u == 0) return 0;
  int t0, count;
  if (!p.causal || s.L == 0) {
    unit_tiles(p, s, 0, S, t0, count);
    return static_cast<int64_t>(u) * (count + p.unit_cost);
  }
  int64_t sum = floor_sum(u, S, static_cast<int64_t>(s.base) + S + kKeys - 1) +
                static_cast<int64_t>(u) * p.unit_cost;
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

// A piece of a unit: key tiles [tile, tile + n) of unit tokens [row, row + ntok).
struct Piece {
  int seq, h, row, ntok, pos;  // pos: position of the first token (causal)
  int tile, n;                 // n = 0: no more pieces
  int L, lo;                   // the sequence's keys lie in [lo, L)
  int starts, ends;            // holds the unit's first / last key tile
};

// The stream over a group of 32 sequences, as one warp sees it: lane i holds sequence i.
struct Group {
  Seq s;
  int units;                   // units up to and with this sequence
  int64_t per_head, upto;      // length of one KV head; of the group up to and with this sequence

  __device__ __forceinline__ void load(const AttendParams &p, int group, int S, int lane,
                                       int32_t *err) {
    const int b = group * 32 + lane;
    s = Seq{};
    per_head = 0;
    int U = 0;
    if (b < p.B) {
      s = load_seq(p, b, err);
      U = (s.n + S - 1) / S;
      per_head = tiles_before(p, s, U, S);
    }
    upto = scan64(p.Hkv * per_head, lane);
    units = U * p.Hkv;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, units, d);
      if (lane >= d) units += o;
    }
  }
};

struct GroupSum {
  int64_t upto;
  int64_t units;
};

// The pieces of one worker, in order.
struct Walker {
  int b, h, u, off, U;
  int remaining;
  Seq s;

  // Stand at place `start` of the stream; returns the key tiles before it.  sums: of each group of
  // 32 sequences (where there are more than 32), total: of the batch.
  __device__ __forceinline__ int64_t place(const AttendParams &p, const GroupSum *sums,
                                           const GroupSum &total, Group &group, int64_t start, int S,
                                           int lane) {
    b = h = u = off = U = 0;
    s = Seq{};
    if (start >= total.upto) return total.upto - p.unit_cost * total.units;
    int64_t before = 0, units = 0;
    int g = 0;
    if (p.B > 32) {
      const int groups = (p.B + 31) / 32;
      for (int g0 = 0; g0 < groups; g0 += 32) {
        const bool real = g0 + lane < groups;
        const int64_t v = scan64(real ? sums[g0 + lane].upto : 0, lane);
        const int64_t n = scan64(real ? sums[g0 + lane].units : 0, lane);
        const uint32_t past = __ballot_sync(0xffffffffu, before + v > start);
        const int first = past ? __ffs(past) - 1 : 32;
        if (first > 0) {
          before += shfl64(v, first - 1);
          units += shfl64(n, first - 1);
        }
        g = g0 + first;
        if (past) break;
      }
      group.load(p, g, S, lane, nullptr);
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + group.upto > start);
    const int l = past ? __ffs(past) - 1 : 31;
    b = g * 32 + l;
    s.q0 = __shfl_sync(0xffffffffu, group.s.q0, l);
    s.n = __shfl_sync(0xffffffffu, group.s.n, l);
    s.L = __shfl_sync(0xffffffffu, group.s.L, l);
    s.base = __shfl_sync(0xffffffffu, group.s.base, l);
    s.lo = __shfl_sync(0xffffffffu, group.s.lo, l);
    const int64_t per_head = shfl64(group.per_head, l);
    int64_t r = start - before - (shfl64(group.upto, l) - p.Hkv * per_head);
    U = (s.n + S - 1) / S;
    units += __shfl_sync(0xffffffffu, group.units, l) - p.Hkv * U;
    // the head: at most 2048, so a quotient in fp32 is off by one at most
    h = static_cast<int>(__fdividef(static_cast<float>(r), static_cast<float>(per_head)));
    h = min(h, p.Hkv - 1);
    if (h * per_head > r) --h;
    if (h + 1 < p.Hkv && (h + 1) * per_head <= r) ++h;
    r -= h * per_head;
    int lo = 0, hi = U;                       // the last unit with tiles_before <= r
    int64_t at_lo = 0;
    while (hi - lo > 1) {
      const int step = (hi - lo + 31) / 32;
      const int cand = lo + lane * step;
      const int64_t f = tiles_before(p, s, min(cand, hi), S);
      const int win = 31 - __clz(__ballot_sync(0xffffffffu, cand < hi && f <= r));   // lane 0 holds
      at_lo = shfl64(f, win);
      lo += win * step;
      hi = min(hi, lo + step);
    }
    u = lo;
    off = static_cast<int>(r - at_lo);
    units += h * U + u;
    int t0, count;
    unit_tiles(p, s, u, S, t0, count);
    return start - off - p.unit_cost * units + min(off, count);
  }

  // rest: tiles of the unit after this piece
  __device__ __forceinline__ bool next(const AttendParams &p, int S, Piece &x, int &rest) {
    x.n = 0;
    int t0, count;
    while (true) {
      if (remaining <= 0) return false;
      while (U == 0) {                        // sequences without query tokens
        s = load_seq(p, ++b, nullptr);
        U = (s.n + S - 1) / S;
      }
      unit_tiles(p, s, u, S, t0, count);
      if (off < count) break;
      remaining -= count + p.unit_cost - off;   // the segment begins behind the unit's last tile
      next_unit(p);
    }
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
    rest = count - off;
    x.ends = rest == 0;
    remaining -= x.n + (x.ends ? p.unit_cost : 0);
    if (x.ends) next_unit(p);
    return true;
  }

  __device__ __forceinline__ void next_unit(const AttendParams &p) {
    off = 0;
    if (++u == U) {
      u = 0;
      if (++h == p.Hkv) {
        h = 0;
        U = 0;                                // the next sequence is read when it is wanted
      }
    }
  }
};

// ------------------------------------------------------------------ tcgen05

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// The same, and the 32 registers are not read before it.
#define PA_W8(r, o) "+r"(r[o]), "+r"(r[o + 1]), "+r"(r[o + 2]), "+r"(r[o + 3]), "+r"(r[o + 4]), \
                    "+r"(r[o + 5]), "+r"(r[o + 6]), "+r"(r[o + 7])
__device__ __forceinline__ void tc_wait_ld32(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : PA_W8(r, 0), PA_W8(r, 8), PA_W8(r, 16), PA_W8(r, 24)::"memory");
}
__device__ __forceinline__ void tc_use32(uint32_t *r) {   // orders reads of r after the wait above it
  asm volatile("" : PA_W8(r, 0), PA_W8(r, 8), PA_W8(r, 16), PA_W8(r, 24)::"memory");
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

// 32 bytes to global memory; wide: the address is 32-byte aligned, and a whole sector goes at once
__device__ __forceinline__ void store32(void *dst, const uint32_t *v, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), PA_I8(v, 0)
                 : "memory");
  } else {
    reinterpret_cast<uint4 *>(dst)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<uint4 *>(dst)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
  return one != 0;
}

// One look at a barrier: whether the phase with the given parity is complete.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// mbar_wait for the warps that everything else waits for: they look again at once, where try_wait
// may put the warp to sleep and wake it late.
__device__ __forceinline__ bool mbar_spin(uint32_t bar, uint32_t parity) {
  for (uint32_t it = 0; it < 16 * kWaitSpins; ++it)
    if (mbar_test(bar, parity)) return true;
  return false;
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

__device__ __forceinline__ float2 lds_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
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

// The codes of a tile's kTokens tokens (as TMA swizzled them) to rows of a bf16 tile (128-byte
// swizzle), by kWarps warps.
// Neighbouring lanes write both 64-column halves of a row at once; the order of a lane's stores
// keeps the two halves off each other's banks.
template <int KIND, int kTokens, int kWarps>
__device__ __forceinline__ void restore_tile(uint32_t raw, uint32_t dst, int w, int lane) {
  if constexpr (KIND == PA_KV_FP8_E4M3) {
    constexpr int kSteps = kTokens / 4 / kWarps;         // of four rows
    const int c = lane & 7;                              // 16 codes: columns [16 c, 16 c + 16)
    {
      uint4 v[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = (i * kWarps + w) * 4 + (lane >> 3);
        v[i] = lds128(raw + r * 128 + ((c ^ (r & 7)) << 4));
      }
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int r = (i * kWarps + w) * 4 + (lane >> 3);
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
    constexpr int kSteps = kTokens / 8 / kWarps;         // of eight rows
    const int c = lane & 3;                              // 32 codes: columns [32 c, 32 c + 32)
    uint4 v[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = (i * kWarps + w) * 8 + (lane >> 2);
      v[i] = lds128(raw + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int r = (i * kWarps + w) * 8 + (lane >> 2);
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

// Step j of a stream of n tiles: the products with V of tile j - 1, then those with K of tile j.
// Its ring holds K and V tiles in turn: tile j's are its 2 j-th and the one after.  Every warp that
// fills or reads a ring goes through all of its tiles in this order: a barrier's parity tells its
// phase only from the phases next to it.
struct RingOrder {
  int n, j;
  __device__ __forceinline__ bool more() const { return j <= n && n > 0; }
  __device__ __forceinline__ bool v() const { return j > 0; }
  __device__ __forceinline__ bool k() const { return j < n; }
  __device__ __forceinline__ uint32_t v_at() const { return 2 * j - 1; }
  __device__ __forceinline__ uint32_t k_at() const { return 2 * j; }
};

// kKind: the pools' pa_kv_dtype.  Codes (D = 128) are restored to bf16 tiles, without their scale,
// by eight warps of their own: K's scale multiplies the scores of a page, V's its weights.
template <int kD, int kKind, bool kShared>
struct AttendCfg {
  static constexpr int D = kD, KIND = kKind;
  static constexpr bool SHARED = kShared, QUANT = kKind != PA_KV_BF16;
  static constexpr int HALVES = D / 64;                 // 128-byte column chunks of a bf16 row
  static constexpr int TILE = kKeys * D * 2;            // bytes of a Q, K or V tile
  static constexpr int CODE_ROW = KIND == PA_KV_INT4 ? 64 : 128;
  // code tiles come in halves where their ring is short
  static constexpr int SPLIT = KIND == PA_KV_FP8_E4M3 && !kShared ? 2 : 1;
  static constexpr int RAW_TILE = kKeys * CODE_ROW / SPLIT;
  // the rings of K and V tiles, one per stream; code pools: rings of code tiles before them (at most
  // 224 KB with Q)
  static constexpr int STAGES =
      D == 64 ? 12 : !kShared ? 4 : KIND == PA_KV_BF16 ? 5 : KIND == PA_KV_FP8_E4M3 ? 3 : 4;
  static constexpr int RAW = QUANT ? 4 : 1;
  static constexpr int RING = 2 * TILE;                 // after the two Q tiles
  static constexpr int RAW_RING = RING + STAGES * TILE;
  static constexpr int SMEM = RAW_RING + (QUANT ? RAW * RAW_TILE : 0) + 1024;
  // Warps 0-7 softmax.  Then the products (a warp for each row tile, so that one's waits are
  // filled by the other's products), the pieces and the loads (separate form: both, of a stream
  // each) and, for code pools, eight that restore codes.  Registers are dealt anew by groups of
  // four warps: 384 threads start with 168, 64,512 in all = 256 x 216 + 128 x 72, and a softmax
  // thread holds its row's 128 scores; 640 with 96, 61,440 = 256 x 144 + 384 x 64, and it reads
  // half of them twice.
  static constexpr int THREADS = QUANT ? 640 : 384;
  static constexpr int MMA_WARP = 8, PIECE_WARP = 10, LOAD_WARP = 11;
  static constexpr int CODE_WARP = 12, CODE_WARPS = 8;  // code pools
  static constexpr int SOFTMAX_REGS = QUANT ? 144 : 216, OTHER_REGS = QUANT ? 64 : 72;
  static constexpr int STREAMS = SHARED ? 1 : 2;        // key streams of a CTA
  static constexpr int PER = STAGES / STREAMS;          // ring stages of a stream
  static constexpr int RAW_PER = QUANT ? RAW / STREAMS : 1;
  static constexpr int RESTORERS = CODE_WARPS / STREAMS;   // warps that restore a stream's codes
  static constexpr int PIECES = 6;                      // pieces known ahead per stream
  static constexpr int SCALES = 5;                      // tiles whose scales are held per stream
  // the scales of tile j + SCALES are stored before its K is issued; by then the copies have
  // come 2 (SCALES - 1) past V of tile j, which must be further than both rings hold
  static_assert(!QUANT || 2 * (SCALES - 1) >= RAW_PER / SPLIT + PER, "scales overwritten too early");
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    attend_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const AttendParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kTileBars = 2 * C::STAGES, kClean = 8, kPieceBars = kTileBars + 14 + kClean;
  constexpr int kRawBars = kPieceBars + 2 * C::STREAMS * C::PIECES;
  constexpr int kBars = kRawBars + (C::QUANT ? 2 * C::RAW + C::STREAMS * C::SCALES : 0);
  __shared__ __align__(8) uint64_t bars[kBars];
  __shared__ Piece pieces[C::STREAMS][C::PIECES];
  __shared__ Walker places[C::STREAMS + 1];              // the bounds of this CTA's segments
  __shared__ int64_t tiles_at[C::STREAMS + 1];
  __shared__ int segment_width;
  __shared__ uint32_t tmem_slot;
  // scales of the tiles on their way: K's pages (16 tokens each), then V's
  __shared__ float4 scales[C::STREAMS][C::QUANT ? C::SCALES : 1][4];
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t sm = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  // K or V tile k of a stream: in shared memory / no longer needed
  auto kv_stage = [](int st, uint32_t k) { return st * C::PER + k % C::PER; };
  auto kv_full = [&](int st, uint32_t k) { return bar0 + 8 * kv_stage(st, k); };
  auto kv_empty = [&](int st, uint32_t k) { return bar0 + 8 * (C::STAGES + kv_stage(st, k)); };
  auto kv_parity = [](uint32_t k) { return (k / C::PER) & 1; };
  auto q_full = [&](int t) { return bar0 + 8 * (kTileBars + t); };
  auto s_full = [&](int t) { return bar0 + 8 * (kTileBars + 2 + t); };
  auto p_early = [&](int t) { return bar0 + 8 * (kTileBars + 4 + t); };
  auto p_ready = [&](int t) { return bar0 + 8 * (kTileBars + 6 + t); };
  auto o_full = [&](int t) { return bar0 + 8 * (kTileBars + 8 + t); };
  auto done_bar = [&](int t) { return bar0 + 8 * (kTileBars + 10 + t); };
  // the i-th V tile with rows that one product warp clears for both (shared form); the ring holds
  // fewer such tiles than there are barriers
  static_assert(C::PER / 2 + 1 < kClean, "a barrier of cleared tiles reused too early");
  auto clean = [&](uint32_t i) { return bar0 + 8 * (kTileBars + 12 + i % kClean); };
  // row tile t's turn at the tensor core (shared form)
  auto turn = [&](int t) { return bar0 + 8 * (kTileBars + 12 + kClean + t); };
  // piece k of a stream is known / no longer needed
  auto pc_full = [&](int st, uint32_t k) {
    return bar0 + 8 * (kPieceBars + st * C::PIECES + k % C::PIECES);
  };
  auto pc_empty = [&](int st, uint32_t k) {
    return bar0 + 8 * (kPieceBars + (C::STREAMS + st) * C::PIECES + k % C::PIECES);
  };
  auto pc_parity = [](uint32_t k) { return (k / C::PIECES) & 1; };
  // code pools: code tiles landed / restored, scales of a stream's tile n stored
  auto raw_stage = [](int st, uint32_t k) { return st * C::RAW_PER + k % C::RAW_PER; };
  auto raw_full = [&](int st, uint32_t k) { return bar0 + 8 * (kRawBars + raw_stage(st, k)); };
  auto raw_empty = [&](int st, uint32_t k) { return bar0 + 8 * (kRawBars + C::RAW + raw_stage(st, k)); };
  auto raw_parity = [](uint32_t k) { return (k / C::RAW_PER) & 1; };
  auto sc_full = [&](int st, uint32_t n) {
    return bar0 + 8 * (kRawBars + 2 * C::RAW + st * C::SCALES + n % C::SCALES);
  };
  auto sc_parity = [](uint32_t n) { return (n / C::SCALES) & 1; };
  const int S = C::SHARED ? 2 * p.tok : p.tok;

  if (tid == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(bar0 + 8 * i, C::QUANT ? C::RESTORERS * C::SPLIT : 1);  // kv_full: the warps that fill it
      mbar_init(bar0 + 8 * (C::STAGES + i), C::SHARED ? 2 : 1);  // kv_empty: the product warps
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(s_full(t), 1);
      mbar_init(p_early(t), 4);
      mbar_init(p_ready(t), 4);
      mbar_init(o_full(t), 1);
      mbar_init(done_bar(t), 1);
      mbar_init(turn(t), 1);
    }
    for (int i = 0; i < kClean; ++i) mbar_init(clean(i), 1);
    for (int st = 0; st < C::STREAMS; ++st)
      for (int k = 0; k < C::PIECES; ++k) {
        mbar_init(pc_full(st, k), 1);
        mbar_init(pc_empty(st, k), C::SHARED ? 1 + 2 + 8 : 1 + 4);     // every reader
      }
    if constexpr (C::QUANT) {
      for (int i = 0; i < C::RAW; ++i) {
        mbar_init(bar0 + 8 * (kRawBars + i), 1);                     // raw_full
        mbar_init(bar0 + 8 * (kRawBars + C::RAW + i), C::RESTORERS);  // raw_empty
      }
      for (int st = 0; st < C::STREAMS; ++st)
        for (int n = 0; n < C::SCALES; ++n) mbar_init(sc_full(st, n), 1);
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

  // Every CTA lays out the batch's tiles.  Past 32 sequences all warps do, one sum per group of 32,
  // in the space of the ring; then a warp for each bound of this CTA's segments finds its place.
  GroupSum *sums = reinterpret_cast<GroupSum *>(smem_raw + (sm - smem_u32(smem_raw)) + C::RING);
  const int groups = (p.B + 31) / 32;
  int32_t *report = blockIdx.x == 0 ? p.err : nullptr;
  if (groups > 1) {
    for (int g = warp; g < groups; g += C::THREADS / 32) {
      Group x;
      x.load(p, g, S, lane, report);
      if (lane == 31) sums[g] = GroupSum{x.upto, x.units};
    }
    __syncthreads();
  }
  if (warp >= 8 && warp <= 8 + C::STREAMS) {
    Group group;
    GroupSum total{0, 0};
    if (groups == 1) {
      group.load(p, 0, S, lane, warp == 8 ? report : nullptr);
      total = GroupSum{shfl64(group.upto, 31), __shfl_sync(0xffffffffu, group.units, 31)};
    } else {
      for (int g = lane; g < groups; g += 32) {
        total.upto += sums[g].upto;
        total.units += sums[g].units;
      }
      total.upto = shfl64(scan64(total.upto, lane), 31);
      total.units = shfl64(scan64(total.units, lane), 31);
    }
    const int64_t width = p.workers == 1 ? total.upto
                                         : static_cast<int64_t>(__umul64hi(
                                               static_cast<uint64_t>(total.upto + p.workers - 1),
                                               p.over_workers));
    const int64_t start = (static_cast<int64_t>(blockIdx.x) * C::STREAMS + warp - 8) * width;
    Walker w;
    const int64_t tiles = w.place(p, sums, total, group, start, S, lane);
    w.remaining = static_cast<int>(max(static_cast<int64_t>(0), min(width, total.upto - start)));
    if (lane == 0) {
      places[warp - 8] = w;
      tiles_at[warp - 8] = tiles;
      if (warp == 8) segment_width = static_cast<int>(width);
    }
  }
  fence_proxy_async();                                   // the sums' space is TMA's from here
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  bool ok = true;
  // the next piece of a stream, for one of the warps that read them; false after the last
  auto read_piece = [&](int st, uint32_t k, Piece &x) {
    ok = ok && mbar_wait(pc_full(st, k), pc_parity(k));
    if (!ok) return false;
    x = pieces[st][k % C::PIECES];
    __syncwarp();
    if (lane == 0) mbar_arrive(pc_empty(st, k));
    return x.n > 0;
  };
  auto ring_order = [&](int st) {
    return RingOrder{static_cast<int>(tiles_at[st + 1] - tiles_at[st]), 0};
  };

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
    auto done_with = [&](uint32_t k) {
      __syncwarp();
      if (lane == 0) mbar_arrive(pc_empty(st, k));
    };
    for (uint32_t k = 0;; ++k) {
      ok = ok && mbar_wait(pc_full(st, k), pc_parity(k));
      if (!ok) break;
      // the piece stays where it is until its rows are written, rather than in registers
      const Piece &x = pieces[st][k % C::PIECES];
      const int n_tiles = x.n, tile_0 = x.tile;
      if (n_tiles == 0) break;
      [[maybe_unused]] const uint32_t tile0 = tiles;
      tiles += n_tiles;
      const int ntok = min(p.tok, x.ntok - tok0);        // tokens of this tile
      if (ntok <= 0) {
        done_with(k);
        continue;
      }
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
      // A barrier's parity tells its phase only from the ones next to it, and a row tile has not
      // followed the scales of pieces that it had no part in.  Once S of a piece's first tile is
      // there its scales are the last ones stored in their place, and they stay until the tile's
      // weights are out (see SCALES); from then on this row tile keeps up.
      if constexpr (C::QUANT && C::SHARED) ok = mbar_wait(s_full(t), s_phase);
      for (int i = 0; i < n_tiles; ++i) {
        const int key0 = (tile_0 + i) * kKeys;
        // code pools: the scales of the tile's pages, K's then V's
        [[maybe_unused]] uint32_t sc = 0;
        if constexpr (C::QUANT) {
          const uint32_t n = tile0 + i;
          ok = ok && mbar_wait(sc_full(st, n), sc_parity(n));
          sc = smem_u32(scales[st][n % C::SCALES]);
        }
        ok = ok && mbar_wait(s_full(t), s_phase);
        if (!ok) break;
        s_phase ^= 1;
        if (i == n_tiles - 1 && row == 0) {
          // the products with this Q tile are done: the next piece's may come, if this row tile has
          // part in it
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
          const bool edge = key0 < all_lo || key0 + kKeys > all_hi;
          const int first = lo - key0;                   // columns [first, first + seen) count
          const unsigned seen = static_cast<unsigned>(max(0, hi - lo));
          auto hide = [&](uint32_t *s, int j0) {         // columns [j0, j0 + 32) of the row
            if (edge) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (static_cast<unsigned>(j0 + j - first) >= seen) s[j] = __float_as_uint(-INFINITY);
            }
          };
          // what the scores of a block's two pages are multiplied by
          auto k_factors = [&](int block) {
            return C::QUANT ? lds_f32x2(sc + 8 * block) : make_float2(p.c, p.c);
          };
          float mx[2] = {-INFINITY, -INFINITY};
          auto maximum = [&](const uint32_t *s, float2 f) {   // of a block of 32 columns
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
              float y[2] = {-INFINITY, -INFINITY};
#pragma unroll
              for (int e = j; e < j + 16; e += 4) {
                y[0] = fmaxf(y[0], fmaxf(__uint_as_float(s[e]), __uint_as_float(s[e + 1])));
                y[1] = fmaxf(y[1], fmaxf(__uint_as_float(s[e + 2]), __uint_as_float(s[e + 3])));
              }
              const float page = fmaxf(y[0], y[1]);
              mx[j / 16] = fmaxf(mx[j / 16], C::QUANT ? page * (j ? f.y : f.x) : page);
            }
          };
          // A block of 32 columns is on its way while another is worked on.  bf16 pools: the row's
          // scores stay in registers; code pools, whose threads have fewer, read half of them twice.
          uint32_t s[C::QUANT ? 64 : kKeys];
          if constexpr (C::QUANT) {
#pragma unroll 1
            for (int j = 2; j >= 0; j -= 2) {            // blocks j and j + 1
              tc_ld32(s, tS + 32 * j);
              tc_ld32(s + 32, tS + 32 * j + 32);
              const float2 f0 = k_factors(j), f1 = k_factors(j + 1);
              tc_wait_ld32(s);
              tc_use32(s + 32);
              hide(s, 32 * j);
              maximum(s, f0);
              hide(s + 32, 32 * j + 32);
              maximum(s + 32, f1);
            }
          } else {
            tc_ld32(s, tS);
            tc_ld32(s + 32, tS + 32);
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              tc_wait_ld32(s + 64 * half);
              tc_use32(s + 64 * half + 32);
              if (half == 0) {
                tc_ld32(s + 64, tS + 64);
                tc_ld32(s + 96, tS + 96);
              }
#pragma unroll
              for (int j = 64 * half; j < 64 * half + 64; j += 32) {
                hide(s + j, j);
                maximum(s + j, make_float2(1.f, 1.f));
              }
            }
          }
          const float top = fmaxf(mx[0], mx[1]) * (C::QUANT ? 1.f : p.c);
          if (m == -INFINITY) m = top;                   // O and l are zero so far
          // the reference moves only past kMaxJump octaves: weights stay below 2^8, far
          // inside bf16 and fp32, and O is seldom rescaled
          const bool jump = live && l > 0.f && top > m + kMaxJump;
          if (__any_sync(0xffffffffu, jump)) {
            const float g = jump ? ex2(m - top) : 1.f;
            if (jump) m = top;
            l *= g;
#pragma unroll 1
            for (int j = 0; j < C::D; j += 32) {
              uint32_t o[32];
              tc_ld32(o, tO + j);
              tc_wait_ld32(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * g);
              tc_st32(tO + j, o);
            }
          }
          const float neg = m == -INFINITY ? 0.f : -m;
          // The weights of block j, over columns that are already read.  Code pools: V's scale enters
          // in the exponent, and leaves the sums of its page again.
          float2 sum[2] = {};
          auto weights = [&](const uint32_t *s, int j, float2 f) {
            float2 v = make_float2(0.f, 0.f);
            if constexpr (C::QUANT) v = lds_f32x2(sc + 32 + 8 * j);
            uint32_t packed[16];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const float c1 = half ? f.y : f.x, lv = half ? v.y : v.x;
              const float2 shift = make_float2(neg + lv, neg + lv);
              float2 page[2] = {};
#pragma unroll
              for (int e = 8 * half; e < 8 * half + 8; ++e) {
                float2 y = fma2(make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])),
                                make_float2(c1, c1), shift);
                y.x = ex2(y.x);
                y.y = ex2(y.y);
                float2 &to = C::QUANT ? page[e & 1] : sum[e & 1];
                to = add2(to, y);
                packed[e] = pack_bf16(y.x, y.y);
              }
              if constexpr (C::QUANT) {
                const float back = ex2(-lv);
                sum[half] = fma2(add2(page[0], page[1]), make_float2(back, back), sum[half]);
              }
            }
            tc_st16(tS + 16 * j, packed);
            if (j == kEarly / 32 - 1) {
              tc_wait_st();
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(p_early(t));    // the second product may begin
            }
          };
          if constexpr (C::QUANT) {
            // (the separate form in a loop: its few tiles a CTA wait for instructions first of all)
#pragma unroll(C::SHARED ? 2 : 1)
            for (int j = 0; j < 4; j += 2) {
              const float2 f0 = k_factors(j), f1 = k_factors(j + 1);
              if (j > 0) {
                tc_wait_ld32(s);
                tc_use32(s + 32);
                hide(s, 64);
                hide(s + 32, 96);
              }
              weights(s, j, f0);
              if (j == 0) tc_ld32(s, tS + 64);           // columns that are not written over yet
              weights(s + 32, j + 1, f1);
              if (j == 0) tc_ld32(s + 32, tS + 96);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) weights(s + 32 * j, j, make_float2(p.c, p.c));
          }
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready(t));
          const float2 both = add2(sum[0], sum[1]);
          l += both.x + both.y;
        } else {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(p_early(t));
            mbar_arrive(p_ready(t));
          }
        }
      }
      if (!ok) break;
      ok = mbar_wait(o_full(t), o_phase);
      if (!ok) break;
      o_phase ^= 1;
      tc_fence_after();
      if (warp_live) {
        const bool whole = x.starts && x.ends;
        // a row without keys has l = 0 and gives zeros; a NaN in its query gives NaN
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint16_t *dst = p.out + (static_cast<int64_t>(x.row + tok0 + my_tok) * p.Hq + x.h * p.G +
                                 (row - my_tok * p.G)) * C::D;
        const int64_t r = (2 * static_cast<int64_t>(blockIdx.x * C::STREAMS + st) + x.starts) * p.rows +
                          (C::SHARED ? t * kRows : 0) + row;
        float *part = p.part_o + r * C::D;
        if (!whole && live) p.part_ml[r] = make_float2(m, l);
#pragma unroll
        for (int j = 0; j < C::D; j += 32) {
          uint32_t o[32];
          tc_ld32(o, tO + j);
          tc_wait_ld32(o);
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = l == 0.f ? 0u
                              : pack_bf16(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            if (live) {
              store32(dst + j, o, p.wide);
              store32(dst + j + 16, o + 8, p.wide);
            }
          } else if (live) {
#pragma unroll
            for (int e = 0; e < 4; ++e) store32(part + j + 8 * e, o + 8 * e, true);
          }
        }
      }
      tc_fence_before();
      done_with(k);
    }
    // after a wait that gave up, a Q tile may still be arriving
    if (!ok && row == 0)
      for (uint32_t k = q_used > 0 ? q_used - 1 : 0; k < q_loads; ++k) mbar_wait(q_full(t), k & 1);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    // make a piece known to its stream's readers
    auto publish = [&](int st, uint32_t k, const Piece &x) {
      ok = ok && mbar_wait(pc_empty(st, k), pc_parity(k) ^ 1);
      if (ok && lane == 0) {
        pieces[st][k % C::PIECES] = x;
        mbar_arrive(pc_full(st, k));
      }
    };
    auto cut_after = [&](const Piece &x, int rest) {
      return make_int4(x.row, x.ntok, x.h, (rest - 1) / segment_width + 1);
    };
    if (C::SHARED && warp == C::PIECE_WARP) {
      // ---------------------------------------------------------------- the pieces of the stream
      Walker walk = places[0];
      int4 cut = make_int4(0, 0, 0, 0);
      bool more = true;
#pragma unroll 1
      for (uint32_t k = 0; more && ok; ++k) {
        Piece x;
        int rest = 0;
        more = walk.next(p, S, x, rest);
        publish(0, k, x);
        if (more && x.starts && !x.ends) cut = cut_after(x, rest);
      }
      if (lane == 0) p.cut[blockIdx.x] = cut;
    } else if (warp == C::LOAD_WARP || (!C::SHARED && warp == C::PIECE_WARP)) {
      // ---------------------------------------------------------------- K and V tiles of a stream
      // (separate form: this warp walks its stream's pieces, too)
      const int st = C::SHARED ? 0 : warp - C::PIECE_WARP;
      // One box per 16 tokens (a page of a tile) and, in bf16 pools, 64 columns.
      constexpr int kBox = C::QUANT ? 16 * C::CODE_ROW : 16 * 128;
      constexpr int kRing = C::QUANT ? C::RAW_PER : C::PER, kPages = 8 / C::SPLIT;
      const int outside = p.nblocks * p.bs;              // a row past the pool reads zeros
      Walker walk;
      int4 cut = make_int4(0, 0, 0, 0);
      if (!C::SHARED) walk = places[st];
      Piece x;
      x.n = 0;
      int at = 0;                                        // tiles of x that are fetched
      uint32_t seen = 0;
      bool over = false;
      auto next_piece = [&] {
        if constexpr (C::SHARED) {
          return read_piece(st, seen++, x);
        } else {
          int rest = 0;
          const bool more = walk.next(p, S, x, rest);
          publish(st, seen++, x);
          if (more && x.starts && !x.ends) cut = cut_after(x, rest);
          return more && ok;
        }
      };
      // Block ids come four tiles (32 runs of 16 tokens, one per lane) at a time, two such chunks
      // ahead of the copies; scales one.
      struct Chunk {
        int h, tile, n;                                  // n = 0: none
        int row;                                         // this lane's first pool row; -1: unseen
        float ks, vs;
      };
      auto fetch_chunk = [&] {
        Chunk c{};
        if (!over && at == x.n) {
          over = !next_piece();
          at = 0;
        }
        if (over) return c;
        c.h = x.h;
        c.tile = x.tile + at;
        c.n = min(4, x.n - at);
        at += c.n;
        c.row = -1;
        const int g = c.tile * kKeys + 16 * lane;
        if (g < x.L && g + 16 > x.lo && lane < 8 * c.n) {
          // (as unsigned, a negative id is past every pool)
          const uint32_t id = p.block_tables[static_cast<int64_t>(x.seq) * p.max_blocks + g / p.bs];
          c.row = static_cast<int>(min(id, 0x7fffffffu));
        }
        return c;
      };
      // block id to pool row (and the scales on their way), when it has come
      auto resolve = [&](Chunk &c) {
        c.ks = c.vs = 0.f;
        if (c.row >= 0) {
          if (c.row < p.nblocks) {
            if constexpr (C::QUANT) {
              const int64_t i = static_cast<int64_t>(c.row) * p.Hkv + c.h;
              c.ks = p.k_scale[i];
              c.vs = p.v_scale[i];
            }
            c.row = c.row * p.bs + (c.tile * kKeys + 16 * lane) % p.bs;
          } else {
            set_err(p.err, PA_DEVERR_BLOCK_ID);
            c.row = outside;
          }
        }
      };
      // tile (or part of a tile) u of the ring that this warp fills
      auto full_bar = [&](uint32_t u) { return C::QUANT ? raw_full(st, u) : kv_full(st, u); };
      const uint32_t all = 2 * C::SPLIT * ring_order(st).n;
      Chunk cur = fetch_chunk(), nxt = fetch_chunk();
      resolve(cur);
      int next = 0, here = 0;                            // the chunk's next tile, and the one at hand
      uint32_t tiles = 0, u = 0;
#pragma unroll 1
      for (; ok && u < all; ++u) {
        const uint32_t k = u / C::SPLIT;
        const int first = static_cast<int>(u % C::SPLIT) * kPages;
        ok = mbar_wait(C::QUANT ? raw_empty(st, u) : kv_empty(st, u), ((u / kRing) & 1) ^ 1);
        if (!ok) break;
        const bool v = k & 1;
        if (!v && first == 0) {
          if (next == cur.n) {
            cur = nxt;
            resolve(cur);
            nxt = fetch_chunk();
            next = 0;
            if (!ok) break;
          }
          here = next++;
          if constexpr (C::QUANT) {
            float *sc = reinterpret_cast<float *>(scales[st][tiles % C::SCALES]);
            if ((lane >> 3) == here) {
              // c times K's scale and log2 of V's, both kept above zero: a zero scale's codes add
              // nothing, and -inf stays -inf
              sc[lane & 7] = fmaxf(cur.ks * p.c, 1e-30f);
              sc[8 + (lane & 7)] = __log2f(fmaxf(cur.vs, 1e-30f));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(sc_full(st, tiles));
            ++tiles;
          }
        }
        // pages of V that no token sees read zeros (bf16): a weight of 0 times what lies there must
        // be 0; codes are never infinite or NaN once restored
        const bool zeros = !C::QUANT && v;
        const uint32_t seen_pages =
            (__ballot_sync(0xffffffffu, cur.row >= 0 || zeros) >> (8 * here + first)) & ((1u << kPages) - 1u);
        const bool leader = elect_one();
        const uint32_t full = full_bar(u);
        if (leader)
          mbar_arrive_expect_tx(full, __popc(seen_pages) * kBox * (C::QUANT ? 1 : C::HALVES));
        const CUtensorMap *map = v ? &tmV : &tmK;
        const uint32_t dst = C::QUANT ? sm + C::RAW_RING + raw_stage(st, u) * C::RAW_TILE
                                      : sm + C::RING + kv_stage(st, u) * C::TILE;
        const int column = cur.h * (C::QUANT ? C::CODE_ROW : C::D);
#pragma unroll 4
        for (int page = 0; page < kPages; ++page) {
          int row = __shfl_sync(0xffffffffu, cur.row, 8 * here + first + page);
          if (!(seen_pages >> page & 1)) continue;
          if (row < 0) row = outside;
          if (leader) {
#pragma unroll
            for (int half = 0; half < (C::QUANT ? 1 : C::HALVES); ++half)
              tma_load_2d(dst + half * (kKeys * 128) + page * kBox, map, column + half * 64, row, full);
          }
        }
        __syncwarp();
      }
      if (!C::SHARED) {
        while (ok && !over) fetch_chunk();               // the end mark
        if (lane == 0) p.cut[2 * blockIdx.x + st] = cut;
      }
      // after a wait that gave up, the copies in flight must have landed before the CTA's memory goes
      if (!ok)
        for (uint32_t i = u > kRing ? u - kRing : 0; i < u; ++i) mbar_wait(full_bar(i), (i / kRing) & 1);
    } else if (C::QUANT && warp >= C::CODE_WARP) {
      // ---------------------------------------------------------------- codes to bf16 tiles
      const int st = (warp - C::CODE_WARP) / C::RESTORERS, w = (warp - C::CODE_WARP) % C::RESTORERS;
      const uint32_t all = 2 * C::SPLIT * ring_order(st).n;
      for (uint32_t u = 0; ok && u < all; ++u) {
        const uint32_t k = u / C::SPLIT, part = u % C::SPLIT;
        ok = mbar_wait(raw_full(st, u), raw_parity(u)) &&
             (part > 0 || mbar_wait(kv_empty(st, k), kv_parity(k) ^ 1));
        if (!ok) break;
        restore_tile<C::KIND, kKeys / C::SPLIT, C::RESTORERS>(
            sm + C::RAW_RING + raw_stage(st, u) * C::RAW_TILE,
            sm + C::RING + kv_stage(st, k) * C::TILE + part * (kKeys / C::SPLIT * 128), w, lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(raw_empty(st, u));
          mbar_arrive(kv_full(st, k));
        }
      }
    } else if (warp < C::MMA_WARP + 2) {
      // ---------------------------------------------------------------- matrix products
      const int t = warp - C::MMA_WARP, st = C::SHARED ? 0 : t;      // this warp's row tile and stream
      const uint32_t idS = mma_desc(kKeys, false) | (p.negate ? kNegateA : 0u);
      constexpr uint32_t idO = mma_desc(C::D, true);
      const uint64_t q_desc = smem_desc(sm, 16, 1024);
      const uint64_t k_desc = smem_desc(sm + C::RING, 16, 1024);
      const uint64_t v_desc = smem_desc(sm + C::RING, kKeys * 128, 1024);
      struct {
        Piece x;
        int i;                                           // the piece's tile that K is due of
        uint32_t piece, q_phase, p_phase;
        // the tile that V is due of: first / last of its piece, the rows [lo, hi) of it that some
        // token sees, whether this row tile has part in it
        bool first, last, mine;
        int lo, hi;
      } y{};
      uint32_t cleared = 0;
      // Shared form: the row tiles take turns at the tensor core, O_t += P_t V and the next S_t at a
      // time.  Left to themselves their products would run interleaved and end together, and then
      // both softmaxes would run while the tensor core waits.
      // A barrier is slow to look at while the tensor core reads shared memory, so everything but
      // the weights' last part is waited for ahead of the turn, and the turn goes on while the last
      // products are still being issued.
      uint32_t turns = 0;
      if (C::SHARED && t == 1 && lane == 0) mbar_arrive(turn(0));
      const uint32_t tS = tmem + t * kKeys, tO = tmem + 256 + t * 128;
      for (RingOrder r = ring_order(st); ok && r.more(); ++r.j) {
        const bool v = r.v(), k = r.k();
        const uint32_t v_at = r.v_at(), k_at = r.k_at();
        const bool o_first = y.first, o_last = y.last, do_o = v && y.mine;
        if (v) {
          ok = ok && mbar_spin(kv_full(st, v_at), kv_parity(v_at));
          // rows next to the seen ones in their page may hold anything
          const int head = C::QUANT || y.lo <= 0 ? 0 : y.lo & 15;
          const int tail = C::QUANT || y.hi >= kKeys || y.hi <= 0 ? 0 : -y.hi & 15;
          if (ok && head + tail > 0) {
            if (!C::SHARED || t == 0) {
              const uint32_t tile = sm + C::RING + kv_stage(st, v_at) * C::TILE;
              for (int e = lane; e < (head + tail) * 8 * C::HALVES; e += 32) {
                const int n = e / (8 * C::HALVES), chunk = e % (8 * C::HALVES);
                const int row = n < head ? y.lo - head + n : y.hi + n - head;
                sts128(tile + (chunk >> 3) * (kKeys * 128) + row * 128 + (chunk & 7) * 16,
                       make_uint4(0, 0, 0, 0));
              }
              fence_proxy_async();
              __syncwarp();
              if (C::SHARED && lane == 0) mbar_arrive(clean(cleared));
            } else {
              ok = mbar_wait(clean(cleared), (cleared / kClean) & 1);
            }
            ++cleared;
          }
        }
        if (k) {
          if (y.i == y.x.n) {
            read_piece(st, y.piece++, y.x);
            y.i = 0;
          }
          y.mine = !C::SHARED || t == 0 || y.x.ntok > p.tok;
          y.first = y.i == 0;
          y.last = y.i == y.x.n - 1;
          y.lo = y.x.lo - (y.x.tile + y.i) * kKeys;
          y.hi = y.x.L - (y.x.tile + y.i) * kKeys;
          ++y.i;
          ok = ok && mbar_spin(kv_full(st, k_at), kv_parity(k_at));
          if (y.mine && y.first) {
            ok = ok && mbar_spin(q_full(t), y.q_phase);
            y.q_phase ^= 1;
          }
        }
        const bool do_s = k && y.mine;
        if (do_o) ok = ok && mbar_spin(p_early(t), y.p_phase);
        if (C::SHARED) ok = ok && mbar_spin(turn(t), turns++ & 1);
        if (do_o) {                                    // O_t += P_t V
          const uint64_t b = v_desc + kv_stage(st, v_at) * (C::TILE >> 4);
          if (ok) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int e = 0; e < kEarly / 16; ++e)
                tc_mma_ts(tO, tS + e * 8, b + ((e * 16 * 128) >> 4), idO, !o_first || e > 0);
            }
            __syncwarp();
            ok = mbar_spin(p_ready(t), y.p_phase);
          }
          y.p_phase ^= 1;
          if (ok) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int e = kEarly / 16; e < kKeys / 16; ++e)
                tc_mma_ts(tO, tS + e * 8, b + ((e * 16 * 128) >> 4), idO, 1);
              if (o_last) tc_commit(o_full(t));
              tc_commit(kv_empty(st, v_at));
            }
            __syncwarp();
          }
        } else if (v && ok && lane == 0) {
          mbar_arrive(kv_empty(st, v_at));
        }
        if (do_s) {                                    // S_t = Q_t K^T
          if (ok && elect_one()) {
            const uint64_t a = q_desc + t * (C::TILE >> 4);
            const uint64_t b = k_desc + kv_stage(st, k_at) * (C::TILE >> 4);
#pragma unroll
            for (int e = 0; e < C::D / 16; ++e) {
              if (C::SHARED && e == C::D / 32) mbar_arrive(turn(t ^ 1));
              const uint32_t o = ((e >> 2) * (kKeys * 128) + (e & 3) * 32) >> 4;
              tc_mma_ss(tS, a + o, b + o, idS, e > 0);
            }
            tc_commit(s_full(t));
            tc_commit(kv_empty(st, k_at));
          }
          __syncwarp();
        } else {
          if (k && ok && lane == 0) mbar_arrive(kv_empty(st, k_at));
          if (C::SHARED && ok && lane == 0) mbar_arrive(turn(t ^ 1));
        }
      }
      // nothing of this warp's products is in flight when the CTA's memory goes
      if (lane == 0) tc_commit(done_bar(t));
      __syncwarp();
      ok = mbar_wait(done_bar(t), 0) && ok;
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
// One warp per row; bound by the latency of its loads, so the first pieces' O are on their way
// before their weights are known, and eight are at a time.
template <int D>
__global__ void __launch_bounds__(256) attend_merge_kernel(const AttendParams p) {
  pdl_trigger();
  pdl_wait();
  const int4 cut = p.cut[blockIdx.x];
  if (cut.w == 0) return;
  constexpr int E = D / 32, kBatch = 8;                  // channels per lane
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int t = r / kRows, rr = r - t * kRows;
  const int in_tile = rr / p.G, tok = t * p.tok + in_tile;
  if (r >= p.rows || in_tile >= p.tok || tok >= cut.y) return;
  const int n = cut.w + 1;
  auto slot = [&](int i) {
    const int64_t s = i == 0 ? 2 * static_cast<int64_t>(blockIdx.x) + 1
                             : 2 * (static_cast<int64_t>(blockIdx.x) + i);
    return s * p.rows + r;
  };
  float v[kBatch][E];
  auto load = [&](int i0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (i0 + i < n) {
        const float *src = p.part_o + slot(i0 + i) * D + lane * E;
        if constexpr (E == 4)
          *reinterpret_cast<float4 *>(v[i]) = *reinterpret_cast<const float4 *>(src);
        else
          *reinterpret_cast<float2 *>(v[i]) = *reinterpret_cast<const float2 *>(src);
      }
  };
  load(0);
  const float2 none = make_float2(-INFINITY, 0.f);
  const float2 first = lane < n ? p.part_ml[slot(lane)] : none;
  float M = first.x;
  for (int i = lane + 32; i < n; i += 32) M = fmaxf(M, p.part_ml[slot(i)].x);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  float l = 0.f, o[E] = {};
  for (int i0 = 0; i0 < n; i0 += 32) {                   // a piece's weight per lane
    const float2 ml = i0 == 0 ? first : i0 + lane < n ? p.part_ml[slot(i0 + lane)] : none;
    // a piece without seen keys has only zero weights, and so is its O
    const float f = ml.y == 0.f ? 0.f : ex2(ml.x - M);
    l += f * ml.y;
    for (int j = 0; j < 32 && i0 + j < n; j += kBatch) {
      if (i0 + j > 0) load(i0 + j);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float g = __shfl_sync(0xffffffffu, f, j + i);
        if (i0 + j + i < n) {
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] += g * v[i][e];
        }
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint16_t *dst = p.out + (static_cast<int64_t>(cut.x + tok) * p.Hq + cut.z * p.G + (rr - in_tile * p.G)) * D +
                  lane * E;
  if constexpr (E == 4)
    *reinterpret_cast<uint2 *>(dst) =
        make_uint2(pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv));
  else
    *reinterpret_cast<uint32_t *>(dst) = pack_bf16(o[0] * inv, o[1] * inv);
}

// ------------------------------------------------------------------ host side

// 3D TMA map of query rows [T, Hq, D] bf16: a box is `tok` tokens x the heads of one KV head x 64
// columns, which land in shared memory as 128-byte swizzled rows (token, head).
bool make_query_map(CUtensorMap *map, const void *q, const pa_shape &s, int T, int tok) {
  static const PFN_cuTensorMapEncodeTiled_v12000 encode = [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult found;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                                     cudaEnableDefault, &found) == cudaSuccess &&
                    found == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
  }();
  if (!encode) return false;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(s.D), static_cast<cuuint64_t>(s.Hq),
                              static_cast<cuuint64_t>(T)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(s.D) * 2,
                                 static_cast<cuuint64_t>(s.Hq) * s.D * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(s.Hq / s.Hkv), static_cast<cuuint32_t>(tok)};
  const cuuint32_t steps[3] = {1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(q), dims, strides, box,
                steps, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Separate key streams while a sequence has at most one row tile of tokens on average.  Measured
// on 8 sequences of 4,000 to 8,000 cached tokens, 64 query and 8 KV heads (16 tokens a row tile):
// 24 tokens each 59 us shared against 83 separate, 40 tokens 95 against 110; below, the second row
// tile of the shared form is empty.
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
  // the registers that the warps ask for must be those that the CTA was launched with: asking for
  // more would wait for ever
  static std::atomic<bool> fits{false};
  if (!fits.load(std::memory_order_relaxed)) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, kernel) != cudaSuccess) return PA_ERR_CUDA;
    if (a.numRegs * C::THREADS < 256 * C::SOFTMAX_REGS + (C::THREADS - 256) * C::OTHER_REGS)
      return PA_ERR_UNSUPPORTED;
    fits.store(true, std::memory_order_relaxed);
  }
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  if (launch_pdl(kernel, dim3(p.workers / C::STREAMS), dim3(C::THREADS), C::SMEM, stream, mq, mk, mv, p) !=
      cudaSuccess)
    return PA_ERR_CUDA;
  // a sequence of one tile has units of one tile, which no segment bound cuts
  if (static_cast<int64_t>(p.max_blocks) * p.bs <= kKeys) return PA_OK;
  const dim3 grid(p.workers, (p.rows + 7) / 8);          // a warp per row
  return launch_pdl(attend_merge_kernel<C::D>, grid, dim3(256), 0, stream, p) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace

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
  // four ragged prompts, shared form: 488, 449, 439, 444, 453 us with 0 to 4; verification of few
  // tokens, separate form: 116, 121 and 127 us with 1 to 3
  p.unit_cost = plan.shared ? 2 : 1;
  p.over_workers = ~uint64_t(0) / plan.workers + 1;       // exact for totals below 2^55
  p.rows = plan.rows;
  // c > 0 keeps a masked score's c s at -inf; 1e-30 scores every key alike, as 0 does
  const float c = sm_scale * kLog2e;
  p.c = fmaxf(fabsf(c), 1e-30f);
  p.negate = c < 0.f;
  p.wide = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
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
