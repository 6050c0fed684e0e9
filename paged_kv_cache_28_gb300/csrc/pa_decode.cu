// pa_decode.cu -- paged decode attention for sm_103a.
//
// What is computed ("Taming the Token Torrent", section "Custom PagedAttention
// Kernels"; "KV Cache Engineering for LLM Serving", section 1): for every
// sequence b and query head h,
//     out[b][h] = softmax_t(sm_scale * <q[b][h], K_b[t]>) V_b[t],  t < seq_lens[b],
// where K_b / V_b are gathered through the block table and query head h reads KV
// head h / G.
//
// How (GB300 design):
//  * The unit of work is a 16-token tile of one (sequence, KV head) pair.  A
//    warp streams its tiles through a private ring of shared-memory stages.
//    Each stage is filled by TMA (two or one 128-byte-swizzled boxes for K, the
//    same for V) plus, when a new pair starts, a bulk copy of the pair's G query
//    rows; completion is tracked by one mbarrier per stage.
//  * The whole query group of a KV head is served at once with warp-level
//    tensor-core mma (m16n8k16): S^T = K Q^T (tokens x heads, the group is the
//    n = 8 side), online softmax in fp32 registers with warp shuffles, then
//    O^T += V^T P^T with P split into a high and a low 16-bit part so that the
//    weights keep ~16 significant bits.
//  * FP8 (E4M3) pools are converted to f16 in registers (exact); the per-block
//    K scale folds into the score scale and the V scale into the running
//    rescale factor, so dequantisation costs no per-element multiply.
//  * pa_decode: one CTA per (sequence, KV head); its warps take interleaved
//    tiles and merge their softmax states in shared memory at the end.
//  * pa_decode_splitkv: the tiles of all pairs, laid end to end, are cut into
//    equal segments, one per warp (flash-decoding with exact load balance).
//    Pairs inside a segment are finished in place; cut pairs leave (o, lse)
//    partials that pa_merge_lse combines.
#include <cudaTypedefs.h>

#include <mutex>

#include "pa_decode.cuh"

namespace pa {

constexpr bool kScored = false;   // what PA_DISPATCH instantiates

// ----------------------------------------------------------------------------
// pa_decode: one CTA per (sequence, KV head), or a cluster of CTAs per unit
// ----------------------------------------------------------------------------

// Thread-block clusters.  When a batch has few (sequence, KV head) units, pa_decode
// launches clusters of CTAs, one cluster per unit: the cluster's CTAs share the unit's
// tiles and CTA 0 merges their states through distributed shared memory.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return static_cast<int>(r);
}
__device__ __forceinline__ int cluster_ctas() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return static_cast<int>(r);
}
// Every thread of every CTA of the cluster arrives, then waits for all the others.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
// The shared::cluster address of `addr` (this CTA's shared memory) in CTA `rank`.
__device__ __forceinline__ uint32_t cluster_map(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
// Arrive on an mbarrier in another CTA of the cluster, releasing this thread's prior
// writes (and those ordered before them by a CTA barrier) at cluster scope.
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
// Bounded wait with acquire at cluster scope; false if the phase never completed.
template <uint32_t kSpins = kWaitSpins>
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity) {
  for (uint32_t it = 0; it < kSpins; ++it) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
  }
  return false;
}

// Fewest tiles a warp takes when a cluster shares a unit: a unit of n tiles keeps
// ceil(n / (kClusterWarpTiles * WARPS)) of the cluster's CTAs (at least one, at most
// all); the others leave at once.
constexpr int kClusterWarpTiles = 16;
// Batches up to this many sequences are served longest first: up to kExactRankMaxB by an
// exact ranking (B^2 / threads key comparisons per CTA), above it by quarter-octave
// buckets of the tile count (linear in B; one byte per sequence in the stage area).
constexpr int kLongestFirstMaxB = 16384;
constexpr int kExactRankMaxB = 128;
constexpr int kRankBuckets = 256;
// Shared scratch of longest_first: bucket counts, the count above each bucket, the
// search's results and per-warp counts, then one bucket byte per sequence.
constexpr int kRankScratch = (2 * kRankBuckets + 8) * 4 + kLongestFirstMaxB;

// Small batches: unit slot c serves the sequence of rank c / Hkv when the sequences
// are ordered by attended tiles, most first (ties by index).  Each sequence gets one
// 32-bit key, tiles above its index (larger = earlier, all distinct), and its rank
// is the number of larger keys: every thread ranks two candidates in one pass over
// the keys, four at a time.  keys: shared scratch of 4 * (round4(B) + 1) bytes,
// 16-byte aligned, free again on return.
__device__ int longest_first_exact(const Params &p, int pair, uint32_t *keys) {
  static_assert(kExactRankMaxB <= 512, "keys hold the sequence index in 9 bits");
  const int cap = p.max_blocks * p.bs;
  const int nb4 = (p.B + 3) >> 2;
  for (int b = threadIdx.x; b < 4 * nb4; b += blockDim.x) {
    uint32_t key = 0u;   // padding: counted by no rank
    if (b < p.B) {
      const int c = pair_tile_count(min(max(__ldg(p.seq_lens + b), 0), cap), p.window, p.topk);
      key = (static_cast<uint32_t>(min(c, (1 << 23) - 1)) << 9) | static_cast<uint32_t>(511 - b);
    }
    keys[b] = key;
  }
  __syncthreads();
  const int want = pair / p.Hkv;
  int *chosen = reinterpret_cast<int *>(keys + 4 * nb4);
  const uint4 *k4 = reinterpret_cast<const uint4 *>(keys);
  for (int b0 = threadIdx.x; b0 < p.B; b0 += 2 * blockDim.x) {
    const int b1 = b0 + blockDim.x;
    const uint32_t c0 = keys[b0], c1 = b1 < p.B ? keys[b1] : 0xFFFFFFFFu;
    int r0 = 0, r1 = 0;
    for (int j = 0; j < nb4; ++j) {
      const uint4 k = k4[j];
      r0 += (k.x > c0) + (k.y > c0) + (k.z > c0) + (k.w > c0);
      r1 += (k.x > c1) + (k.y > c1) + (k.z > c1) + (k.w > c1);
    }
    // ranks are a permutation of 0..B-1: exactly one thread writes
    if (r0 == want) *chosen = b0;
    if (b1 < p.B && r1 == want) *chosen = b1;
  }
  __syncthreads();
  const int seq = *chosen;
  __syncthreads();   // every thread has read it before the stages are filled
  return seq * p.Hkv + (pair - want * p.Hkv);
}

// Unit slot c (a CTA, or a cluster) serves the sequence of rank c / Hkv when the
// sequences are ordered by their bucket of attended tiles, fullest first, then by index:
// the longest units start first and do not end the launch alone.  Buckets are quarter
// octaves (n tiles: 4 floor(log2 n) + the next two bits of n, plus one), so a wave of
// CTAs mixes lengths within about a fifth of each other: on batches of near-equal
// lengths an exact order makes whole waves start and finish in step, with the DRAM idle
// at each boundary.  A histogram of the buckets and a scan from the top give the bucket
// holding the rank; a scan over runs of consecutive sequences finds its member.  The
// cost is linear in B.  scratch: kRankScratch bytes of shared memory, 16-byte
// aligned, free again on return.
__device__ __forceinline__ int tile_bucket(int n) {
  if (n <= 0) return 0;
  const int e = 31 - __clz(n);                                 // n in [2^e, 2^(e+1))
  const int frac = e >= 2 ? (n >> (e - 2)) & 3 : (n << (2 - e)) & 3;
  return 4 * e + frac + 1;                                     // <= 4 * 30 + 3 + 1
}

__device__ int longest_first_bucketed(const Params &p, int pair, uint8_t *scratch) {
  constexpr int NB = kRankBuckets;
  static_assert(NB == 2 * 128, "two buckets per thread of a 128-thread CTA");
  int *hist = reinterpret_cast<int *>(scratch);
  int *above = hist + NB;                        // sequences in higher buckets
  int *sel = above + NB;                         // bucket, rank within it, the sequence
  int *wcnt = sel + 4;                           // per-warp counts
  uint8_t *bucket = reinterpret_cast<uint8_t *>(wcnt + 4);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cap = p.max_blocks * p.bs;
  static_assert(4 * 30 + 3 + 1 < NB, "every tile count has a bucket");
  for (int k = tid; k < NB; k += blockDim.x) hist[k] = 0;
  __syncthreads();
  for (int b = tid; b < p.B; b += blockDim.x) {
    const int c = pair_tile_count(min(max(__ldg(p.seq_lens + b), 0), cap), p.window, p.topk);
    const int k = tile_bucket(c);
    bucket[b] = static_cast<uint8_t>(k);
    atomicAdd(&hist[k], 1);
  }
  __syncthreads();
  // above[k] = sum of hist[k'] over k' > k: thread t holds buckets NB-1-2t and NB-2-2t
  {
    const int k0 = NB - 1 - 2 * tid, k1 = k0 - 1;
    const int v = hist[k0] + hist[k1];
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) wcnt[warp] = inc;
    __syncthreads();
    int ex = inc - v;
    for (int w = 0; w < warp; ++w) ex += wcnt[w];
    above[k0] = ex;
    above[k1] = ex + hist[k0];
  }
  __syncthreads();
  const int want = pair / p.Hkv;                 // < B: exactly one bucket holds it
  for (int k = tid; k < NB; k += blockDim.x)
    if (above[k] <= want && want < above[k] + hist[k]) {
      sel[0] = k;
      sel[1] = want - above[k];
    }
  __syncthreads();
  // the j-th member of bucket kb in index order: each thread counts the members in its
  // own run of consecutive sequences, a scan over the threads finds the run holding it
  {
    const int kb = sel[0], j = sel[1];
    const int per = (p.B + static_cast<int>(blockDim.x) - 1) / static_cast<int>(blockDim.x);
    const int lo = min(p.B, tid * per), hi = min(p.B, lo + per);
    int mine = 0;
    for (int b = lo; b < hi; ++b) mine += bucket[b] == kb;
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) wcnt[warp] = inc;
    __syncthreads();
    int ex = inc - mine;
    for (int w = 0; w < warp; ++w) ex += wcnt[w];
    if (j >= ex && j < ex + mine) {
      int r = j - ex;
      for (int b = lo; b < hi; ++b)
        if (bucket[b] == kb && r-- == 0) {
          sel[2] = b;
          break;
        }
    }
    __syncthreads();
  }
  const int seq = sel[2];
  __syncthreads();   // every thread has read it before the stages are filled
  return seq * p.Hkv + (pair - want * p.Hkv);
}

__device__ __forceinline__ int longest_first(const Params &p, int pair, uint8_t *scratch) {
  return p.B <= kExactRankMaxB ? longest_first_exact(p, pair, reinterpret_cast<uint32_t *>(scratch))
                               : longest_first_bucketed(p, pair, scratch);
}

// CLUSTER: launched in clusters, one per unit (else one CTA per unit).
template <class C, bool CLUSTER>
__global__ void __launch_bounds__(C::THREADS, C::MIN_BLOCKS)
    decode_pair_kernel(const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const Params p) {
  static_assert(kRankScratch <= C::WARPS * C::STAGES * C::STAGE_BYTES && C::THREADS == 128,
                "the ordering's scratch lives in the stage area");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  const int ncl = CLUSTER ? cluster_ctas() : 1, crank = CLUSTER ? cluster_rank() : 0;
  int pair = blockIdx.x / ncl;
  // a window or a Quest selection bounds every unit's tiles: near-uniform units gain
  // nothing from an order that costs more than the exact ranking of a small batch
  const bool bounded = p.window > 0 || p.topk > 0;
  if (p.B <= (bounded ? kExactRankMaxB : kLongestFirstMaxB))
    pair = longest_first(p, pair, base);
  const int b = pair / p.Hkv, kvh = pair - b * p.Hkv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int L = p.seq_lens[b];
  const int cap = p.max_blocks * p.bs;
  if (L < 0 || L > cap) {
    if (threadIdx.x == 0 && kvh == 0) set_err(p.err, PA_DEVERR_SEQ_LEN);
    L = min(max(L, 0), cap);
  }
  WarpSmem ws = setup_smem<C>(smem_raw, warp, p.G, lane);
  State<C> st;
  st.reset();
  PairSource src;
  src.row = p.block_tables + static_cast<size_t>(b) * p.max_blocks;
  src.err = p.err;
  src.pair = pair;
  src.kvh = kvh;
  src.hkv = p.Hkv;
  src.geo = seq_tiles(L, p.window);
  src.npages = (L + kTile - 1) / kTile;
  src.shared_len = p.shared_prefix_lens ? __ldg(p.shared_prefix_lens + b) : -1;
  src.sel = nullptr;
  if (p.sel) {
    src.sel = p.sel + static_cast<size_t>(pair) * p.topk;
    src.geo.first = 0;
    src.geo.count = pair_tile_count(L, 0, p.topk);
  }
  constexpr int GP = 8 * C::NT;
  float *sm_acc = reinterpret_cast<float *>(base);               // [WARPS][GP][D], stage area
  float *sm_m = reinterpret_cast<float *>(split_tail<C>(smem_raw));   // [WARPS][GP]
  float *sm_l = sm_m + C::WARPS * GP;                            // [WARPS][GP]
  float *cta_m = sm_l + C::WARPS * GP;                           // [GP] folded over warps
  float *cta_l = cta_m + GP;                                     // [GP]
  const uint32_t cl_bar = smem_u32(cta_l + GP);                  // cluster mbarrier
  // A cluster shares the unit's tiles among its first `active` CTAs; the others leave.
  int active = 1;
  if (ncl > 1) {
    const int per_cta = kClusterWarpTiles * C::WARPS;
    active = min(ncl, max(1, (src.geo.count + per_cta - 1) / per_cta));
    if (threadIdx.x == 0) {   // CTA 0 hears from the other active CTAs, each of them from CTA 0
      mbar_init(cl_bar, crank == 0 ? max(active - 1, 1) : 1);
      fence_mbar_init();
    }
    cluster_barrier();   // every CTA's cluster mbarrier is initialised
    if (crank >= active) return;
  }
  src.w = crank * C::WARPS + warp;
  src.nw = active * C::WARPS;
  src.bs = p.bs;
  src.nblocks = p.nblocks;
  src.init(lane);
  run_warp<C>(src, ws, st, p, &tmK, &tmV, [](int4, bool, State<C> &) {}, lane);

  // ---- merge the warps' states: warp w leaves m, l, acc (in absolute units)
  __syncthreads();
  {
    float ltot[C::NT][2];
    reduce_l<C>(st, ltot);
    const int qd = lane & 3;
#pragma unroll
    for (int nt = 0; nt < C::NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int g = nt * 8 + 2 * qd + j;
        if ((lane >> 2) == 0) {
          sm_m[warp * GP + g] = st.m[nt][j];
          sm_l[warp * GP + g] = ltot[nt][j];
        }
        const float f = C::QUANT ? st.vref[nt] : 1.f;
#pragma unroll
        for (int dt = 0; dt < C::DT; ++dt) {
          sm_acc[(warp * GP + g) * C::D + acc_d<C>(dt, j, lane)] = st.acc[nt][dt][j] * f;
          sm_acc[(warp * GP + g) * C::D + acc_d<C>(dt, j + 2, lane)] = st.acc[nt][dt][j + 2] * f;
        }
      }
  }
  __syncthreads();
  float *out = p.out + (static_cast<size_t>(b) * p.Hq + kvh * p.G) * C::D;
  for (int e = threadIdx.x; e < p.G * C::D; e += C::THREADS) {
    const int g = e / C::D, d = e - g * C::D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < C::WARPS; ++w) M = fmaxf(M, sm_m[w * GP + g]);
    float num = 0.f, den = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int w = 0; w < C::WARPS; ++w) {
        const float mw = sm_m[w * GP + g];
        if (mw == -INFINITY) continue;
        const float f = ex2(mw - M);
        num += f * sm_acc[(w * GP + g) * C::D + d];
        den += f * sm_l[w * GP + g];
      }
    }
    if (ncl == 1) {
      out[e] = den > 0.f ? num / den : 0.f;
    } else {   // this CTA's state, relative to its own maximum M, for CTA 0 to merge
      sm_acc[g * C::D + d] = num;   // warp 0's entry (g, d): no other thread touches it
      if (d == 0) {
        cta_m[g] = M;
        cta_l[g] = den;
      }
    }
  }
  if (ncl == 1) return;

  // ---- cluster: CTA 0 merges the active CTAs' states through distributed shared memory
  __syncthreads();
  if (crank > 0) {
    if (threadIdx.x == 0) mbar_arrive_cluster(cluster_map(cl_bar, 0));
    // stay until CTA 0 has read this CTA's shared memory; this wait is bounded four times
    // longer than CTA 0's, so a CTA 0 that gave up (and reads nothing) is the only way
    // it runs out
    if (!mbar_wait_cluster<4 * kWaitSpins>(cl_bar, 0) && threadIdx.x == 0)
      set_err(p.err, PA_DEVERR_TIMEOUT);
    return;
  }
  // the other CTAs' states are complete once the phase completed for any thread
  const bool merged = __syncthreads_or(active <= 1 || mbar_wait_cluster(cl_bar, 0));
  if (!merged) {                     // no remote read: report, write zeros, release nobody
    if (threadIdx.x == 0) set_err(p.err, PA_DEVERR_TIMEOUT);
    for (int e = threadIdx.x; e < p.G * C::D; e += C::THREADS) out[e] = 0.f;
    return;
  }
  constexpr int kMaxCluster = 8;
  for (int e = threadIdx.x; e < p.G * C::D; e += C::THREADS) {
    const int g = e / C::D, d = e - g * C::D;
    const uint32_t am = smem_u32(&cta_m[g]), al = smem_u32(&cta_l[g]);
    const uint32_t aa = smem_u32(&sm_acc[g * C::D + d]);
    float mc[kMaxCluster];
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < kMaxCluster; ++c) {
      mc[c] = c < active ? ld_cluster_f32(cluster_map(am, c)) : -INFINITY;
      M = fmaxf(M, mc[c]);
    }
    float num = 0.f, den = 0.f;
    if (M != -INFINITY) {
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        if (mc[c] == -INFINITY) continue;
        const float f = ex2(mc[c] - M);
        num += f * ld_cluster_f32(cluster_map(aa, c));
        den += f * ld_cluster_f32(cluster_map(al, c));
      }
    }
    out[e] = den > 0.f ? num / den : 0.f;
  }
  __syncthreads();   // every read of the other CTAs' shared memory is done: release them
  if (threadIdx.x > 0 && threadIdx.x < active) mbar_arrive_cluster(cluster_map(cl_bar, threadIdx.x));
}

// ----------------------------------------------------------------------------
// pa_decode without a workspace on many units: persistent CTAs
// ----------------------------------------------------------------------------

// A bf16 batch with more (sequence, KV head) units than two per resident CTA, and no
// window or page selection, runs one CTA of eight warps per SM instead of one CTA per
// unit.  Every CTA computes the same static schedule from the lengths ("water
// filling"): the units, longest first, are dealt out in rounds; each round's units
// fill the least loaded CTAs up to a common level, a unit going to the CTA in whose
// share the midpoint of its tiles falls.  Each CTA so gets about the mean number of
// tiles, and no unit is split across CTAs (there is no memory to merge them in).  A
// CTA's units form one stream of tiles, cut into eight equal contiguous segments, one
// per warp: each warp's ring runs on from one unit into the next, a long unit is read
// by several warps, and a unit inside one segment is finished by its warp alone.  A
// unit that crosses segments is joined in shared memory: each warp before the last
// that holds part of it leaves its state in its mailbox (a warp's only part that ends
// before the unit does), and the warp holding the unit's last tile folds those parts,
// in warp order, into its own and writes the output.  The schedule, the segments and
// the fold order are fixed by the inputs, so results repeat bit for bit.
constexpr int kPersistWarps = 8;
constexpr int kPersistMaxUnits = 4096;   // the unit list's capacity: any batch's units fit
constexpr int kPersistMaxBins = 256;     // CTAs of the launch (one per SM)
constexpr int kPersistMaxRounds = 24;    // rounds of the water filling (at least U / 16 units each)

template <class B>
struct PersistCfg : B {
  static constexpr int WARPS = kPersistWarps;
  static constexpr int THREADS = WARPS * 32;
  static constexpr int GP = 8 * B::NT;
  static constexpr int RING = 1024 + WARPS * (B::STAGES * (B::STAGE_BYTES + 8 + B::META_BYTES) +
                                              B::QF_BYTES);
  static constexpr int MAILBOX_BYTES = WARPS * GP * (B::D + 2) * 4;   // acc, m, l per warp
  static constexpr int LIST_BYTES = kPersistMaxUnits * 2 + (kPersistMaxUnits + 1 + WARPS + 4) * 4;
  static constexpr int SMEM = RING + MAILBOX_BYTES + LIST_BYTES;
  static_assert(!B::QUANT && B::NT == 1, "persistent CTAs serve bf16 units of up to 8 heads");
  static_assert(SMEM <= 227 * 1024, "one persistent CTA per SM");
};

// Shared scratch of the schedule (in the stage area, before any copy is issued).
template <int NW>
struct PersistScratch {
  static constexpr int NB = kRankBuckets;
  int32_t gp[kPersistMaxUnits + 1];         // tiles of the units before position k
  int32_t lo[kPersistMaxBins];              // a round's first unit of each CTA
  int32_t tiles[kPersistMaxUnits];          // attended tiles per sequence
  int32_t order[kPersistMaxUnits];          // longest-first position -> sequence
  int32_t uid[kPersistMaxUnits];            // longest-first position -> unit
  int32_t hist[NW][NB];                     // per-warp bucket counts, then sort bases
  int32_t wsum[NW];                         // block scans: per-warp totals
  long long wsum64[NW];
  long long red[2][NW];                     // the fill level's reductions (two in turn)
  int32_t mine[kPersistMaxRounds][2];       // this CTA's unit range of each round
  uint8_t bucket[kPersistMaxUnits];
};

// Block-wide exclusive scan of one value per thread (every thread gets the total).
template <int THREADS, class T>
__device__ __forceinline__ T block_scan_excl(T v, T *wsum, T &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += u;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  T off = 0, tot = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    off += w < warp ? wsum[w] : 0;
    tot += wsum[w];
  }
  __syncthreads();   // wsum is free again
  total = tot;
  return off + inc - v;
}

// The schedule: this CTA's units (ids sequence * Hkv + KV head) in stream order, with
// starts[k] = tiles of the units before unit k (starts[n] = the CTA's tiles).  Returns n.
// The launch keeps every sum of tiles below 2^30.
template <int THREADS>
__device__ int persist_schedule(const Params &p, PersistScratch<THREADS / 32> &s,
                                uint16_t *units, int32_t *starts) {
  constexpr int NW = THREADS / 32, NB = PersistScratch<NW>::NB;
  static_assert(THREADS >= NB && THREADS >= kPersistMaxBins, "a bucket and a CTA per thread");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.B, H = p.Hkv, U = B * H, bins = gridDim.x;
  const int cap = p.max_blocks * p.bs;
  for (int b = tid; b < B; b += THREADS) {
    const int L = __ldg(p.seq_lens + b);
    if ((L < 0 || L > cap) && blockIdx.x == 0) set_err(p.err, PA_DEVERR_SEQ_LEN);
    const int n = seq_tiles(min(max(L, 0), cap), 0).count;
    s.tiles[b] = n;
    s.bucket[b] = static_cast<uint8_t>(tile_bucket(n));
  }
  for (int i = tid; i < NW * NB; i += THREADS) (&s.hist[0][0])[i] = 0;
  __syncthreads();
  // ---- stable order of the sequences: bucket descending, then index.  Warp w counts
  // and places the sequences of its own contiguous range.
  const int per = (B + NW - 1) / NW;
  const int lo = min(B, warp * per), hi = min(B, lo + per);
  for (int b = lo + lane; b < hi; b += 32) atomicAdd(&s.hist[warp][s.bucket[b]], 1);
  __syncthreads();
  {
    // first position of bucket k: the sequences in higher buckets (thread t: bucket NB-1-t)
    const int k = NB - 1 - tid;
    int cnt = 0;
    if (tid < NB)
#pragma unroll
      for (int w = 0; w < NW; ++w) cnt += s.hist[w][k];
    int total;
    int first = block_scan_excl<THREADS>(cnt, s.wsum, total);
    if (tid < NB)
#pragma unroll
      for (int w = 0; w < NW; ++w) {   // warp w's first position in bucket k
        const int c = s.hist[w][k];
        s.hist[w][k] = first;
        first += c;
      }
  }
  __syncthreads();
  for (int b0 = lo; b0 < hi; b0 += 32) {
    const int b = b0 + lane;
    const int key = b < hi ? s.bucket[b] : -1;
    const uint32_t peers = __match_any_sync(0xffffffffu, key);
    const uint32_t below = peers & ((1u << lane) - 1u);
    if (b < hi) s.order[s.hist[warp][key] + __popc(below)] = b;
    __syncwarp();
    if (b < hi && below == 0) s.hist[warp][key] += __popc(peers);
    __syncwarp();
  }
  __syncthreads();
  // ---- the units in that order (KV heads in turn) and the prefix of their tiles
  {
    const int run = (U + THREADS - 1) / THREADS;
    const int k0 = min(U, tid * run), k1 = min(U, k0 + run);
    int mine = 0;
    for (int k = k0; k < k1; ++k) {
      const int q = k / H, b = s.order[q];
      s.uid[k] = b * H + (k - q * H);
      mine += s.tiles[b];
    }
    int total;
    int at = block_scan_excl<THREADS>(mine, s.wsum, total);
    for (int k = k0; k < k1; ++k) {
      s.gp[k] = at;
      at += s.tiles[s.uid[k] / H];
    }
    if (tid == 0) s.gp[U] = total;
  }
  __syncthreads();
  // ---- water filling.  Round r deals the next max(bins * (r + 1), U / 16) units of the
  // order; thread b < bins keeps CTA b's load.
  const bool has_bin = tid < bins;
  int lb = 0;
  int rounds = 0;
  for (int next = 0, r = 0; next < U; ++r) {
    const int c = min(U - next, max(bins * (r + 1), (U + 15) / 16));
    const int base = s.gp[next], tot = s.gp[next + c] - base;
    // The fill level: the CTAs S below it take the round's tiles, h = (tot + their
    // loads) / |S|.  From S = every CTA, dropping those at or above the level lowers
    // it; S is final when none drops (a round of no tiles keeps the least loaded).
    bool in = has_bin;
    long long A = 0;
    int m = 0;
    for (int it = 0;; ++it) {
      long long v = in ? ((1ll << 40) | lb) : 0ll;   // members in bits 40.., loads below
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) s.red[it & 1][warp] = v;
      __syncthreads();
      long long t = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) t += s.red[it & 1][w];
      m = static_cast<int>(t >> 40);
      A = tot + (t & ((1ll << 40) - 1));
      const bool stay = in && static_cast<long long>(lb) * m < A;
      const int nm = __syncthreads_count(stay);
      if (nm == m || nm == 0) break;
      in = stay;
    }
    // shares in CTA order: h - load for each member, one tile more for its first rem
    // members, so that they add up to tot; CTA b's share is [cum, cum + share)
    const long long h = A / m, rem = A - h * m;
    long long shares;
    const long long px = block_scan_excl<THREADS>(in ? ((1ll << 40) | (h - lb)) : 0ll, s.wsum64,
                                                  shares);
    // CTA b takes the units whose tile midpoints fall in its share: from the first unit
    // whose midpoint reaches cum up to the next CTA's first (CTAs without a share take none)
    if (has_bin) {
      const long long cum2 = 2 * ((px & ((1ll << 40) - 1)) + min(px >> 40, rem));
      int a = next, z = next + c;   // first k in [next, next + c) with 2 mid(k) >= cum2
      while (a < z) {
        const int md = (a + z) >> 1;
        if (static_cast<long long>(s.gp[md]) + s.gp[md + 1] - 2ll * base >= cum2) z = md;
        else a = md + 1;
      }
      s.lo[tid] = a;
    }
    __syncthreads();
    if (has_bin) {
      const int k0 = tid == 0 ? next : s.lo[tid], k1 = tid + 1 < bins ? s.lo[tid + 1] : next + c;
      lb += s.gp[k1] - s.gp[k0];
      if (tid == static_cast<int>(blockIdx.x)) {
        s.mine[r][0] = k0;
        s.mine[r][1] = k1;
      }
    }
    __syncthreads();   // lo is read before the next round writes it
    next += c;
    rounds = r + 1;
  }
  // ---- this CTA's list: its ranges of the order, round by round
  int n = 0;
  for (int r = 0; r < rounds; ++r) {
    const int k0 = s.mine[r][0], k1 = s.mine[r][1];
    for (int k = k0 + tid; k < k1; k += THREADS) {
      units[n + k - k0] = static_cast<uint16_t>(s.uid[k]);
      starts[n + k - k0] = s.gp[k] - s.gp[k0];   // within the range, made absolute below
    }
    n += k1 - k0;
  }
  __syncthreads();
  for (int r = 0, at = 0, off = 0; r < rounds; ++r) {   // ranges' tile offsets
    const int k0 = s.mine[r][0], k1 = s.mine[r][1];
    for (int k = k0 + tid; k < k1; k += THREADS) starts[at + k - k0] += off;
    at += k1 - k0;
    off += s.gp[k1] - s.gp[k0];
    if (r == rounds - 1 && tid == 0) starts[n] = off;
  }
  __syncthreads();
  return n;
}

// Warp w's segment [begin, end) of its CTA's tile stream.
struct PersistSource {
  const uint16_t *units;           // shared: the CTA's list
  const int32_t *starts;
  const int32_t *seq_lens, *block_tables, *shared_prefix_lens;
  int32_t *err;
  int n, begin, end, Hkv, bs, nblocks, max_blocks;
  int base;
  int4 cur, nxt;

  __device__ __forceinline__ int count() const { return end - begin; }
  __device__ __forceinline__ int4 load(int i) const {
    const int g = begin + i;
    if (g >= end) return make_int4(0, 0, -1, 0);   // never issued
    int a = 0, z = n - 1;   // the unit holding position g: largest k with starts[k] <= g
    while (a < z) {
      const int md = (a + z + 1) >> 1;
      if (starts[md] <= g) a = md; else z = md - 1;
    }
    const int unit = units[a], b = unit / Hkv, kvh = unit - b * Hkv;
    const int nk = starts[a + 1] - starts[a], j = g - starts[a];
    const int L = min(max(__ldg(seq_lens + b), 0), max_blocks * bs);
    const SeqTiles geo = seq_tiles(L, 0);
    int phys = __ldg(block_tables + static_cast<size_t>(b) * max_blocks + (j * kTile) / bs);
    if (phys < 0 || phys >= nblocks) {
      set_err(err, PA_DEVERR_BLOCK_ID);
      phys = kInvalidPhys;
    }
    int info = (j == nk - 1) ? geo.last_valid : kTile;
    if (j == 0) info |= kFirstOfPair | kPieceStart;
    if (j == nk - 1) info |= kLastOfPair | kPieceEnd;
    if (i == 0) info |= kPieceStart;
    if (g == end - 1) info |= kPieceEnd;
    if (shared_prefix_lens)
      info |= ((j + 1) * kTile <= __ldg(shared_prefix_lens + b)) ? kHintShared : kHintPrivate;
    return tile_record(phys, j, unit, kvh, Hkv, bs, nblocks, info | (kvh << kKvhShift));
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

// Lane 0 polls a shared flag until it reads nonzero (bounded: a wait that runs out sets
// the error flag and returns false).  Returns for the whole warp.
__device__ __forceinline__ bool persist_wait(const volatile int32_t *flag, int32_t *err, int lane) {
  int ok = 1;
  if (lane == 0) {
    uint32_t i = 0;
    while (*flag == 0) {
      if (++i == kWaitSpins) {
        ok = 0;
        set_err(err, PA_DEVERR_TIMEOUT);
        break;
      }
      __nanosleep(64);
    }
  }
  ok = __shfl_sync(0xffffffffu, ok, 0);
  __threadfence_block();
  return ok != 0;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    decode_persist_kernel(const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV, const Params p) {
  constexpr int GP = C::GP, W = C::WARPS;
  using Scratch = PersistScratch<C::THREADS / 32>;
  static_assert(sizeof(Scratch) <= W * C::STAGES * C::STAGE_BYTES,
                "the schedule's scratch lives in the stage area");
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
  float *box_acc = reinterpret_cast<float *>(split_tail<C>(smem_raw));   // [W][GP][D]
  float *box_m = box_acc + W * GP * C::D;                                 // [W][GP]
  float *box_l = box_m + W * GP;                                          // [W][GP]
  uint16_t *units = reinterpret_cast<uint16_t *>(box_l + W * GP);        // [max units]
  int32_t *starts = reinterpret_cast<int32_t *>(units + kPersistMaxUnits); // [max units + 1]
  int32_t *filled = starts + kPersistMaxUnits + 1;                        // [W] mailbox flags
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_trigger();
  // the schedule reads only caller inputs (lengths); the output and the pools (written
  // by the cache write) are touched only after the previous grid has finished
  const int n = persist_schedule<C::THREADS>(p, *reinterpret_cast<Scratch *>(base), units, starts);
  pdl_wait();
  if (threadIdx.x < W) filled[threadIdx.x] = 0;
  // units without tiles (empty sequences) have no warp to write them
  for (int k = warp; k < n; k += W) {
    if (starts[k + 1] > starts[k]) continue;
    const int unit = units[k], b = unit / p.Hkv, kvh = unit - b * p.Hkv;
    float *out = p.out + (static_cast<size_t>(b) * p.Hq + kvh * p.G) * C::D;
    for (int e = lane; e < p.G * C::D; e += 32) out[e] = 0.f;
  }
  __syncthreads();   // the scratch is read: the stages may be filled

  const int T = starts[n];
  auto seg = [&](int w) { return static_cast<int>(static_cast<long long>(w) * T / W); };
  WarpSmem ws = setup_smem<C>(smem_raw, warp, p.G, lane);
  State<C> st, held;
  st.reset();
  held.reset();
  PersistSource src;
  src.units = units;
  src.starts = starts;
  src.seq_lens = p.seq_lens;
  src.block_tables = p.block_tables;
  src.shared_prefix_lens = p.shared_prefix_lens;
  src.err = p.err;
  src.n = n;
  src.begin = seg(warp);
  src.end = seg(warp + 1);
  src.Hkv = p.Hkv;
  src.bs = p.bs;
  src.nblocks = p.nblocks;
  src.max_blocks = p.max_blocks;
  src.init(lane);
  auto out_of = [&](int unit) {
    const int b = unit / p.Hkv, kvh = unit - b * p.Hkv;
    return p.out + (static_cast<size_t>(b) * p.Hq + kvh * p.G) * C::D;
  };
  const int qd = lane & 3;
  // this warp's mailbox: m, l (totals over the warp) and acc of a state
  auto deposit = [&](const float (&m)[2], const float (&l)[2], auto &&acc_of) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int g = 2 * qd + j;
      if ((lane >> 2) == 0) {
        box_m[warp * GP + g] = m[j];
        box_l[warp * GP + g] = l[j];
      }
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          box_acc[(warp * GP + g) * C::D + acc_d<C>(dt, j + 2 * h, lane)] = acc_of(dt, j + 2 * h);
    }
    __threadfence_block();
    __syncwarp();
    if (lane == 0) *reinterpret_cast<volatile int32_t *>(&filled[warp]) = 1;
  };
  int held_unit = -1;
  bool held_last = false;
  auto on_end = [&](int4 u, bool piece_first, State<C> &s) {
    const bool last = (u.w & kLastOfPair) != 0;
    if (piece_first && last) {              // a whole unit: finished here
      write_normalised<C>(s, out_of(u.y), nullptr, p.G, lane);
    } else if (!piece_first) {              // the unit came from the warps before
      held = s;
      held_unit = u.y;
      held_last = last;
    } else {                                // the unit goes on into the next warp
      float lt[1][2];
      reduce_l<C>(s, lt);
      const float mm[2] = {s.m[0][0], s.m[0][1]}, ll[2] = {lt[0][0], lt[0][1]};
      deposit(mm, ll, [&](int dt, int i) { return s.acc[0][dt][i]; });
    }
  };
  const bool ok = run_warp<C>(src, ws, st, p, &tmK, &tmV, on_end, lane);
  if (held_unit < 0 || !ok) return;
  float lt[1][2];
  reduce_l<C>(held, lt);
  if (!held_last) {   // the unit goes on past this segment: its last warp folds this part
    const float mm[2] = {held.m[0][0], held.m[0][1]}, ll[2] = {lt[0][0], lt[0][1]};
    deposit(mm, ll, [&](int dt, int i) { return held.acc[0][dt][i]; });
    return;
  }
  // ---- the unit's last warp: fold the parts the warps before left in their mailboxes,
  // in warp order, then its own, and write the output
  int k = 0;   // the unit: the one holding this segment's first tile
  for (int z = n - 1; k < z;) {
    const int md = (k + z + 1) >> 1;
    if (starts[md] <= src.begin) k = md; else z = md - 1;
  }
  float M[2] = {-INFINITY, -INFINITY}, L[2] = {0.f, 0.f}, acc[C::DT][4];
#pragma unroll
  for (int dt = 0; dt < C::DT; ++dt) acc[dt][0] = acc[dt][1] = acc[dt][2] = acc[dt][3] = 0.f;
  auto fold = [&](const float (&mo)[2], const float (&lo)[2], auto &&acc_of) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float Mn = fmaxf(M[j], mo[j]);
      const float fa = M[j] == -INFINITY ? 0.f : ex2(M[j] - Mn);
      const float fb = mo[j] == -INFINITY ? 0.f : ex2(mo[j] - Mn);
#pragma unroll
      for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
        for (int h = 0; h < 2; ++h) acc[dt][j + 2 * h] = acc[dt][j + 2 * h] * fa + acc_of(dt, j + 2 * h) * fb;
      L[j] = L[j] * fa + lo[j] * fb;
      M[j] = Mn;
    }
  };
  for (int w = 0; w < warp; ++w) {
    if (seg(w + 1) <= starts[k] || seg(w) == seg(w + 1)) continue;   // holds none of the unit
    if (!persist_wait(&filled[w], p.err, lane)) return;
    float mo[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      mo[j] = box_m[w * GP + 2 * qd + j];
      lo[j] = box_l[w * GP + 2 * qd + j];
    }
    fold(mo, lo, [&](int dt, int i) {
      return box_acc[(w * GP + 2 * qd + (i & 1)) * C::D + acc_d<C>(dt, i, lane)];
    });
  }
  {
    const float mo[2] = {held.m[0][0], held.m[0][1]}, lo[2] = {lt[0][0], lt[0][1]};
    fold(mo, lo, [&](int dt, int i) { return held.acc[0][dt][i]; });
  }
  float *out = out_of(held_unit);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int g = 2 * qd + j;
    if (g >= p.G) continue;
    const float inv = L[j] > 0.f ? 1.f / L[j] : 0.f;
#pragma unroll
    for (int dt = 0; dt < C::DT; ++dt)
#pragma unroll
      for (int h = 0; h < 2; ++h) out[g * C::D + acc_d<C>(dt, j + 2 * h, lane)] = acc[dt][j + 2 * h] * inv;
  }
}

// One CTA per (b, kvh) pair; threads over (head, 4 consecutive d).  The pieces of a
// pair are visited eight at a time with their loads issued together.  The decode
// leaves the number of KV heads per unit (1, or 2 for paired 4-bit heads) after
// the tile prefix: head kvh's partials are then rows (kvh % 2) G .. of unit kvh / 2.
__global__ void __launch_bounds__(256) merge_kernel(float *out, const int32_t *prefix,
                                                    const float *o_part, const float *lse_part,
                                                    int B, int Hq, int Hkv, int G, int D,
                                                    int num_splits) {
  pdl_trigger();
  pdl_wait();
  const int pair = blockIdx.x;
  const int b = pair / Hkv, kvh = pair - b * Hkv;
  const int heads = prefix[B + 1] == 2 ? 2 : 1;
  const int unit = kvh / heads, row0 = (kvh - unit * heads) * G;
  const int Hu = Hkv / heads, Gu = G * heads;      // units per sequence, rows per unit
  const int start_b = prefix[b];
  const int nt = (prefix[b + 1] - start_b) / Hu;
  const int total = prefix[B];
  const int W = max(1, (total + num_splits - 1) / num_splits);
  float *o = out + (static_cast<size_t>(b) * Hq + kvh * G) * D;
  const int D4 = D / 4;
  // a cascaded sequence adds the partials of its shared prefix (cascade workspace);
  // a unit finished inside one segment was joined with them there
  const uint64_t cws = (static_cast<uint64_t>(static_cast<uint32_t>(prefix[B + 3])) << 32) |
                       static_cast<uint32_t>(prefix[B + 2]);
  const float *clse = nullptr, *co = nullptr;
  const int cpieces = cascade_partials(cws, B, Hq, Hkv, G, D, b, kvh, clse, co);
  if (nt == 0 && cpieces == 0) {
    for (int e = threadIdx.x; e < G * D4; e += blockDim.x)
      reinterpret_cast<float4 *>(o)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    return;
  }
  const int start = start_b + unit * nt, end = start + nt;
  // split pieces p0..p1 (none when the cascade covers the whole sequence)
  int p0 = nt > 0 ? start / W : 0, p1 = nt > 0 ? (end - 1) / W : -1;
  const bool inplace = nt > 0 && p0 == p1;         // finished inside one segment
  if (inplace && cpieces == 0) return;
  // a cascaded unit finished in place left its (o, lse) in the unit slots
  const float *ulse = nullptr, *uo = nullptr;
  if (inplace) {
    const CascadeLayout cl = cascade_layout(B, Hq, D);
    const uint8_t *cw = reinterpret_cast<const uint8_t *>(cws);
    const size_t row = static_cast<size_t>(b) * Hq + kvh * G;
    ulse = reinterpret_cast<const float *>(cw + cl.ulse) + row;
    uo = reinterpret_cast<const float *>(cw + cl.uo) + row * D;
    p1 = p0 - 1;                                   // no split pieces
  }
  // one pass: each batch of up to U pieces' (lse, o) is loaded together, then folded into
  // a running maximum M with num and den rescaled when it rises
  constexpr int U = 8;
  for (int e = threadIdx.x; e < G * D4; e += blockDim.x) {
    const int g = e / D4, d4 = e - g * D4, gu = row0 + g;
    auto slot = [&](int s) { return static_cast<size_t>(s) * 2 + (s == p0 ? 1 : 0); };
    float M = -INFINITY, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fold = [&](float l, float4 x) {           // one piece; l = -inf adds nothing
      if (l > M) {
        const float r = expf(M - l);               // 0 while M is -inf
        num = make_float4(num.x * r, num.y * r, num.z * r, num.w * r);
        den *= r;
        M = l;
      }
      const float w = l == -INFINITY ? 0.f : expf(l - M);
      num.x += w * x.x;
      num.y += w * x.y;
      num.z += w * x.z;
      num.w += w * x.w;
      den += w;
    };
    if (ulse) fold(ulse[g], reinterpret_cast<const float4 *>(uo + g * D)[d4]);
    for (int c = 0; c < cpieces; ++c)              // the cascade's pieces of the prefix
      fold(clse[c * G + g], reinterpret_cast<const float4 *>(co + (c * G + g) * D)[d4]);
    for (int s0 = p0; s0 <= p1; s0 += U) {
      float l[U];
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool ok = s0 + u <= p1;
        l[u] = ok ? __ldg(lse_part + slot(s0 + u) * Gu + gu) : -INFINITY;
        x[u] = ok ? __ldg(reinterpret_cast<const float4 *>(o_part + (slot(s0 + u) * Gu + gu) * D) + d4)
                  : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float bm = l[0];
#pragma unroll
      for (int u = 1; u < U; ++u) bm = fmaxf(bm, l[u]);
      if (bm > M) {                                // raise M once per batch
        const float r = expf(M - bm);
        num = make_float4(num.x * r, num.y * r, num.z * r, num.w * r);
        den *= r;
        M = bm;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float w = l[u] == -INFINITY ? 0.f : expf(l[u] - M);
        num.x += w * x[u].x;
        num.y += w * x[u].y;
        num.z += w * x[u].z;
        num.w += w * x[u].w;
        den += w;
      }
    }
    const float inv = 1.f / den;
    reinterpret_cast<float4 *>(o)[e] = make_float4(num.x * inv, num.y * inv, num.z * inv,
                                                   num.w * inv);
  }
}

// pa_merge_lse: one warp per query head (b, h), a CTA per (sequence, KV head) group.
// Partials of the head are o_part[b][h][i][:], lse[b][h][i] for i < S; an lse of -inf
// (or a weight that underflows to 0) marks an empty slot, whose o row is not read.
// Lane i reads slot i of each 32-slot chunk: the running maximum and the normaliser take
// warp reductions, and only the non-empty slots' o rows are read (each row coalesced
// over the warp, D / 32 elements per lane).  A head with no partial gets zeros.
template <int D>
__global__ void __launch_bounds__(512) merge_parts_kernel(float *out, const float *o_part,
                                                          const float *lse, int G, int S) {
  pdl_trigger();
  pdl_wait();
  constexpr int E = D / 32;   // elements per lane
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t r = static_cast<size_t>(blockIdx.x) * G + warp;   // head row b * Hq + h
  const float *lr = lse + r * S;
  const float *orow = o_part + r * S * D;
  float M = -INFINITY;
  for (int s0 = 0; s0 < S; s0 += 32)
    M = fmaxf(M, s0 + lane < S ? __ldg(lr + s0 + lane) : -INFINITY);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  float acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  float den = 0.f;
  if (M != -INFINITY) {
    for (int s0 = 0; s0 < S; s0 += 32) {
      const float l = s0 + lane < S ? __ldg(lr + s0 + lane) : -INFINITY;
      const float w = l == -INFINITY ? 0.f : expf(l - M);
      den += w;
      // the live slots' rows in increasing slot order, four rows' loads in flight at
      // once (a head of a long sequence has tens of live slots)
      for (uint32_t live = __ballot_sync(0xffffffffu, w > 0.f); live;) {
        constexpr int U = 4;
        float wj[U], x[U][E];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int j = live ? __ffs(live) - 1 : -1;   // warp-uniform
          live &= live - 1;
          wj[u] = __shfl_sync(0xffffffffu, w, j < 0 ? 0 : j);
          const float *row = orow + static_cast<size_t>(s0 + (j < 0 ? 0 : j)) * D;
#pragma unroll
          for (int e = 0; e < E; ++e) x[u][e] = j < 0 ? 0.f : __ldg(row + e * 32 + lane);
          if (j < 0) wj[u] = 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[e] += wj[u] * x[u][e];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  }
  const float inv = den > 0.f ? 1.f / den : 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) out[r * D + e * 32 + lane] = acc[e] * inv;
}

// ----------------------------------------------------------------------------
// host side
// ----------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                         cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// 2D view of a pool: rows = nblocks * bs tokens, columns = one token's Hkv head rows
// (bf16 elements, or bytes for the code pools); box = 16 rows x one head row of up to
// 128 bytes, swizzled by the box width (128 or 64 bytes).
// s: the decode's view of the shape (Hkv counts units of `heads` adjacent KV heads).
bool make_pool_map(CUtensorMap *map, const void *pool, const pa_shape &s, int heads) {
  auto fn = encode_fn();
  if (!fn) return false;
  const bool bf16 = s.kv_dtype == PA_KV_BF16;
  const int row_bytes = heads * (s.kv_dtype == PA_KV_INT4 ? s.D / 2 : (bf16 ? 2 * s.D : s.D));
  const int box_bytes = row_bytes < 128 ? row_bytes : 128;
  const int eb = bf16 ? 2 : 1;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(s.Hkv) * row_bytes / eb,
                        static_cast<cuuint64_t>(s.nblocks) * s.block_size};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(s.Hkv) * row_bytes};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(box_bytes / eb), static_cast<cuuint32_t>(kTile)};
  cuuint32_t estr[2] = {1, 1};
  // promote L2 fills to one head row: 256 B for bf16 D = 128, 128 B for 128-byte
  // rows, none for 64-byte rows (a wider fill would pull in the next head's row)
  const CUtensorMapL2promotion promo =
      row_bytes >= 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                       : (row_bytes >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                           : CU_TENSOR_MAP_L2_PROMOTION_NONE);
  CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                  const_cast<void *>(pool), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  box_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, promo,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// CTAs per (sequence, KV head) unit in pa_decode.  With at most two units per resident
// CTA, one long sequence would be left to a single CTA at the end of the launch: such
// batches get a cluster of four CTAs per unit (of which a short unit keeps only as
// many as it has tiles for).  Larger batches keep one CTA per unit.  So do launches
// whose window or page selection bounds every unit's tiles when the units fill the GPU
// (bounded units are near-uniform: a cluster would only add CTAs), and launches whose
// bound is one CTA's share (the cluster's other CTAs would all sit idle).
template <class C>
static int pair_cluster_ctas(int units, int resident_ctas, int window, int topk) {
  if (units > 2 * resident_ctas) return 1;
  const bool bounded = topk > 0 || window > 0;
  if (bounded && units >= resident_ctas) return 1;
  const int share = kClusterWarpTiles * C::WARPS;   // tiles one CTA takes before another joins
  const int max_tiles = topk > 0 ? topk : (window > 0 ? (window + kTile - 2) / kTile + 1 : 1 << 30);
  return max_tiles <= share ? 1 : 4;
}

// pa_decode without a workspace on a bf16 batch of more units than two per resident
// CTA (and at most kPersistMaxUnits), with no window or page selection: one persistent
// CTA of eight warps per SM on a static water-filled schedule.
template <class C>
static pa_status launch_persist(const Params &p, const CUtensorMap &mk, const CUtensorMap &mv,
                                cudaStream_t stream, int sms) {
  using P = PersistCfg<C>;
  if (prep_kernel(decode_persist_kernel<P>, P::SMEM) != cudaSuccess) return PA_ERR_CUDA;
  return launch_pdl(decode_persist_kernel<P>, dim3(sms), dim3(P::THREADS), P::SMEM, stream, mk, mv,
                    p) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

template <class C>
static pa_status launch_pair_units(const Params &p, const CUtensorMap &mk, const CUtensorMap &mv,
                                   cudaStream_t stream) {
  const int units = p.B * p.Hkv;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  if constexpr (C::KIND == kKindBf16 && C::NT == 1) {
    // (every sum of tiles the schedule forms stays below 2^31)
    const long long max_tiles = (static_cast<long long>(p.max_blocks) * p.bs + kTile - 1) / kTile;
    if (units > 2 * sms * C::MIN_BLOCKS && units <= kPersistMaxUnits && sms <= kPersistMaxBins &&
        p.window == 0 && p.topk == 0 && units * max_tiles < (1ll << 30))
      return launch_persist<C>(p, mk, mv, stream, sms);
  }
  const int ncl = pair_cluster_ctas<C>(units, sms * C::MIN_BLOCKS, p.window, p.topk);
  auto one_cta_per_unit = [&]() {
    if (prep_kernel(decode_pair_kernel<C, false>, C::PAIR_SMEM) != cudaSuccess) return PA_ERR_CUDA;
    decode_pair_kernel<C, false><<<units, C::THREADS, C::PAIR_SMEM, stream>>>(mk, mv, p);
    return cudaGetLastError() == cudaSuccess ? PA_OK : PA_ERR_CUDA;
  };
  if (ncl == 1) return one_cta_per_unit();
  if (prep_kernel(decode_pair_kernel<C, true>, C::PAIR_SMEM) != cudaSuccess) return PA_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * ncl);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::PAIR_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ncl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, decode_pair_kernel<C, true>, mk, mv, p) == cudaSuccess) return PA_OK;
  // a device (or a partition of one) that cannot place the cluster: the same
  // decode with one CTA per unit (the failed launch left no sticky error)
  (void)cudaGetLastError();
  return one_cta_per_unit();
}

// pa_decode without a workspace reads E4M3 heads singly (heads_per_unit), so the paired
// E4M3 kind has no instantiation of its kernel.
template <class C>
static pa_status launch_pair(const Params &p, const CUtensorMap &mk, const CUtensorMap &mv,
                             cudaStream_t stream) {
  if constexpr (C::KIND == kKindFp8x2)
    return PA_ERR_UNSUPPORTED;
  else
    return launch_pair_units<C>(p, mk, mv, stream);
}

// s: the unit view; p.G query heads per unit
static pa_status dispatch_pair(const pa_shape &s, int heads, const Params &p,
                               const CUtensorMap &mk, const CUtensorMap &mv, cudaStream_t st) {
  const int nt = (p.G + 7) / 8;
  const int kind = kind_of(s, heads);
  PA_DISPATCH_ALL(launch_pair, p, mk, mv, st)
  return PA_ERR_UNSUPPORTED;
}

static pa_status dispatch_segments(const pa_shape &s, int heads, const Params &p,
                                   const CUtensorMap &mk, const CUtensorMap &mv,
                                   cudaStream_t st) {
  const int nt = (p.G + 7) / 8;
  const int kind = kind_of(s, heads);
  PA_DISPATCH_ALL(launch_segments, p, mk, mv, st)
  return PA_ERR_UNSUPPORTED;
}

template <class C>
static int cfg_split_smem(int B) { return split_smem<C>(B); }
template <class C>
static int cfg_min_blocks(int) { return C::MIN_BLOCKS; }

// Sizing of the split kernel a decode with these options (NULL: none) launches.
int splitkv_smem_bytes(const pa_shape &shape, const pa_decode_opts *opts) {
  const int heads = heads_per_unit(shape, opts, opts && opts->num_prefix_groups > 0);
  const pa_shape s = unit_view(shape, heads);
  const int nt = (s.Hq / s.Hkv + 7) / 8;
  const int kind = kind_of(s, heads);
  PA_DISPATCH_ALL(cfg_split_smem, s.B)
  return 0;
}

int decode_warps_per_cta() { return Cfg<128, 1, false>::WARPS; }

int splitkv_min_blocks(const pa_shape &shape, const pa_decode_opts *opts) {
  const int heads = heads_per_unit(shape, opts, opts && opts->num_prefix_groups > 0);
  const pa_shape s = unit_view(shape, heads);
  const int nt = (s.Hq / s.Hkv + 7) / 8;
  const int kind = kind_of(s, heads);
  PA_DISPATCH_ALL(cfg_min_blocks, 0)
  return 1;
}

// prefix int32[B + 4] (tile prefix, KV heads per unit, cascade workspace address),
// lse f32[splits][2][Gu],
// o_part f32[splits][2][Gu][D]; Gu = query heads of the largest unit the shape allows.
WorkspaceLayout splitkv_layout(const pa_shape &s, int num_splits) {
  WorkspaceLayout w{};
  auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
  const size_t G = static_cast<size_t>(s.Hq / s.Hkv) * (pairable(s) ? 2 : 1);
  w.prefix = 0;
  w.lse = up(w.prefix + (static_cast<size_t>(s.B) + 4) * 4);
  w.o_part = up(w.lse + static_cast<size_t>(num_splits) * 2 * G * 4);
  w.total = up(w.o_part + static_cast<size_t>(num_splits) * 2 * G * s.D * 4);
  return w;
}

pa_status run_decode(const pa_shape &s, float *out, const void *q, const void *k_pool,
                     const void *v_pool, const float *k_scale, const float *v_scale,
                     const int32_t *bt, const int32_t *sl, const pa_decode_opts *opts,
                     float sm_scale, int32_t *err, cudaStream_t stream) {
  const int heads = heads_per_unit(s, opts, false, true);
  const pa_shape v = unit_view(s, heads);
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, k_pool, v, heads) || !make_pool_map(&mv, v_pool, v, heads))
    return PA_ERR_CUDA;
  Params p = make_params(v, out, q, k_scale, v_scale, bt, sl, opts, sm_scale, err);
  p.shared_prefix_lens = opts ? opts->shared_prefix_lens : nullptr;
  return dispatch_pair(v, heads, p, mk, mv, stream);
}

pa_status run_decode_splitkv(const pa_shape &s, float *out, void *workspace, int num_splits,
                             const void *q, const void *k_pool, const void *v_pool,
                             const float *k_scale, const float *v_scale, const int32_t *bt,
                             const int32_t *sl, const pa_decode_opts *opts, float sm_scale,
                             int32_t *err, cudaStream_t stream) {
  const WorkspaceLayout w = splitkv_layout(s, num_splits);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  const int heads = heads_per_unit(s, opts, opts && opts->num_prefix_groups > 0);
  const pa_shape v = unit_view(s, heads);
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, k_pool, v, heads) || !make_pool_map(&mv, v_pool, v, heads))
    return PA_ERR_CUDA;
  Params p = make_params(v, out, q, k_scale, v_scale, bt, sl, opts, sm_scale, err);
  p.shared_prefix_lens = opts ? opts->shared_prefix_lens : nullptr;
  p.prefix_out = reinterpret_cast<int32_t *>(ws + w.prefix);
  p.lse_part = reinterpret_cast<float *>(ws + w.lse);
  p.o_part = reinterpret_cast<float *>(ws + w.o_part);
  p.num_splits = num_splits;
  if (!opts || opts->num_prefix_groups <= 0) return dispatch_segments(v, heads, p, mk, mv, stream);

  // Cascade: plan on the caller's stream.  Given a side stream, fork: the cascade
  // kernel (tensor work on the shared prefixes) runs there with one CTA per SM, next
  // to the split kernel (HBM streaming of the rest, two CTAs per SM); a second cascade
  // launch after the split kernel takes the items still left at full occupancy; the
  // caller's stream waits for both before anything it runs next (the merge).  Without
  // one, the cascade runs after the split kernel on the caller's stream.
  pa_status st = run_cascade_plan(v, *opts, err, stream);
  if (st != PA_OK) return st;
  const CascadeLayout cl = cascade_layout(s.B, s.Hq, s.D);
  p.casc_tiles =
      reinterpret_cast<const int32_t *>(static_cast<const uint8_t *>(opts->cascade_workspace) + cl.tiles);
  p.casc_ws = reinterpret_cast<uint64_t>(opts->cascade_workspace);
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return PA_ERR_CUDA;
  cudaStream_t side = reinterpret_cast<cudaStream_t>(opts->cascade_stream);
  cudaEvent_t fork = reinterpret_cast<cudaEvent_t>(opts->cascade_events[0]);
  cudaEvent_t join = reinterpret_cast<cudaEvent_t>(opts->cascade_events[1]);
  if (side) {
    if (cudaEventRecord(fork, stream) != cudaSuccess || cudaStreamWaitEvent(side, fork, 0) != cudaSuccess)
      return PA_ERR_CUDA;
    st = run_cascade(v, mk, mv, q, bt, k_scale, v_scale, *opts, sm_scale, err, sms, side);
    if (st != PA_OK) return st;
    if (cudaEventRecord(join, side) != cudaSuccess) return PA_ERR_CUDA;
  }
  st = dispatch_segments(v, heads, p, mk, mv, stream);
  if (st != PA_OK) return st;
  st = run_cascade(v, mk, mv, q, bt, k_scale, v_scale, *opts, sm_scale, err, 3 * sms, stream);
  if (st != PA_OK) return st;
  if (side && cudaStreamWaitEvent(stream, join, 0) != cudaSuccess) return PA_ERR_CUDA;
  return PA_OK;
}

pa_status run_decode_parts(const pa_shape &s, float *o_part, float *lse, int S, int workers,
                           const void *q, const void *k_pool, const void *v_pool,
                           const float *k_scale, const float *v_scale, const int32_t *bt,
                           const int32_t *sl, const pa_decode_opts *opts, float sm_scale,
                           int32_t *err, cudaStream_t stream) {
  const int heads = heads_per_unit(s, opts);
  const pa_shape v = unit_view(s, heads);
  CUtensorMap mk, mv;
  if (!make_pool_map(&mk, k_pool, v, heads) || !make_pool_map(&mv, v_pool, v, heads))
    return PA_ERR_CUDA;
  Params p = make_params(v, nullptr, q, k_scale, v_scale, bt, sl, opts, sm_scale, err);
  p.shared_prefix_lens = opts ? opts->shared_prefix_lens : nullptr;
  p.num_splits = workers;
  p.parts_S = S;
  p.parts_o = o_part;
  p.parts_lse = lse;
  return dispatch_segments(v, heads, p, mk, mv, stream);
}

pa_status run_merge_parts(const pa_shape &s, float *out, const float *o_part, const float *lse,
                          int S, cudaStream_t stream) {
  const int G = s.Hq / s.Hkv;   // <= 16: a CTA of at most 512 threads
  const dim3 grid(s.B * s.Hkv), block(32 * G);
  const cudaError_t e =
      s.D == 128 ? launch_pdl(merge_parts_kernel<128>, grid, block, 0, stream, out, o_part, lse, G, S)
                 : launch_pdl(merge_parts_kernel<64>, grid, block, 0, stream, out, o_part, lse, G, S);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

pa_status run_merge(const pa_shape &s, float *out, const void *workspace, int num_splits,
                    cudaStream_t stream) {
  const WorkspaceLayout w = splitkv_layout(s, num_splits);
  const uint8_t *ws = static_cast<const uint8_t *>(workspace);
  const int G = s.Hq / s.Hkv;
  // a CTA per (sequence, KV head); with thousands of them (large batches, where most
  // units finished inside one segment and exit at once) smaller CTAs keep more resident
  const int cap = s.B * s.Hkv >= 2048 ? 128 : 256;
  const int threads = min(cap, max(32, ((G * s.D / 4) + 31) / 32 * 32));
  return launch_pdl(merge_kernel, dim3(s.B * s.Hkv), dim3(threads), 0, stream, out,
                    reinterpret_cast<const int32_t *>(ws + w.prefix),
                    reinterpret_cast<const float *>(ws + w.o_part),
                    reinterpret_cast<const float *>(ws + w.lse), s.B, s.Hq, s.Hkv, G, s.D,
                    num_splits) == cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

}  // namespace pa
