// Decode attention for a batch whose requests share a prefix (a cached prompt): the keys of the
// prefix are read and multiplied once for all requests, the rest request by request.
//
// Softmax attention over a key set that is split into parts needs of each part only
//   m = max s,  l = sum 2^(s - m),  O = sum 2^(s - m) v      (s in log2 units)
// and the parts join as M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l. So the work is cut
// into segments (a tile of query rows x a run of 64-key steps) that any CTA may compute, and a
// second kernel joins each row's segments in a fixed order.
//
//  * Prefix. The B*N*G query rows of a KV group form tiles of 128 rows (the M of tcgen05.mma).
//    Two tiles share each K/V step a CTA loads; an odd last tile is handled like private work.
//  * Private keys. A tile is one request's N*G rows (padded to M): the MMAs run far below their
//    rate, but a step's 32 KB take longer to arrive than the padded MMAs take.
//  * CTAs [0, n_s) cut the prefix steps of all tile pairs into equal runs; the other CTAs' two
//    "lanes" cut the private work, steps and what a tile costs besides, into equal runs; n_s
//    follows from the two totals. The plan is made on the GPU from the lengths, so the call can be
//    captured once and replayed with other lengths.
//  * Only whole 64-key steps below every active request's first visible row go to the prefix;
//    its remainder is read through each request's own page table, where it also stands. So the
//    prefix pass needs no mask, and shared_len is a hint about sharing, never about visibility.
//  * A row that does not see one of its request's last N - 1 keys multiplies that key's V by a weight
//    of 0 all the same, and 0 * NaN is NaN. So a warp brings these rows of V by plain loads, with
//    zeros for what is not finite; when there was any, the softmax warps add it to the partials of
//    the rows that see it.
//
// Per lane S = Q K^T (128 x 64 x 128) and O += P V run on tcgen05 with S, P and O in tensor
// memory; one softmax warpgroup per lane keeps the running reference and sum in fp32. P is rounded
// to bf16 for its product, as tensor cores take it (beside V in bf16 the other operand is bf16 too;
// a second product for what is rounded off would be half as many MMAs again). o's relative RMS
// error on random values is 2.3e-3 so, of which the rounding of o itself gives 1.7e-3. P's sum l is
// taken before that rounding. A step is 64 keys because then S has two buffers per lane next to O
// (2 lanes x (2 x 64 + 128) = 512 columns): S(i+1) is ready when the softmax of step i ends, and the
// chain S -> softmax -> O of one step does not bound the rate.
//
// Measured (64 query heads on 8 KV heads, N = 1, one call replayed from a graph): 256 requests on
// 32K shared tokens with 1 to 1024 private ones 253 to 271 us, by the GPU (1030 to 1100 TFLOP/s); 64
// on 64K with 1 to 2048 127 to 132 us (4.1 to 4.3 TB/s); 64 with 1 to 8192 behind 2000 178 us (6.1
// TB/s); 8 on 60K with 1 to 512 53 us (4.8 TB/s). The pairs alone (256 requests, 32K shared tokens,
// one private) run at 1320 TFLOP/s, 70% of what a dense bf16 product reaches: what is left is the
// handover between each step's softmax and MMAs, and the power limit (1360 W in a loop, the SM
// clock at 1.72 to 1.95 GHz). Private work alone (64 requests of 8K tokens) reads 6.6 TB/s, 98% of a
// copy.
// What was slower: one issuer for both lanes (207 -> 260 us), the lanes' softmax taking turns
// (207 -> 292 us), two warpgroups per lane on half of the keys each, four issuers (equal).
#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "softmax_math.cuh"

MSA_DEFINE_ERROR_WORD(spd)

namespace msa {

namespace {

constexpr int kThreads = 512;                    // warpgroups: loads, softmax x 2, MMA issue
constexpr int kLaunchRegs = 128;                 // registers per thread at launch, then split
constexpr int kRegsLoad = 56, kRegsIssue = 56, kRegsSoftmax = 200;
constexpr int kStep = 64;                        // keys per step
constexpr uint32_t kQHalf = 128 * 128;           // 128 rows x 64 channels bf16
constexpr uint32_t kQTile = 2 * kQHalf;
constexpr uint32_t kKvHalf = kStep * 128;        // 64 keys x 64 channels bf16
constexpr uint32_t kKvTile = 2 * kKvHalf;        // K or V of one step: 16 KB
constexpr uint32_t kStage = 2 * kKvTile;         // one load stage: V(i) and K(i + 2)
// Shared memory: two query tiles and a ring of stages. A pair's tiles have 128 rows and leave 5
// stages; private tiles of at most 64 rows leave 6, three per lane instead of two (a stage takes
// about 2500 cycles to arrive and a lane's step 1500).
constexpr int kRing = 5;
constexpr int kMaxStages = 6;
constexpr uint32_t kOffBar = 2 * kQTile + kRing * kStage;
static_assert(kOffBar == kQTile + kMaxStages * kStage, "the two layouts fill the same space");
constexpr uint32_t kTmemCols = 512;              // S buffers of lane X at 128 X, O at 256 + 128 X
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Relative time of one step of one CTA, of a pair and of private lanes with everything running, and
// the steps' time that a private tile's end and beginning take. (Pair costs of 2200, 2600, 3000 and
// 3400: 132, 129, 126 and 137 us for 64 requests on 64K tokens, 267, 266, 267 and 277 us for 256 on
// 32K. Tile costs of 0, 1, 2, 3 and 5: 145, 104, 106, 106 and 110 us for 64 requests of one private
// token on 64K, 79, 65, 65, 66 and 66 us for 256 requests of 1 to 512 tokens.)
constexpr float kPairCost = 2800.f, kPrivateCost = 1500.f;
constexpr int kTileCost = 1;
constexpr float kFarSum = 16384.f;  // of a step's P: beyond it the softmax's reference moves

// A run of steps of one tile: what the roles of a lane need to know of it.
struct __align__(16) Seg {
  int32_t n;          // steps; 0: the lane has no more
  int32_t key0;       // first key
  int32_t b, g;       // page-table row, group
  int32_t seq;        // keys the request holds (INT32_MAX in the prefix)
  int32_t kind;       // 0: pair of prefix tiles, 1: odd prefix tile, 2: one request
  int32_t slot;       // of the partial, within its kind
  int32_t rows;       // valid rows of the tile
  int32_t vis;        // keys that the tile's first row sees (INT32_MAX in the prefix)
  int32_t last;       // 1: the lane's last
  int32_t q_row, pad; // first query row
};
constexpr int kQueue = 4;  // segments a lane's feeder is ahead of the slowest reader
// Rows of V [y, min(z, 64)) of a stage that do not come by bulk copies; z = 0: no more. Each open
// entry has a stage of its own, of which a private lane has at most three: behind these and the
// closing entry nothing is overwritten.
struct Late {
  int32_t y, z, tok, g, slot;
};
constexpr int kLateQueue = 4;
static_assert(kLateQueue == kQueue, "initialised together");

struct Bars {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t q_full[2][2], q_empty[2][2];  // [lane][segment & 1]
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];  // [lane][step & 1]
  uint64_t o_free[2];                    // per segment: O read
  uint64_t seg_full[2][kQueue], seg_free[2][kQueue];
  uint64_t drained[2];
  Seg seg[2][kQueue];
  uint32_t tmem_base;
  int32_t fail;
  // plan
  int32_t w_min[kThreads / 32], w_first[kThreads / 32], w_sum[kThreads / 32];
  int32_t start_b[2], start_rem[2];
  // with late rows
  uint64_t late_full[2][kLateQueue];
  Late late[2][kLateQueue];
  int32_t odd[2];  // a late row of the lane was not finite, in this segment or one before
};
constexpr size_t kSmemBytes = kOffBar + ((sizeof(Bars) + 15) / 16) * 16;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

// V maps with boxes of one channel half of 1, 2, 4, ..., 32 tokens.
struct TailMaps {
  CUtensorMap m[6];
};
__device__ uint4 g_zero_rows[kKvHalf / 16];  // never written

struct KParams {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* shared_len;
  int32_t B, N, G, Hq, Hkv, max_blocks;
  int64_t num_pages;
  int32_t gs, hs;     // log2 of G and Hkv
  int32_t ctas;
  int32_t rows_g;     // B*N*G: query rows of a group
  int32_t tpt;        // tokens per tile: 128 / G
  int32_t pairs;      // pairs of prefix tiles per group
  int32_t abreast;    // pairs that walk the prefix together
  int32_t odd;        // 1: a last unpaired prefix tile
  int32_t units;      // tiles of one request's rows
  int32_t rows_u;     // rows of a request tile (box height): G * min(N, tpt)
  int32_t q_rows;     // rows of a private CTA's query areas: 64, or 128
  int32_t rows_l;     // rows kept of an odd prefix tile's partial: a multiple of 8
  // partials: O as [32 channel quads][rows][4] fp32, then (m, l) per row
  float *po_s, *po_l, *po_u;
  float2 *ml_s, *ml_l, *ml_u;
  // what the join needs to know: the prefix pass's tokens, and the first and last worker of each
  // tile's segments
  int32_t* prefix;
  int2 *range_s, *range_l, *range_u;  // [Hkv, pairs], [Hkv], [B, units, Hkv]
  const uint16_t* v_cache;  // for the late rows
  uint16_t* o;
  float* lse;
};

__device__ __forceinline__ int32_t seq_of(const KParams& p, int b) {
  const int32_t s = p.seq_lens[b];
  const int32_t hi = p.max_blocks * MSA_BLOCK_TOKENS;
  return s < 0 ? 0 : (s > hi ? hi : s);
}
// Private steps of one tile of request b.
__device__ __forceinline__ int32_t private_steps(int32_t seq, int32_t prefix) {
  return seq > prefix ? (seq - prefix + kStep - 1) / kStep : 0;
}
// The same in units of work: what ends and begins a tile counts as kTileCost steps behind its own.
__device__ __forceinline__ int32_t tile_units(int32_t steps) { return steps > 0 ? steps + kTileCost : 0; }
// Items cut into runs of q, the first r of them one item longer: the first item of run w.
__device__ __forceinline__ int32_t run_start(int32_t q, int32_t r, int32_t w) { return w * q + min(w, r); }

struct Plan {
  int32_t prefix;        // tokens of the prefix pass, a multiple of kStep
  int32_t first;         // an active request (its page table gives the prefix's pages)
  int32_t nst;           // prefix steps
  int32_t ts;            // prefix steps of one pair: all groups
  int32_t tp, tpl;       // private units (steps, and kTileCost per tile); of these the odd tiles'
  int32_t n_s, n_p;      // CTAs of either kind
  int32_t runs, w_p;     // runs of the ts steps, private workers: none of them without a step
  int32_t qs, rs, qp, rp;  // ts / runs, ts % runs, tp / w_p, tp % w_p
};

// Walks the segments of one worker's run of steps.
struct Walker {
  int32_t kind, left, worker, index, step, b, u, g, seq, nst;
  int32_t round, x0, len;  // pairs: steps left in this pair's run, the run

  __device__ __forceinline__ void to_request(const KParams& p, const Plan& pl, int32_t from) {
    kind = 2;
    u = g = step = 0;
    b = from;
    nst = 0;
#pragma unroll 1
    for (; b < p.B; ++b) {
      seq = seq_of(p, b);
      nst = private_steps(seq, pl.prefix);
      if (nst > 0) return;
    }
    left = 0;
  }
  // A CTA of pairs: run cta / abreast of the prefix steps, for the pairs cta % abreast,
  // + abreast, ... So the pairs abreast read the same keys at the same time and DRAM once.
  __device__ __forceinline__ void init_pairs(const KParams& p, const Plan& pl, int32_t cta) {
    kind = 0;
    worker = cta / p.abreast;
    u = cta - worker * p.abreast;
    nst = pl.nst;
    x0 = len = left = 0;
    if (worker < pl.runs && u < p.pairs) {
      x0 = run_start(pl.qs, pl.rs, worker);
      len = pl.qs + (worker < pl.rs ? 1 : 0);
      left = len * ((p.pairs - 1 - u) / p.abreast + 1);
      index = x0 / nst;  // the run's first group
      g = index;
      step = x0 -= index * nst;
    }
    round = len;
  }
  // To the private tile behind the current one.
  __device__ __forceinline__ void next_tile(const KParams& p, const Plan& pl) {
    step = 0;
    ++g;
    if (g < p.Hkv || left <= 0) return;
    g = 0;
    if (kind == 1) to_request(p, pl, 0);
    else if (++u == p.units) to_request(p, pl, b + 1);
  }
  // Private worker w; sb/srem: request and offset in it where its run starts, when it starts in
  // a request.
  __device__ __forceinline__ void init_private(const KParams& p, const Plan& pl, int32_t w, int32_t sb,
                                               int32_t srem) {
    worker = w;
    const int32_t start = w < pl.w_p ? run_start(pl.qp, pl.rp, w) : 0;
    left = w < pl.w_p ? pl.qp + (w < pl.rp ? 1 : 0) : 0;
    u = g = b = seq = index = step = nst = 0;
    kind = start < pl.tpl ? 1 : 2;
    if (left > 0) {
      int32_t rest = start;
      nst = pl.nst;
      if (kind == 2) {
        b = sb;
        seq = seq_of(p, b);
        nst = private_steps(seq, pl.prefix);
        rest = srem;
      }
      const int32_t units = tile_units(nst), t = rest / units;
      step = rest - t * units;
      u = t >> p.hs;
      g = t & (p.Hkv - 1);
      if (step >= nst) {  // behind the tile's steps
        left -= units - step;
        next_tile(p, pl);
      }
    }
  }
  // The next segment of lane X into s (n = 0: none is left).
  __device__ __forceinline__ bool next(const KParams& p, const Plan& pl, int X, Seg& s) {
    s.n = 0;
    if (left <= 0) return false;
    s.kind = kind;
    s.n = min(kind == 0 ? round : left, nst - step);
    left -= s.n;
    const bool begins = step == 0, ends = step + s.n == nst;
    int2* range;
    s.key0 = step * kStep;
    s.g = g;
    s.b = pl.first;
    s.seq = s.vis = INT32_MAX;
    if (kind == 2) {
      const int32_t t0 = u * p.tpt;
      const int32_t unit = ((b * p.units + u) << p.hs) | g;
      s.key0 += pl.prefix;
      s.slot = worker + unit;
      s.b = b;
      s.seq = seq;
      s.vis = seq - p.N + t0 + 1;
      s.rows = min(p.rows_u, (p.N - t0) << p.gs);
      s.q_row = b * p.N + t0;
      range = p.range_u + unit;
    } else {
      const int32_t tile = kind == 0 ? 2 * u + X : 2 * p.pairs;
      s.rows = min(128, p.rows_g - tile * 128);
      s.q_row = tile * p.tpt;
      s.slot = kind == 0 ? (worker + g) * p.pairs + u : worker + g;
      range = kind == 0 ? p.range_s + g * p.pairs + u : p.range_l + g;
    }
    if (kind == 0) {
      step = 0;
      ++g;
      round -= s.n;
      if (round == 0) {
        u += p.abreast;
        round = len;
        g = index;
        step = x0;
      }
    } else if (ends) {
      left -= kTileCost;
      next_tile(p, pl);
    }
    s.last = left <= 0;
    if ((threadIdx.x & 31) == 0) {
      if (begins) range->x = worker;
      if (ends) range->y = worker;
    }
    return true;
  }
};

// A worker of n steps loads n + 1 stages, in the order in which the MMAs use them: stage 0 holds
// K(0) and K(1), stage i + 1 holds V(i) and K(i + 2).
struct RingPos {
  int32_t slot;
  uint32_t phase;  // parity of the slot's current use
  __device__ __forceinline__ void advance(int32_t len) {
    if (++slot == len) {
      slot = 0;
      phase ^= 1u;
    }
  }
};

// Bounded wait of a converged warp; every thread gets the same answer. The flag that another
// role's timeout sets is read only while the phase is open: on the way through a barrier that
// has completed it would cost a second shared-memory trip.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, volatile int32_t* fail) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *fail != 0)) return false;
  }
  msa_record_error(kErrTimeout);
  *fail = 1;
  return false;
}

// A value that is the same in all threads of a converged warp, in a form that lets the compiler see
// it: operands of tensor-core and bulk-copy instructions that it cannot prove uniform cost a loop
// over the threads each (the issuers were 70 KB of code, and bound by it).
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// wait_or_fail for two barriers at once: half of the warp tests either.
__device__ __forceinline__ bool wait_two_or_fail(uint32_t bar0, uint32_t par0, uint32_t bar1,
                                                 uint32_t par1, volatile int32_t* fail) {
  const bool lo = (threadIdx.x & 16) == 0;
  const uint32_t bar = lo ? bar0 : bar1, par = lo ? par0 : par1;
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait_addr(bar, par))) return true;
    if (__any_sync(0xffffffffu, *fail != 0)) return false;
  }
  msa_record_error(kErrTimeout);
  *fail = 1;
  return false;
}

// Half of S = Q K^T: the four K-16 products of one channel half of 128-byte-swizzled tiles, issued
// by one elected lane of the converged warp.
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t qd, uint64_t kd, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 a, b;\n"
      " elect.sync _|e, 0xffffffff;\n setp.ne.b32 t, 0, 1;\n setp.ne.b32 f, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n"
      " add.s64 a, %1, 2;\n add.s64 b, %2, 2;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 4;\n add.s64 b, %2, 4;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n"
      " add.s64 a, %1, 6;\n add.s64 b, %2, 6;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n}" ::"r"(d),
      "l"(qd), "l"(kd), "r"(idesc), "r"(accumulate)
      : "memory");
}
// O (+)= P V: four K-16 products, P in tensor memory (8 columns per 16 keys), V rows 2 KB apart.
__device__ __forceinline__ void issue_o(uint32_t d, uint32_t p_tmem, uint64_t vd, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred e, t, f;\n .reg .b64 b;\n .reg .b32 a;\n"
      " elect.sync _|e, 0xffffffff;\n setp.ne.b32 t, 0, 1;\n setp.ne.b32 f, %4, 0;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n"
      " add.s32 a, %1, 8;\n add.s64 b, %2, 128;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 16;\n add.s64 b, %2, 256;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n"
      " add.s32 a, %1, 24;\n add.s64 b, %2, 384;\n"
      " @e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n}" ::"r"(d),
      "r"(p_tmem), "l"(vd), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Two bf16 numbers, zero in the place of one that is not finite.
__device__ __forceinline__ uint32_t finite_bf16x2(uint32_t x) {
  if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
  if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
  return x;
}
__device__ __forceinline__ void st_shared_v2(uint32_t at, uint2 x) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(x.x), "r"(x.y) : "memory");
}

template <bool LATE>
__global__ void __launch_bounds__(kThreads, 1)
    shared_prefix_kernel(const __grid_constant__ CUtensorMap qmap_t,
                         const __grid_constant__ CUtensorMap qmap_o,
                         const __grid_constant__ CUtensorMap qmap_u,
                         const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap,
                         const __grid_constant__ TailMaps vtail, const __grid_constant__ KParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // 1024: the swizzle atoms
  Bars& B = *reinterpret_cast<Bars*>(smem + kOffBar);
  volatile int32_t* fail = &B.fail;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = uniform(tid >> 5);
  if (smem_u32(smem) & 1023u) {  // not seen: the declared alignment is kept
    msa_record_error(kErrTimeout);
    return;
  }
  if (tid == 64) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&B.kv_full[i], 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(&B.o_free[x], 4);
      mbar_init(&B.drained[x], 1);
      for (int i = 0; i < kQueue; ++i) {
        mbar_init(&B.seg_full[x][i], 1);
        if (LATE) mbar_init(&B.late_full[x][i], 1);
        mbar_init(&B.seg_free[x][i], 6);  // readers: four softmax warps, an issuer, a K/V producer
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(&B.q_full[x][i], 1);
        mbar_init(&B.q_empty[x][i], 1);
        mbar_init(&B.s_full[x][i], 1);
        mbar_init(&B.o_full[x][i], 1);
        mbar_init(&B.p_full[x][i], 4);
      }
    }
    B.fail = 0;
    if (LATE) B.odd[0] = B.odd[1] = 0;
    mbar_fence_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(&B.tmem_base)), "n"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
    tma_prefetch_desc(&qmap_t);
    tma_prefetch_desc(&qmap_u);
    tma_prefetch_desc(&qmap_o);
  }
  // What precedes this kernel in the stream ends here: lengths, queries and caches are its output,
  // the workspace was its join's input. The join in turn may be scheduled as CTAs of this kernel
  // leave; it waits for all of their stores.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // ------------------------------------------------------------------ plan
  Plan pl;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int pb0 = min(p.B, tid * per), pb1 = min(p.B, pb0 + per);
  {
    const int32_t want = p.shared_len[0];
    const int32_t seq0 = pb0 < pb1 ? seq_of(p, pb0) : 0;
    auto seq_at = [&](int b) { return b == pb0 ? seq0 : seq_of(p, b); };
    int32_t vis = INT32_MAX, first = INT32_MAX;  // keys every active row sees; first active request
#pragma unroll 1
    for (int b = pb0; b < pb1; ++b) {
      const int32_t s = seq_at(b);
      if (s > 0) {
        vis = min(vis, max(0, s - p.N + 1));
        first = min(first, b);
      }
    }
    vis = __reduce_min_sync(0xffffffffu, vis);
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0) {
      B.w_min[warp] = vis;
      B.w_first[warp] = first;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      vis = min(vis, B.w_min[w]);
      first = min(first, B.w_first[w]);
    }
    const bool any = first != INT32_MAX;
    pl.first = any ? first : 0;
    pl.prefix = any ? max(0, min(want, vis)) / kStep * kStep : 0;
    pl.nst = pl.prefix / kStep;
    pl.ts = p.pairs > 0 ? p.Hkv * pl.nst : 0;
    pl.tpl = p.odd ? p.Hkv * tile_units(pl.nst) : 0;
    const int32_t tiles = p.units * p.Hkv;
    int32_t sum = 0;  // units of the requests
#pragma unroll 1
    for (int b = pb0; b < pb1; ++b) {
      sum += tile_units(private_steps(seq_at(b), pl.prefix)) * tiles;
    }
    int32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) B.w_sum[warp] = incl;
    __syncthreads();
    int32_t before = incl - sum, total = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += B.w_sum[w];
      total += B.w_sum[w];
    }
    pl.tp = pl.tpl + total;
    // CTAs of either kind: the split whose slower side is faster
    const int32_t C = gridDim.x;
    if (pl.ts == 0) {
      pl.runs = 0;
    } else {
      const float cs = kPairCost * p.pairs * pl.ts, cp = kPrivateCost * pl.tp;
      const int32_t most = max(1, (C - (pl.tp > 0 ? 1 : 0)) / p.abreast);
      auto slower = [&](int32_t runs) {
        const int32_t n = runs * p.abreast;
        return fmaxf(cs / n, pl.tp > 0 ? cp / max(1, C - n) : 0.f);
      };
      const int32_t lo = max(1, min(most, (int32_t)(C * (cs / (cs + cp)) / p.abreast)));
      const int32_t hi = min(most, lo + 1);
      pl.runs = min(pl.ts, slower(lo) <= slower(hi) ? lo : hi);
    }
    pl.n_s = pl.runs * p.abreast;
    pl.n_p = C - pl.n_s;
    pl.w_p = min(2 * pl.n_p, pl.tp);
    const uint32_t runs = max(1, pl.runs), w_p = max(1, pl.w_p);
    pl.qs = (uint32_t)pl.ts / runs;
    pl.rs = pl.ts - pl.qs * runs;
    pl.qp = (uint32_t)pl.tp / w_p;
    pl.rp = pl.tp - pl.qp * w_p;
    // where the two lanes of this CTA start, when they start in a request
    const bool priv = (int)blockIdx.x >= pl.n_s;
#pragma unroll 1
    for (int x = 0; x < 2; ++x) {
      const int32_t wk = x * pl.n_p + (int)blockIdx.x - pl.n_s;
      if (!priv || wk >= pl.w_p) break;
      const int32_t at = run_start(pl.qp, pl.rp, wk) - pl.tpl;
      if (at >= before && at < before + sum) {
        int32_t rem = at - before;
        int b = pb0;
#pragma unroll 1
        for (; b < pb1; ++b) {
          const int32_t c = tile_units(private_steps(seq_at(b), pl.prefix)) * tiles;
          if (rem < c) break;
          rem -= c;
        }
        B.start_b[x] = b;
        B.start_rem[x] = rem;
      }
    }
    if (blockIdx.x == 0) {
      bool bad = false;
#pragma unroll 1
      for (int b = pb0; b < pb1; ++b) bad |= seq_at(b) != p.seq_lens[b];
      if (bad) msa_record_error(kErrBadBlock);
      if (tid == 0) *p.prefix = pl.prefix;
    }
  }
  const bool shared = (int)blockIdx.x < pl.n_s;
  if (tid == 64) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&B.kv_empty[i], shared ? 2 : 1);  // lanes that read it
    mbar_fence_init();
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform((int32_t)B.tmem_base);
  const uint32_t sbase = smem_u32(smem);
  const bool wide = shared || p.q_rows == 128;          // query areas of 128 rows
  const uint32_t q_half = wide ? kQHalf : kQHalf / 2;   // a channel half of one
  const uint32_t off_ring = 4 * q_half;
  const int32_t lane_ring = wide ? 2 : 3;               // stages of a private lane
  const int32_t rlen = shared ? kRing : lane_ring;
  const bool has_late = LATE && !shared;
  // request tiles that leave half of their area free are double-buffered
  const bool twice = !shared && 2 * p.rows_u <= p.q_rows;
  static_assert(128 * (kRegsLoad + kRegsIssue) + 256 * kRegsSoftmax == kThreads * kLaunchRegs,
                "register split");
  // The next segment of lane X (its k-th) for one of its readers.
  auto take = [&](int X, int32_t& k, Seg& s) {
    const int q = k & (kQueue - 1);
    if (!wait_or_fail(&B.seg_full[X][q], (k / kQueue) & 1, fail)) return false;
    const Seg& e = B.seg[X][q];
    s = {uniform(e.n),    uniform(e.key0), uniform(e.b),   uniform(e.g),     uniform(e.seq),   uniform(e.kind),
         uniform(e.slot), uniform(e.rows), uniform(e.vis), uniform(e.last),  uniform(e.q_row), 0};
    __syncwarp();
    mbar_arrive_if(&B.seg_free[X][q], lane == 0);
    ++k;
    return true;
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    const int X = warp & 1;
    const int32_t rbase = shared ? 0 : X * lane_ring;
    if (shared && warp == 1) {
      // a pair has one K/V producer, on lane 0: nothing to load here, but lane 1's feeder counts on
      // a reader
      int32_t k = 0;
      Seg s;
      while (take(1, k, s) && s.n > 0) {
      }
    } else if (warp < 2) {
      // ============================================================== K/V producers
      // warp 0 for lane 0 or a pair, warp 1 for lane 1
      RingPos r{0, 0};
      int32_t used = 0;                                 // stages begun
      int32_t tok1 = 0, g1 = 0, z1 = 0, tok2 = 0, g2 = 0, z2 = 0;  // steps i - 1 and i - 2
      bool good = true;
      // Of a step in which the request has z more keys: the first late one (kStep: none), how many.
      auto late_from = [&](int32_t z) { return max(0, min(z - (p.N - 1), kStep)); };
      auto late_rows = [&](int32_t z) { return LATE ? max(0, min(z, kStep) - late_from(z)) : 0; };
      // To the lane's late-row warp: the late rows of V's step i - 2 for the current stage; z = 0: no more.
      int32_t late_k = 0;
      auto send_late = [&](int32_t z) {
        if (lane == 0) {
          B.late[X][late_k % kLateQueue] = {late_from(z), z, tok2, g2, rbase + r.slot};
          mbar_arrive(&B.late_full[X][late_k % kLateQueue]);
        }
        ++late_k;
      };
      // Opens a stage of that many bytes, whose V has z more keys (INT32_MAX: no V). V's late rows come
      // from the late-row warp, whose arrival is then the stage's.
      auto begin = [&](uint32_t bytes, int32_t z) {
        if (used >= rlen && !wait_or_fail(&B.kv_empty[rbase + r.slot], r.phase ^ 1u, fail)) return false;
        if (LATE && late_rows(z) > 0) {
          if (lane == 0) mbar_expect_tx_only(&B.kv_full[rbase + r.slot], bytes - late_rows(z) * 256);
          send_late(z);
        } else if (lane == 0) {
          mbar_expect_tx(&B.kv_full[rbase + r.slot], bytes);
        }
        __syncwarp();
        ++used;
        return true;
      };
      auto load = [&](const CUtensorMap* map, uint32_t off, int32_t tok, int32_t g) {
        const int32_t ut = uniform(tok), ug = uniform(g), us = uniform(r.slot);
        if (lane == 0)
          tma_load_4d(smem + off_ring + (rbase + us) * kStage + off, map, &B.kv_full[rbase + us], 0, ut,
                      0, ug);
      };
      // V of step i - 2, of which the first z2 rows are the request's. The cache cells behind its
      // last token may hold anything, NaN included, and 0 * NaN is NaN, so those rows are not
      // loaded: zeros come in their place, by the same engine.
      auto load_v = [&]() {
        const int32_t y = LATE ? late_from(z2) : z2;
        if (y >= kStep) {
          load(&vmap, 0, tok2, g2);
          return;
        }
        if (lane < 2) {  // one channel half each
          uint8_t* dst = smem + off_ring + (rbase + r.slot) * kStage + lane * kKvHalf;
          uint64_t* full = &B.kv_full[rbase + r.slot];
          int32_t at = 0;
#pragma unroll 1
          for (int b = 5; b >= 0; --b)
            if (y >> b & 1) {
              tma_load_4d(dst + at * 128, &vtail.m[b], full, 0, tok2 + at, lane, g2);
              at += 1 << b;
            }
          if (LATE) at = min(z2, kStep);
          if (!LATE || at < kStep) bulk_load(dst + at * 128, g_zero_rows, (kStep - at) * 128, full);
        }
        __syncwarp();
      };
      // the token rows of 32 steps from j on, one per thread
      auto look_up = [&](const Seg& s, int32_t j) {
        const int32_t jj = j + lane, key = s.key0 + jj * kStep;
        return jj < s.n ? p.page_table[(int64_t)s.b * p.max_blocks + key / MSA_BLOCK_TOKENS] : 0;
      };
      int32_t k = 0, i = 0;
      Seg s, ahead;
      good = take(X, k, s);
      int32_t page = 0, page_ahead = 0;
      if (good) page = look_up(s, 0);
      const bool single = s.n == 1 && s.last;  // one step in all
#pragma unroll 1
      while (good && s.n > 0) {
        if (!(good = take(X, k, ahead))) break;
        page_ahead = look_up(ahead, 0);  // arrives while this segment is loaded
#pragma unroll 1
        for (int32_t j = 0; j < s.n; ++j, ++i) {
          if (j > 0 && (j & 31) == 0) page = look_up(s, j);
          if ((j & 31) == 0) {
            const bool bad = page < 0 || page >= p.num_pages;
            if (bad) page = 0;
            if (__any_sync(0xffffffffu, bad) && lane == 0) msa_record_error(kErrBadPage);
          }
          const int32_t key = s.key0 + j * kStep;
          const int32_t tok = __shfl_sync(0xffffffffu, page, j & 31) * MSA_BLOCK_TOKENS + key % MSA_BLOCK_TOKENS;
          if (i == 0) {
            begin(single ? kKvTile : kStage, INT32_MAX);
            load(&kmap, 0, tok, s.g);
            if (single) r.advance(rlen);
          } else {
            if (i > 1) {
              if (!(good = begin(kStage, z2))) break;
              load_v();
            }
            load(&kmap, kKvTile, tok, s.g);
            r.advance(rlen);
          }
          tok2 = tok1;
          g2 = g1;
          z2 = z1;
          tok1 = tok;
          g1 = s.g;
          z1 = s.seq - key;
          if (LATE && lane < 2 * late_rows(z1)) {  // two lines a row: they are there when V's turn comes
            const uint16_t* v = p.v_cache + ((int64_t)(tok + late_from(z1) + (lane >> 1)) * p.Hkv + s.g) * 128;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(v + (lane & 1) * 64));
          }
        }
        s = ahead;
        page = page_ahead;
      }
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {  // the last two steps' V
        if (good && i > 1 - e && (good = begin(kKvTile, z2))) {
          load_v();
          r.advance(rlen);
        }
        tok2 = tok1;
        g2 = g1;
        z2 = z1;
      }
      if (good && has_late) send_late(0);
      if (!good)  // let the copies in flight land before the CTA leaves
        for (int32_t q = max(0, used - rlen); q < used; ++q)
          mbar_wait(&B.kv_full[rbase + q % rlen], (q / rlen) & 1);
    } else if (warp >= 2) {
      // ============================================================== segments and query tiles
      // Walks the lane's segments for all of its roles (each walking them for itself made the
      // kernel 1.7 times its code, and every step waited for instructions) and loads their queries.
      // Request tiles of at most half the lane's area alternate between its halves, so that the
      // next request's rows are there before the current one's last S.
      Walker w;
      // the first n_p private workers are the CTAs' lanes 0, so few steps spread over all CTAs
      if (shared) w.init_pairs(p, pl, blockIdx.x);
      else w.init_private(p, pl, X * pl.n_p + (int32_t)blockIdx.x - pl.n_s, B.start_b[X], B.start_rem[X]);
      int32_t k = 0, done = 0;  // segments published, query tiles loaded
      bool good = true, alone = true;  // alone: the last tile fills the area
      int32_t kind = -1, q_row = 0, g = 0;  // of segment k - 1
#pragma unroll 1
      for (bool more = true; more;) {
        Seg s;
        more = w.next(p, pl, X, s);
        const int q = k & (kQueue - 1);
        if (k >= kQueue && !(good = wait_or_fail(&B.seg_free[X][q], (k / kQueue - 1) & 1, fail))) break;
        if (lane == 0) {
          B.seg[X][q] = s;
          mbar_arrive(&B.seg_full[X][q]);
        }
        __syncwarp();
        if (k++ > 0) {  // the queries of the segment before
          const bool small = kind == 2 && twice;
          // the segment whose S must have completed before this tile's rows may be overwritten
          const int32_t after = done - (small && !alone ? 2 : 1);
          if (after >= 0 && !(good = wait_or_fail(&B.q_empty[X][after & 1], (after >> 1) & 1, fail))) break;
          if (lane == 0) {
            uint64_t* full = &B.q_full[X][done & 1];
            uint8_t* dst = smem + X * 2 * q_half + (small ? (done & 1) * (q_half / 2) : 0);
            const CUtensorMap* map = kind == 2 ? &qmap_u : (kind == 0 ? &qmap_t : &qmap_o);
            mbar_expect_tx(full, (kind == 2 ? p.rows_u : (kind == 0 ? 128 : p.q_rows)) * 256);
            tma_load_5d(dst, map, full, 0, 0, q_row, 0, g);
            tma_load_5d(dst + q_half, map, full, 0, 0, q_row, 1, g);
          }
          __syncwarp();
          ++done;
          alone = !small;
        }
        kind = s.kind;
        q_row = s.q_row;
        g = s.g;
      }
      if (!good)  // let the copies in flight land before the CTA leaves
        for (int32_t q = max(0, done - 2); q < done; ++q)
          mbar_wait(&B.q_full[X][q & 1], (q >> 1) & 1);
    }
    __syncwarp();
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // ================================================================ MMA issuers, one per lane
    // Warps 12 and 13. In order S(0), S(1), then O(i), S(i+2):
    // O(i) needs P(i) and V(i); S(i+2) needs K(i+2) and overwrites the tensor memory from which
    // O(i) reads P(i), which it may as the tensor pipe runs one thread's MMAs in issue order; the
    // commit that signals S(i+2) covers O(i). The warp runs in lockstep, an elected lane issues.
    if (warp < 14) {
      const int X = warp - 12;
      const int32_t rbase = shared ? 0 : X * lane_ring;
      const uint32_t s_tmem = tmem + X * 128, o_tmem = tmem + 256 + X * 128;
      const uint32_t full0 = smem_u32(&B.kv_full[rbase]), p0 = smem_u32(&B.p_full[X][0]);
      const uint32_t idesc_s = umma_idesc_bf16(128, kStep, 0, 0);
      const uint32_t idesc_o = umma_idesc_bf16(128, 128, 0, 1);
      const uint64_t qd0 = umma_desc_sw128(sbase + X * 2 * q_half, 16, 1024);
      const uint64_t kd0 = umma_desc_sw128(sbase + off_ring + rbase * kStage, 16, 1024);
      const uint64_t vd0 = umma_desc_sw128(sbase + off_ring + rbase * kStage, kKvHalf, 1024);
      Seg s;
      RingPos r{0, 0};
      int32_t k = 0, o_seg = 0;
      bool good = take(X, k, s);
      int32_t left = good ? s.n : 0;  // steps of the segment still to come
      bool more = left > 0;           // S(i+2) exists
      int32_t end = INT32_MAX;        // steps, once known
      uint32_t opens = 4;  // bit j: step i + j is a segment's first
      uint64_t qd = qd0;
      r.advance(rlen);
      if (more) good = wait_or_fail(&B.kv_full[rbase], 0, fail);
      else end = 0;
  #pragma unroll 1
      for (int32_t i = -2; good && i < end; ++i) {
        const uint32_t buf = i & 1;
        if (i >= 0) {
          if ((opens & 1u) && o_seg++ > 0 && !(good = wait_or_fail(&B.o_free[X], o_seg & 1, fail))) break;
          if (!(good = wait_two_or_fail(full0 + r.slot * 8, r.phase, p0 + buf * 8, (i >> 1) & 1, fail))) break;
          tmem_fence_after();
          issue_o(o_tmem, s_tmem + buf * 64, vd0 + r.slot * (kStage >> 4), idesc_o, (opens & 1u) ^ 1u);
          umma_commit_elect(&B.o_full[X][buf]);
        }
        if (more) {
          if (left == 0) {
            if (!(good = take(X, k, s))) break;
            left = s.n;
            opens |= 4u;
          }
          if (opens & 4u) {
            qd = qd0 + (s.kind == 2 && twice ? ((k - 1) & 1) * (q_half / 2 >> 4) : 0);
            if (!(good = wait_or_fail(&B.q_full[X][(k - 1) & 1], ((k - 1) >> 1) & 1, fail))) break;
            tmem_fence_after();
          }
          // K(0) and K(1) are stage 0, K(i+2) is the second half of stage i + 1
          const uint64_t kd = kd0 + (i < 0 ? (i + 2) * (kKvTile >> 4) : r.slot * (kStage >> 4) + (kKvTile >> 4));
          issue_s(s_tmem + buf * 64, qd, kd, idesc_s, 0);
          issue_s(s_tmem + buf * 64, qd + (q_half >> 4), kd + (kKvHalf >> 4), idesc_s, 1);
          umma_commit_elect(&B.s_full[X][buf]);
          if (--left == 0) {
            umma_commit_elect(&B.q_empty[X][(k - 1) & 1]);
            if (s.last) {
              more = false;
              end = i + 3;
            }
          }
        }
        // stage 0 is free after its last S, stage i + 1 after O(i) and S(i+2)
        if (i >= 0) {
          umma_commit_elect(&B.kv_empty[rbase + r.slot]);
          r.advance(rlen);
        } else if (i == -1) {
          umma_commit_elect(&B.kv_empty[rbase]);
        }
        opens >>= 1;
      }
      if (!good) {  // the MMAs in flight end before tensor memory is given back
        umma_commit_elect(&B.drained[X]);
        mbar_wait(&B.drained[X], 0);
      }
    } else if (has_late) {
      // ============================================================== late rows of V, a warp per lane
      // Brings the rows that the producer names, four channels per thread, to the places that the
      // bulk copies' 128-byte swizzle gives them. (16 x 4 rows on 20011 tokens take 47.9 us so, 47.2
      // with all rows by bulk copies, and 50.9 with these loads in the producers' own turn. Without the
      // prefetch, two steps before, 16 x 16 rows take 141.3 us instead of 140.)
      const int X = warp - 14;
#pragma unroll 1
      for (int32_t k = 0;; ++k) {
        if (!wait_or_fail(&B.late_full[X][k % kLateQueue], (k / kLateQueue) & 1, fail)) break;
        const Late e = B.late[X][k % kLateQueue];
        if (e.z <= 0) break;  // no more
        const int32_t z = min(e.z, kStep);
        const uint32_t to = sbase + off_ring + e.slot * kStage + (lane >> 4) * kKvHalf + (lane & 1) * 8;
        const uint2* from = reinterpret_cast<const uint2*>(p.v_cache + ((int64_t)e.tok * p.Hkv + e.g) * 128) + lane;
        bool odd = false;
#pragma unroll 1
        for (int32_t x0 = e.y; x0 < z; x0 += 4) {
          uint2 v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (x0 + u < z) v[u] = from[(int64_t)(x0 + u) * p.Hkv * 32];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int32_t x = x0 + u;
            if (x < z) {
              const uint2 f = make_uint2(finite_bf16x2(v[u].x), finite_bf16x2(v[u].y));
              odd |= f.x != v[u].x || f.y != v[u].y;
              st_shared_v2(to + x * 128 + ((((lane >> 1) & 7) ^ (x & 7)) << 4), f);
            }
          }
        }
        odd = __any_sync(0xffffffffu, odd);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read them by that proxy
        __syncwarp();
        if (lane == 0) {
          if (odd) *(volatile int32_t*)&B.odd[X] = 1;
          mbar_arrive(&B.kv_full[e.slot]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================================================================ softmax + partials
    const int X = (warp - 4) >> 2;
    const int row = (tid - 128) & 127;  // tile row = tensor memory lane
    const uint32_t lane_addr = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_tmem = tmem + lane_addr + X * 128;
    const uint32_t o_tmem = tmem + lane_addr + 256 + X * 128;
    const int32_t token = row >> p.gs;
    int32_t n = 0, k = 0;
    Seg s;
    bool good = true;
#pragma unroll 1
    while (good && take(X, k, s) && s.n > 0) {
      const bool act = 32 * (warp & 3) < s.rows;  // a warp of padding rows only keeps the barriers
      const bool mine = row < s.rows;  // the rows behind hold whatever the query area held before
      float m_run = -INFINITY, l = 0.f;  // running max (log2 units) and sum
      int32_t kb = s.key0;
#pragma unroll 1
      for (int32_t j = 0; j < s.n; ++j, ++n, kb += kStep) {
        if (!(good = wait_or_fail(&B.s_full[X][n & 1], (n >> 1) & 1, fail))) break;
        tmem_fence_after();
        const uint32_t sb = s_tmem + (n & 1) * 64;
        if (act) {
          float l4[4];
          uint32_t pk[32];
          // Any reference near the row's maximum serves for m: P and its sums keep their relative
          // precision as long as nothing overflows. So P is taken against the reference there is,
          // and its sum, needed anyway, tells whether a score lies far above it; only then, and on
          // a segment's first step, a second pass takes the maximum.
#pragma unroll 1
          for (bool exact = j == 0;; exact = true) {
            float v[kStep];
            tmem_ld32(sb, v);
            tmem_ld32(sb + 32, v + 32);
            tmem_wait_ld();
            if (s.vis - kb < kStep) {  // uniform: the step holds a key some row does not see
              const int32_t vis = s.vis + token - kb;
#pragma unroll
              for (int x = 0; x < kStep; ++x)
                if (x >= vis) v[x] = -INFINITY;
            }
            if (exact) {
              float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
              for (int x = 4; x < kStep; x += 2) m4[(x >> 1) & 3] = max3(m4[(x >> 1) & 3], v[x], v[x + 1]);
              const float m2 = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]) * kLog2e;
              float factor = 1.f;
              if (m_run == -INFINITY) {
                m_run = m2;  // nothing in O yet
              } else if (mine && m2 > m_run) {
                factor = ex2(m_run - m2);
                m_run = m2;
                l *= factor;
              }
              if (__any_sync(0xffffffffu, factor != 1.f)) {
                // rescale O once O(n-1) has completed (S(n) says that O(n-2) has, so the barrier's
                // parity is unambiguous)
                if (!(good = wait_or_fail(&B.o_full[X][(n - 1) & 1], ((n - 1) >> 1) & 1, fail))) break;
                tmem_fence_after();
#pragma unroll 1
                for (int c = 0; c < 8; ++c) {
                  uint32_t o[16];
                  tmem_ld16(o_tmem + c * 16, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * factor);
                  tmem_st16(o_tmem + c * 16, o);
                }
              }
            }
            const float off = m_run == -INFINITY ? 0.f : -m_run;
            l4[0] = l4[1] = l4[2] = l4[3] = 0.f;
#pragma unroll
            for (int x = 0; x < kStep; x += 2) {
              fma2(v[x], v[x + 1], v[x], v[x + 1], kLog2e, kLog2e, off, off);
              v[x] = ex2(v[x]);
              v[x + 1] = ex2(v[x + 1]);
              add2(l4[x & 2], l4[(x & 2) + 1], v[x], v[x + 1]);
              pk[x >> 1] = pack_bf16x2(v[x], v[x + 1]);
            }
            l4[0] = (l4[0] + l4[1]) + (l4[2] + l4[3]);
            if (exact || !__any_sync(0xffffffffu, mine && (l4[0] > kFarSum || m_run == -INFINITY))) break;
          }
          if (!good) break;
          l += l4[0];
          tmem_st32(sb, pk);
          tmem_wait_st();
        }
        tmem_fence_before();
        __syncwarp();
        mbar_arrive_if(&B.p_full[X][n & 1], lane == 0);
      }
      if (!good) break;
      // ---------------- the segment's partial
      float4* po = nullptr;
      int32_t cap = 128;
      if (mine) {
        float2* ml;
        if (s.kind == 0) {
          const int64_t slot = (int64_t)s.slot * 2 + X;
          po = reinterpret_cast<float4*>(p.po_s + slot * 128 * 128);
          ml = p.ml_s + slot * 128;
        } else if (s.kind == 1) {
          cap = p.rows_l;
          po = reinterpret_cast<float4*>(p.po_l + (int64_t)s.slot * cap * 128);
          ml = p.ml_l + (int64_t)s.slot * cap;
        } else {
          cap = p.rows_u;
          po = reinterpret_cast<float4*>(p.po_u + (int64_t)s.slot * cap * 128);
          ml = p.ml_u + (int64_t)s.slot * cap;
        }
        ml[row] = make_float2(m_run, l);
        po += row;
      }
      if (!(good = wait_or_fail(&B.o_full[X][(n - 1) & 1], ((n - 1) >> 1) & 1, fail))) break;
      tmem_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float o[64];
        if (act) {
          tmem_ld32(o_tmem + c * 64, o);
          tmem_ld32(o_tmem + c * 64 + 32, o + 32);
          tmem_wait_ld();
        }
        if (c == 1) {  // all of O is read: the next segment may overwrite it
          tmem_fence_before();
          __syncwarp();
          mbar_arrive_if(&B.o_free[X], lane == 0);
        }
        if (mine)
#pragma unroll
          for (int x = 0; x < 16; ++x, po += cap)
            *po = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
      }
      if (LATE && mine && s.kind == 2 && *(volatile int32_t*)&B.odd[X] != 0) {
        // rare: what is not finite in V of the segment's late keys that the row sees (their weights are
        // above 0, so it is added as it is)
        po -= 32 * cap;
        const int32_t end = min(s.vis + token, s.key0 + s.n * kStep);
#pragma unroll 1
        for (int32_t key = max(s.key0, s.seq - p.N + 1); key < end; ++key) {
          int32_t page = p.page_table[(int64_t)s.b * p.max_blocks + key / MSA_BLOCK_TOKENS];
          if (page < 0 || page >= p.num_pages) page = 0;
          const int64_t cell = (int64_t)page * MSA_BLOCK_TOKENS + key % MSA_BLOCK_TOKENS;
          const uint2* v = reinterpret_cast<const uint2*>(p.v_cache + (cell * p.Hkv + s.g) * 128);
#pragma unroll 1
          for (int x = 0; x < 32; ++x) {
            const uint2 f = make_uint2(finite_bf16x2(v[x].x), finite_bf16x2(v[x].y));
            if (f.x == v[x].x && f.y == v[x].y) continue;
            float4 a = po[x * cap];
            a.x += bf16_lo(v[x].x ^ f.x);
            a.y += bf16_hi(v[x].x ^ f.x);
            a.z += bf16_lo(v[x].y ^ f.y);
            a.w += bf16_hi(v[x].y ^ f.y);
            po[x * cap] = a;
          }
        }
      }
    }
  }
  // ------------------------------------------------------------------ teardown
  tmem_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTmemCols)
                 : "memory");
  }
}

// ------------------------------------------------------------------------------ join
// A CTA joins eight consecutive query rows of a group; a thread owns four channels of one row,
// so a warp reads whole 128-byte lines of the partials' [channel quad][row][4] layout. With
// SPLIT > 1 the row's segments are dealt to SPLIT threads, four loads in flight each, and joined
// through shared memory: few rows leave SMs idle and have many segments each (8 requests on 60K
// tokens: 38), which one thread would wait for four by four.
constexpr int kJoinRows = 8;
constexpr int kJoinSplit = 4;

struct Parts {
  const float* o;
  const float2* ml;
  int64_t o_step, ml_step;  // to the next segment of the row
  int32_t n;
};
// First worker and number of workers of a tile, within the slots there are (after a timeout the
// attention kernel may not have written them).
__device__ __forceinline__ int2 worker_range(int2 r, int32_t workers) {
  const int32_t x = max(0, min(r.x, workers - 1));
  return make_int2(x, max(0, min(r.y - x + 1, workers - x)));
}
struct Joined {
  float m, l;
  float4 acc;
};

// Adds up to four parts (n of them valid) to j.
__device__ __forceinline__ void join_four(Joined& j, const float2 (&ml)[4], const float4 (&o)[4], int n) {
  float m = j.m;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < n) m = fmaxf(m, ml[u].x);
  const float f = j.m == m ? 1.f : ex2(j.m - m);  // 2^(-inf) = 0 for the first parts
  j.m = m;
  j.l *= f;
  j.acc.x *= f;
  j.acc.y *= f;
  j.acc.z *= f;
  j.acc.w *= f;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    if (u >= n || (ml[u].x == -INFINITY && ml[u].y == 0.f)) continue;  // the row saw no key there
    const float w = ex2(ml[u].x - m);
    j.l += w * ml[u].y;
    j.acc.x += w * o[u].x;
    j.acc.y += w * o[u].y;
    j.acc.z += w * o[u].z;
    j.acc.w += w * o[u].w;
  }
}

template <int SPLIT>
__global__ void __launch_bounds__(kJoinRows * 32 * SPLIT)
    shared_prefix_join_kernel(const __grid_constant__ KParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t g = blockIdx.x % p.Hkv;
  const int t = threadIdx.x % (kJoinRows * 32), split = threadIdx.x / (kJoinRows * 32);
  const int32_t pr = (int32_t)(blockIdx.x / p.Hkv) * kJoinRows + (t & (kJoinRows - 1));
  const int32_t quad = t / kJoinRows;
  const bool valid = pr < p.rows_g;
  const int32_t r = valid ? pr >> p.gs : 0, e = pr & (p.G - 1), b = r / p.N, i = r - b * p.N;
  Joined j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (valid) {
    // requested together: where the row's segments are, whether there are any
    const int32_t tile = pr >> 7, u = i >> (7 - p.gs);
    const bool paired = tile < 2 * p.pairs;
    const int64_t unit = ((int64_t)b * p.units + u) * p.Hkv + g;
    const int32_t prefix = *p.prefix, seq = seq_of(p, b);
    const int2 ra = worker_range(paired ? p.range_s[g * p.pairs + (tile >> 1)] : p.range_l[g],
                                 paired ? p.ctas / p.abreast : 2 * p.ctas);
    const int2 rc = worker_range(p.range_u[unit], 2 * p.ctas);
    Parts a{}, c{};
    if (prefix > 0 && seq > 0) {  // a padding request's rows sit in the prefix tiles too
      const int32_t row = pr & 127;
      if (paired) {
        const int64_t slot = ((int64_t)(ra.x + g) * p.pairs + (tile >> 1)) * 2 + (tile & 1);
        a = {p.po_s + (slot * 128 * 32 + (int64_t)quad * 128 + row) * 4, p.ml_s + slot * 128 + row,
             (int64_t)p.pairs * 2 * 128 * 128, (int64_t)p.pairs * 2 * 128, ra.y};
      } else {
        const int64_t slot = (int64_t)ra.x + g;
        const int64_t cap = p.rows_l;
        a = {p.po_l + ((slot * 32 + quad) * cap + row) * 4, p.ml_l + slot * cap + row, cap * 128, cap,
             ra.y};
      }
    }
    if (seq > prefix) {
      const int32_t row = (i - u * p.tpt) * p.G + e;
      const int64_t slot = rc.x + unit, cap = p.rows_u;
      c = {p.po_u + ((slot * 32 + quad) * cap + row) * 4, p.ml_u + slot * cap + row, cap * 128, cap,
           rc.y};
    }
    const int32_t n = a.n + c.n;
    for (int32_t k = split; k < n; k += 4 * SPLIT) {
      float2 ml[4];
      float4 o[4];
      int have = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int32_t x = k + u * SPLIT;
        if (x < n) {
          const bool pre = x < a.n;
          const int64_t y = pre ? x : x - a.n;
          ml[u] = __ldcs((pre ? a.ml : c.ml) + y * (pre ? a.ml_step : c.ml_step));
          o[u] = __ldcs(reinterpret_cast<const float4*>((pre ? a.o : c.o) + y * (pre ? a.o_step : c.o_step)));
          ++have;
        }
      }
      join_four(j, ml, o, have);
    }
  }
  if (SPLIT > 1) {
    __shared__ float2 s_ml[SPLIT > 1 ? SPLIT : 1][kJoinRows * 32];
    __shared__ float4 s_o[SPLIT > 1 ? SPLIT : 1][kJoinRows * 32];
    s_ml[split][t] = make_float2(j.m, j.l);
    s_o[split][t] = j.acc;
    __syncthreads();
    if (split > 0) return;
    float2 ml[4];
    float4 o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = u + 1 < SPLIT ? u + 1 : 0;
      ml[u] = s_ml[x][t];
      o[u] = s_o[x][t];
    }
    join_four(j, ml, o, SPLIT - 1);
  }
  if (!valid) return;
  const float inv = j.l == 0.f ? 0.f : 1.0f / j.l;  // a row that sees no key: o = 0, lse = -inf
  const int64_t out = (int64_t)r * p.Hq + g * p.G + e;
  uint2 u;
  u.x = pack_bf16x2(j.acc.x * inv, j.acc.y * inv);
  u.y = pack_bf16x2(j.acc.z * inv, j.acc.w * inv);
  *reinterpret_cast<uint2*>(p.o + out * 128 + quad * 4) = u;
  if (quad == 0 && p.lse) p.lse[out] = j.l == 0.f ? -INFINITY : (j.m + log2f(j.l)) * kLn2;
}

struct Layout {
  int32_t rows_g, tpt, pairs, abreast, odd, units, rows_u, q_rows, rows_l;
  size_t po_s, po_l, po_u, ml_s, ml_l, ml_u, prefix, range_s, range_l, range_u, total;
};

Layout layout_of(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int ctas) {
  Layout y{};
  const int32_t G = Hq / Hkv;
  y.rows_g = B * N * G;
  y.tpt = 128 / G;
  const int32_t tiles = (y.rows_g + 127) / 128;
  y.pairs = tiles / 2;
  y.odd = tiles & 1;
  y.units = (N + y.tpt - 1) / y.tpt;
  y.rows_u = G * (N < y.tpt ? N : y.tpt);
  y.q_rows = y.rows_u <= 64 && y.rows_g - 256 * y.pairs <= 64 ? 64 : 128;
  y.rows_l = (y.rows_g - 256 * y.pairs + 7) / 8 * 8;
  // pairs that walk the prefix together, at most 16: enough that DRAM feeds them (four or more on one
  // stream of keys where there are as many), few enough that whole runs of them split the CTAs
  // evenly, and without idle places in the last round (9, 11 or 13 pairs all walk together)
  y.abreast = 1;
  float best = 1e30f;
  for (int32_t n = 1; n <= 16 && n <= y.pairs; ++n) {
    const float rounds = (float)((y.pairs + n - 1) / n) * n / y.pairs;
    const float cost = rounds * (1.f + 0.5f * n / ctas) + (n < 4 && n < y.pairs ? 0.3f * (4 - n) : 0.f);
    if (cost < best) {
      best = cost;
      y.abreast = n;
    }
  }
  // a worker's segments of one kind have distinct worker + tile (or worker + group) sums
  const size_t n_s = y.pairs ? ((size_t)ctas / y.abreast + Hkv) * y.pairs : 0;
  const size_t n_l = y.odd ? (size_t)2 * ctas + Hkv : 0;
  const size_t n_u = (size_t)2 * ctas + (size_t)B * y.units * Hkv;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  y.prefix = take(sizeof(int32_t));
  y.range_s = take((size_t)Hkv * y.pairs * sizeof(int2));
  y.range_l = take((size_t)Hkv * sizeof(int2));
  y.range_u = take((size_t)B * y.units * Hkv * sizeof(int2));
  y.ml_s = take(n_s * 256 * sizeof(float2));
  y.ml_l = take(n_l * y.rows_l * sizeof(float2));
  y.ml_u = take(n_u * y.rows_u * sizeof(float2));
  y.po_s = take(n_s * 256 * 128 * sizeof(float));
  y.po_l = take(n_l * y.rows_l * 128 * sizeof(float));
  y.po_u = take(n_u * y.rows_u * 128 * sizeof(float));
  y.total = at;
  return y;
}

struct Maps {
  CUtensorMap qt, qo, qu, km, vm;
  TailMaps vt;
};

template <bool LATE>
cudaError_t launch_kernels(const Maps& m, const KParams& p, cudaStream_t stream) {
  cudaError_t e;
  static std::atomic<int> regs{0};  // of the kernel as built: the register split counts on it
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, shared_prefix_kernel<LATE>);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  static std::atomic<size_t> raised[kMaxDevices];
  e = launch_with_smem(shared_prefix_kernel<LATE>, kSmemBytes, raised, [&] {
    return cudaLaunchKernelEx(&cfg, shared_prefix_kernel<LATE>, m.qt, m.qo, m.qu, m.km, m.vm, m.vt, p);
  });
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.Hkv * (((int64_t)p.rows_g + kJoinRows - 1) / kJoinRows)));
  cfg.dynamicSmemBytes = 0;
  const bool many = (int64_t)cfg.gridDim.x <= p.ctas;  // a CTA of 1024 threads fills an SM
  cfg.blockDim = dim3(kJoinRows * 32 * (many ? kJoinSplit : 1));
  e = many ? cudaLaunchKernelEx(&cfg, shared_prefix_join_kernel<kJoinSplit>, p)
           : cudaLaunchKernelEx(&cfg, shared_prefix_join_kernel<1>, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace

size_t shared_prefix_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int ctas) {
  return layout_of(B, N, Hq, Hkv, ctas).total;
}

cudaError_t launch_shared_prefix_decode(const SharedPrefixArgs& a, cudaStream_t stream) {
  const int ctas = sm_count();
  const Layout y = layout_of(a.B, a.N, a.Hq, a.Hkv, ctas);
  const int32_t G = a.Hq / a.Hkv;
  KParams p{};
  p.page_table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.shared_len = a.shared_len;
  p.B = a.B;
  p.N = a.N;
  p.G = G;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  while ((1 << p.gs) < G) ++p.gs;
  while ((1 << p.hs) < a.Hkv) ++p.hs;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  p.ctas = ctas;
  p.rows_g = y.rows_g;
  p.tpt = y.tpt;
  p.pairs = y.pairs;
  p.abreast = y.abreast;
  p.odd = y.odd;
  p.units = y.units;
  p.rows_u = y.rows_u;
  p.q_rows = y.q_rows;
  p.rows_l = y.rows_l;
  p.v_cache = a.v_cache;
  uint8_t* w = a.workspace;
  p.prefix = reinterpret_cast<int32_t*>(w + y.prefix);
  p.range_s = reinterpret_cast<int2*>(w + y.range_s);
  p.range_l = reinterpret_cast<int2*>(w + y.range_l);
  p.range_u = reinterpret_cast<int2*>(w + y.range_u);
  p.ml_s = reinterpret_cast<float2*>(w + y.ml_s);
  p.ml_l = reinterpret_cast<float2*>(w + y.ml_l);
  p.ml_u = reinterpret_cast<float2*>(w + y.ml_u);
  p.po_s = reinterpret_cast<float*>(w + y.po_s);
  p.po_l = reinterpret_cast<float*>(w + y.po_l);
  p.po_u = reinterpret_cast<float*>(w + y.po_u);
  p.o = a.o;
  p.lse = a.lse;
  // query rows as (channel half, head of the group, row, half, group): a box is G heads of
  // consecutive rows, one 128-byte line each
  Maps m;
  const uint64_t qd[5] = {64, (uint64_t)G, (uint64_t)a.B * a.N, 2, (uint64_t)a.Hkv};
  const uint64_t qs[4] = {256, (uint64_t)a.Hq * 256, 128, (uint64_t)G * 256};
  const uint32_t bt[5] = {64, (uint32_t)G, (uint32_t)y.tpt, 1, 1};
  const uint32_t bo[5] = {64, (uint32_t)G, (uint32_t)(y.q_rows / G), 1, 1};
  const uint32_t bu[5] = {64, (uint32_t)G, (uint32_t)(y.rows_u / G), 1, 1};
  // cache cells as (channel half, token, half, group): a box is both halves of 64 tokens
  const uint64_t kd[4] = {64, (uint64_t)a.num_pages * 128, 2, (uint64_t)a.Hkv};
  const uint64_t ks[3] = {(uint64_t)a.Hkv * 256, 128, 256};
  const uint32_t bk[4] = {64, kStep, 2, 1};
  if (!encode_bf16_map(&m.qt, a.q, 5, qd, qs, bt, true) ||
      !encode_bf16_map(&m.qo, a.q, 5, qd, qs, bo, true) ||
      !encode_bf16_map(&m.qu, a.q, 5, qd, qs, bu, true) ||
      !encode_bf16_map(&m.km, a.k_cache, 4, kd, ks, bk, true) ||
      !encode_bf16_map(&m.vm, a.v_cache, 4, kd, ks, bk, true))
    return cudaErrorInvalidValue;
  for (int b = 0; b < 6; ++b) {
    const uint32_t box[4] = {64, 1u << b, 1, 1};
    if (!encode_bf16_map(&m.vt.m[b], a.v_cache, 4, kd, ks, box, true)) return cudaErrorInvalidValue;
  }
  return a.N > 1 ? launch_kernels<true>(m, p, stream) : launch_kernels<false>(m, p, stream);
}

}  // namespace msa
