// Causal attention of a ragged batch over the paged cache: request b's new tokens (any number of them,
// its last positions) see every key of the request up to their own. One call serves prompts, chunks of
// prompts behind a cached prefix, and decode rows, mixed in one batch as a scheduler packs them.
//
// Softmax attention over a key set that is split into parts needs of each part only
//   m = max s,  l = sum 2^(s - m),  O = sum 2^(s - m) v      (s in log2 units)
// and the parts join as M = max m, o = sum 2^(m - M) O / sum 2^(m - M) l.
//
//  * Tiles. The G heads of a KV group see the same keys, so 128 / G tokens x G heads are the 128 rows of a
//    tcgen05.mma tile. Two tiles with the same keys share each K/V step that a CTA loads ("shared" units).
//    Tokens that fill one tile at most (decode rows, the rest of a chunk) give each of the CTA's two
//    lanes a KV group, or half of the keys, of its own: their MMAs run far below their rate, but a step's
//    keys take longer to arrive than the padded MMAs take.
//  * Units. A tile pair (or tile) is cut along its keys into runs of steps. A run that is its whole tile
//    writes the output itself; others leave partials that a second kernel joins in their order. The runs
//    are made from the lengths on the GPU, so a call can be captured once and replayed with other lengths,
//    in one of two ways that the host chooses by what the sizes allow (see the launch):
//      - equal runs: every CTA walks the lengths itself and takes its share of all steps, without another
//        launch. For few tiles, where the launch and the reading of a list would be most of the time;
//      - a list: a plan kernel writes units of at most two thirds of a CTA's share of what is left (kMinPiece
//        steps at least), so that the last ones to start are short, and CTAs take one after the other.
//        Which CTA takes which changes no result. Tiles need different times (causal ends, kinds), which
//        evens out this way.
//  * The order (request, group, last tiles first, pieces) lets the CTAs that run at the same time read
//    the same keys, and DRAM once (4096 tokens on 16384: 152 MB read, as many as the caches and Q hold).
//  * V cells that a row must not use (later tokens of its request, what lies behind its last token) are
//    multiplied by weights of 0, and 0 * NaN is NaN. So in steps that hold such cells two warps
//    look through V in shared memory before the MMAs: rows behind the request's end become zeros, and so
//    does what is not finite, which the softmax warps then add to the rows that see it.
//
// Per lane S = Q K^T (128 x 64 x 128) and O += P V run on tcgen05 with S, P and O in tensor memory; one
// softmax warpgroup per lane keeps the running reference and sum in fp32. P is rounded to bf16 for its
// product, as tensor cores take it beside V in bf16 (2^-8 of each weight at most); its sum l is taken
// before that rounding. A step is 64 keys because then S has two buffers per lane next to O (2 lanes x
// (2 x 64 + 128) = 512 columns): S(i+1) is ready when the softmax of step i ends. K and V come through a
// ring and a producer warp each: one warp for both needs 1.4 us a step, as long as the decode rows' step.
//
// What bounds it, Hq/Hkv/D = 64/8/128 and 1.87 PFLOP/s bf16, 6.79 TB/s measured:
//   one prompt of 16384             3.00-3.15 ms  (1.40-1.47 PFLOP/s, 75-78 % of the burst rate)
//   2048 tokens on 60032 keys       2.83-2.87 ms  (1.43-1.45 PFLOP/s)
//   64 decode rows, 4k-16k keys     0.381-0.391 ms (the copy rate: HBM)
//   64 chunks of 32-64 tokens behind 250-1000   0.117 ms; 1 row on 2048 keys 13.4 us (latency, two launches)
// Long chunks are bound by the S products. An N = 64 product reads its 128 x 16 Q operand from shared
// memory again at every instruction: 48 cycles measured where its arithmetic takes 32 (N = 128: 64 of 64; P
// from tensor memory, N = 128: 64 of 64). Without the S products 3.09 ms became 2.22, without the O products
// 2.88, without the softmax's arithmetic 2.94. Steps of 128 keys do away with that, but leave one
// S buffer per lane, so a lane's softmax and its S product take turns: 3.31 ms.
// Also slower: both lanes' issue strictly in turn (4.76 ms), the softmax in scalar instead of paired fp32.
#include <math.h>

#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "softmax_math.cuh"

MSA_DEFINE_ERROR_WORD(chunk)

namespace msa {

namespace {

constexpr int kThreads = 512;                    // warpgroups: loads, softmax x 2, MMA issue
constexpr int kLaunchRegs = 128;                 // registers per thread at launch, then split
constexpr int kRegsLoad = 56, kRegsIssue = 56, kRegsSoftmax = 200;
static_assert(128 * (kRegsLoad + kRegsIssue) + 256 * kRegsSoftmax == kThreads * kLaunchRegs, "register split");
constexpr int kStep = 64;                        // keys per step
constexpr uint32_t kQHalf = 128 * 128;           // 128 rows x 64 channels bf16
constexpr uint32_t kQTile = 2 * kQHalf;
constexpr uint32_t kKvHalf = kStep * 128;        // 64 keys x 64 channels bf16
constexpr uint32_t kKvTile = 2 * kKvHalf;        // K or V of one step: 16 KB, one slot of the ring
constexpr int kSlots = 5;                        // of K, and of V
constexpr uint32_t kOffK = 2 * kQTile, kOffV = kOffK + kSlots * kKvTile;
constexpr uint32_t kOffBar = kOffV + kSlots * kKvTile;
constexpr uint32_t kTmemCols = 512;              // S buffers of lane X at 128 X, O at 256 + 128 X
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFarSum = 16384.f;  // of a step's P: beyond it the softmax's reference moves
// s log2(e) - m in one fma is off by what m was rounded by, the same for all keys of a row: a common
// factor of P and l. Beyond this magnitude of m it would leave fp32's range, and m is subtracted first.
constexpr float kFarRef = 16777216.f;
constexpr int kMinPiece = 16;       // steps of a piece, where the whole call has as many per CTA
// Of the cut into equal runs: relative time of a step of a shared unit and of lanes with keys of their own
// (which HBM feeds at the copy rate when all CTAs have such), and what a tile's end and beginning take.
constexpr int32_t kSharedCost = 4, kOwnCost = 7, kTileCost = 7;
constexpr int32_t kLeastRun = 2 * kOwnCost;
constexpr uint32_t kMostCost = 2147483647;  // of a call

// What the two lanes of a unit have.
enum : int32_t {
  kHeads = 0,   // a tile of a KV group each, on the same keys
  kShared = 1,  // neighbouring tiles of one group: they share the steps
  kHalves = 2,  // one tile, of a single KV group: lane 1 takes its later keys and hands lane 0 its part
};
// What a CTA does next: for each lane a tile and a run of steps.
struct __align__(16) Unit {
  int32_t n[2];     // steps; 0: nothing for the lane. Both 0: there are no more units.
  int32_t key0[2];  // first keys
  int32_t g[2];     // groups
  int32_t part;     // first row of the partials, lane 1's tile_rows behind lane 0's; -1: whole tiles
  int32_t kind;
  int32_t b;        // page-table row
  int32_t row;      // first token row of the (first) tile
  int32_t tokens;   // of the tile, or of both
  int32_t pos;      // position of the first token
  int32_t seq;      // keys that the request holds
  int32_t pad[3];
};
static_assert(sizeof(Unit) == 64, "four 16-byte loads");
// A tile whose pieces are to be joined.
struct __align__(16) JoinTile {
  int32_t row, rows, g;  // first token row, valid rows, group
  int32_t first, rest;   // first rows of the first and the second piece's partial; then 2 * tile_rows further each
  int32_t pieces, cap;   // cap: rows of a partial, a multiple of 8
  int32_t pad;
};
struct Header {
  int32_t units, joins, ticket;
};

struct KParams {
  const int32_t* page_table;
  const int32_t* seq_lens;
  const int32_t* cu_tokens;
  int32_t B, T, G, Hq, Hkv, max_blocks;
  int64_t num_pages;
  int32_t gs;         // log2 of G
  int32_t tpt;        // tokens per tile: 128 / G
  int32_t ctas;
  int32_t cap_units, cap_joins;
  int32_t cap_pieces;  // of 2 * tile_rows rows
  int32_t tile_rows;   // rows of a tile's partial: 128, or as many as all new tokens fill
  Header* head;
  Unit* units;
  JoinTile* joins;
  float* po;          // partials: O as [32 channel quads][cap rows][4] fp32 from row * 128 on
  float2* ml;         // (m, l) per row
  float* half_po;     // kHalves: lane 1's part, per CTA
  const uint16_t* v_cache;
  uint16_t* o;
  float* lse;
};

// ------------------------------------------------------------------------------ plan
constexpr int kPlanThreads = 1024;

struct Request {
  int32_t t0, n, seq;  // first token row, new tokens, keys held
};
__device__ __forceinline__ Request request_of(const KParams& p, int b, bool& bad) {
  Request r;
  const int32_t c0 = p.cu_tokens[b], c1 = p.cu_tokens[b + 1], s = p.seq_lens[b];
  r.t0 = min(max(c0, 0), p.T);
  r.n = max(min(c1, p.T) - r.t0, 0);
  const int32_t hi = p.max_blocks * MSA_BLOCK_TOKENS;
  r.seq = min(max(s, 0), hi);
  bad = c0 < 0 || c1 > p.T || c1 < c0 || s < r.n || s > hi;
  return r;
}
// Items of a request: its pairs of tiles x groups, then a last single tile's lane pairs.
struct Shape {
  int32_t np, single, ps, items;
};
__device__ __forceinline__ Shape shape_of(const KParams& p, int32_t n) {
  Shape s;
  const int32_t w = 2 * p.tpt;
  s.np = (n + w - 1) / w;
  s.single = n > 0 && n - (s.np - 1) * w <= p.tpt;
  s.ps = s.np - s.single;
  s.items = s.ps * p.Hkv + (s.single ? max(1, p.Hkv / 2) : 0);
  return s;
}
struct Item {
  int32_t b, row, tokens, pos, seq, g, kind;
  int32_t steps, cost;  // cost: steps of the CTA
  __device__ __forceinline__ int32_t tiles() const { return kind == kHalves ? 1 : 2; }
  __device__ __forceinline__ int32_t cap(const KParams& p) const {
    return kind == kShared ? 128 : ((tokens << p.gs) + 7) / 8 * 8;
  }
};
__device__ __forceinline__ Item item_of(const KParams& p, int b, const Request& r, const Shape& s, int32_t i) {
  Item t;
  const int32_t w = 2 * p.tpt;
  t.b = b;
  t.seq = r.seq;
  int32_t j = s.np - 1;
  t.kind = i < s.ps * p.Hkv ? kShared : (p.Hkv > 1 ? kHeads : kHalves);
  if (t.kind == kShared) {
    t.g = i / s.ps;
    j = s.ps - 1 - (i - t.g * s.ps);
  } else {
    t.g = 2 * (i - s.ps * p.Hkv);
  }
  t.row = r.t0 + j * w;
  t.tokens = min(w, r.n - j * w);
  t.pos = r.seq - r.n + j * w;
  t.steps = max(1, (t.pos + t.tokens + kStep - 1) / kStep);
  t.cost = t.kind == kHalves ? (t.steps + 1) / 2 : t.steps;
  return t;
}
// Steps [s0, s1) of an item's cost; its partials go to rows `part` on.
__device__ __forceinline__ Unit unit_of(const Item& t, int32_t s0, int32_t s1, int32_t part) {
  Unit u{};
  u.n[0] = s1 - s0;
  u.key0[0] = s0 * kStep;
  u.g[0] = u.g[1] = t.g;
  if (t.kind == kHalves) {
    u.key0[1] = (t.cost + s0) * kStep;
    u.n[1] = max(0, min(t.steps, t.cost + s1) - (t.cost + s0));
  } else {
    u.key0[1] = u.key0[0];
    u.n[1] = u.n[0];
    u.g[1] += t.kind == kHeads;
  }
  u.part = part;
  u.kind = t.kind;
  u.b = t.b;
  u.row = t.row;
  u.tokens = t.tokens;
  u.pos = t.pos;
  u.seq = t.seq;
  return u;
}
// Tile X of an item for the join; `valid`: whether there is anything to join.
__device__ __forceinline__ JoinTile join_of(const KParams& p, const Item& t, int32_t X, bool valid, int32_t first,
                                            int32_t rest, int32_t pieces) {
  JoinTile j{};
  const int32_t tile = t.kind == kShared ? X * p.tpt : 0;
  j.row = t.row + tile;
  j.rows = valid && X < t.tiles() ? min(p.tpt, t.tokens - tile) << p.gs : 0;
  j.g = t.kind == kHeads ? t.g + X : t.g;
  j.first = first + X * p.tile_rows;
  j.rest = rest + X * p.tile_rows;
  j.pieces = pieces;
  j.cap = t.cap(p);
  return j;
}
__device__ __forceinline__ void store_join(JoinTile* to, const JoinTile& j) {
  reinterpret_cast<int4*>(to)[0] = make_int4(j.row, j.rows, j.g, j.first);
  reinterpret_cast<int4*>(to)[1] = make_int4(j.rest, j.pieces, j.cap, 0);
}

// The cut into equal runs counts in units of time.
__device__ __forceinline__ int32_t step_cost(int32_t kind) { return kind == kShared ? kSharedCost : kOwnCost; }
__device__ __forceinline__ int32_t run_cost(const Item& t) { return t.cost * step_cost(t.kind) + kTileCost; }
// ... of all pairs of one group of a request, and of the whole request.
__device__ __forceinline__ int32_t pairs_cost(const KParams& p, const Request& r, const Shape& s) {
  int32_t sum = 0;
#pragma unroll 1
  for (int32_t j = 0; j < s.ps; ++j) sum += run_cost(item_of(p, 0, r, s, j));
  return sum;
}
__device__ __forceinline__ int32_t request_cost(const KParams& p, const Request& r) {
  const Shape s = shape_of(p, r.n);
  int32_t sum = p.Hkv * pairs_cost(p, r, s);
  if (s.single) sum += run_cost(item_of(p, 0, r, s, p.Hkv * s.ps)) * max(1, p.Hkv / 2);
  return sum;
}

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  return x;
}
// Exclusive scan over the CTA; total of all threads.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t incl = warp_scan(x, lane);
  __syncthreads();  // sums is free
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  if (warp == 0) sums[lane] = warp_scan(sums[lane], lane);
  __syncthreads();
  total = sums[31];
  return incl - x + (warp > 0 ? sums[warp - 1] : 0);
}
static_assert(kPlanThreads == 1024, "block_scan: 32 warps");

// Pieces of an item at which `left` steps of the whole call, its own among them, are still to come:
// two thirds of a CTA's share of them each, so that the CTAs end together. (kMinPiece 8 and half of the share
// left 3.5 partials per row of 2048 tokens on 60032 and took 1 % longer there, 64 chunks of 64 tokens 145 instead of
// 117 us; the whole share 2 % longer.)
__device__ __forceinline__ int32_t pieces_of(const KParams& p, int32_t cost, int64_t left, int32_t least) {
  const int32_t most = (int32_t)max((int64_t)least, (2 * left + 3 * p.ctas - 1) / (3 * p.ctas));
  return (cost + most - 1) / most;
}

__global__ void __launch_bounds__(kPlanThreads) chunk_plan_kernel(const __grid_constant__ KParams p) {
  extern __shared__ int32_t first_item[];  // [B + 1]
  __shared__ int64_t sums[32];
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the requests' items
  int64_t items = 0;
  bool any_bad = false;
  for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    int32_t n = 0;
    if (b < p.B) {
      bool bad;
      const Request r = request_of(p, b, bad);
      any_bad |= bad;
      n = shape_of(p, r.n).items;
    }
    int64_t total;
    const int64_t at = items + block_scan(n, sums, total);
    if (b < p.B) first_item[b] = (int32_t)min(at, kMaxChunkItems);
    items += total;
  }
  if (items > kMaxChunkItems) {  // token ranges that overlap: not seen with lengths that add up
    items = kMaxChunkItems;
    any_bad = true;
  }
  if (tid == 0) first_item[p.B] = (int32_t)items;
  if (any_bad) msa_record_error(kErrBadBlock);
  __syncthreads();
  // a thread has a run of items
  const int32_t per = (int32_t)((items + kPlanThreads - 1) / kPlanThreads);
  const int32_t i0 = (int32_t)min(items, (int64_t)tid * per), i1 = (int32_t)min(items, (int64_t)i0 + per);
  int32_t b_first = 0;
  if (i0 < i1) {
    int32_t lo = 0, hi = p.B;  // first_item[lo] <= i0 < first_item[hi]
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) / 2;
      if (first_item[mid] <= i0) lo = mid;
      else hi = mid;
    }
    b_first = lo;
  }
  auto each = [&](auto&& f) {
    int32_t b = b_first, i = i0;
    while (i < i1) {
      while (first_item[b + 1] <= i) ++b;
      bool bad;
      const Request r = request_of(p, b, bad);
      const Shape s = shape_of(p, r.n);
      const int32_t end = min(i1, first_item[b + 1]);
      for (; i < end; ++i) f(item_of(p, b, r, s, i - first_item[b]));
    }
  };
  int64_t cost = 0, all;
  each([&](const Item& t) { cost += t.cost; });
  const int64_t before = block_scan(cost, sums, all);
  const int32_t least = (int32_t)min((int64_t)kMinPiece, max((int64_t)2, (all + p.ctas - 1) / p.ctas));
  // units and, of these, pieces of items that are cut, and cut items
  int64_t left = all - before;
  int32_t n_units = 0, n_cut = 0, n_pieces = 0;
  each([&](const Item& t) {
    const int32_t pieces = pieces_of(p, t.cost, left, least);
    n_units += pieces;
    n_cut += pieces > 1;
    n_pieces += pieces > 1 ? pieces : 0;
    left -= t.cost;
  });
  int64_t total_units, total_cut;  // two counts of 32 bits in one scan
  int64_t at_unit = block_scan(n_units, sums, total_units);
  const int64_t at = block_scan((int64_t)n_cut << 32 | n_pieces, sums, total_cut);
  int32_t at_cut = (int32_t)(at >> 32), at_piece = (int32_t)at;
  const bool over = total_units > p.cap_units || (total_cut >> 32) * 2 > p.cap_joins || (int32_t)total_cut > p.cap_pieces;
  if (tid == 0) {
    p.head->units = (int32_t)min(total_units, (int64_t)p.cap_units);
    p.head->joins = (int32_t)min((total_cut >> 32) * 2, (int64_t)p.cap_joins);
    p.head->ticket = p.ctas;  // the first units are the CTAs' own numbers
    if (over) msa_record_error(kErrBadBlock);  // not seen with lengths that add up: the workspace is sized for those
  }
  left = all - before;
  each([&](const Item& t) {
    const int32_t pieces = pieces_of(p, t.cost, left, least);
    const bool cut = pieces > 1, fits = !cut || at_piece + pieces <= p.cap_pieces;
    for (int32_t k = 0; k < pieces && at_unit + k < p.cap_units; ++k) {
      Unit u = unit_of(t, (int32_t)((int64_t)t.cost * k / pieces), (int32_t)((int64_t)t.cost * (k + 1) / pieces),
                       cut ? (at_piece + k) * 2 * p.tile_rows : -1);
      if (!fits) u.tokens = 0;  // nowhere to go
      const int4* src = reinterpret_cast<const int4*>(&u);
      int4* dst = reinterpret_cast<int4*>(p.units + at_unit + k);
#pragma unroll
      for (int x = 0; x < 4; ++x) dst[x] = src[x];
    }
    if (cut) {
      for (int32_t X = 0; X < 2 && 2 * at_cut + X < p.cap_joins; ++X)
        store_join(p.joins + 2 * at_cut + X, join_of(p, t, X, fits, at_piece * 2 * p.tile_rows,
                                                     (at_piece + 1) * 2 * p.tile_rows, pieces));
      ++at_cut;
      at_piece += pieces;
    }
    at_unit += pieces;
    left -= t.cost;
  });
}

// ------------------------------------------------------------------------------ attention
// Rows of V [y, 64) of a slot that some row of the tiles must not use; from z on they lie behind the
// request's end. slot < 0: no more. Each open entry has a slot of its own.
struct Late {
  int32_t y, z, slot, lanes;  // lanes: bit X: lane X reads it
};
constexpr int kLate = 16;
static_assert(kLate > kSlots + 1, "an entry is not overwritten while it is open");
constexpr int kQueue = 4;  // units that the feeder is ahead of the slowest reader at most

struct Bars {
  uint64_t kv_full[2][kSlots], kv_empty[2][kSlots];  // K, V
  uint64_t q_full[2][2], q_empty[2][2];  // [lane][the lane's tile & 1]
  uint64_t s_full[2][2], p_full[2][2], o_full[2][2];  // [lane][the lane's step & 1]
  uint64_t o_free[2];
  uint64_t unit_full[kQueue], unit_free[kQueue];
  uint64_t want;  // the producer nears the end of a unit
  uint64_t late_full[kLate];
  uint64_t drained[2];
  uint64_t half_full, half_free;  // kHalves: lane 1's part is there, is read
  float2 half_ml[128];
  Unit unit[kQueue];
  Late late[kLate];
  int32_t odd[2];  // what is not finite was taken out of V, in this unit of the lane or one before
  uint32_t tmem_base;
  int32_t fail;
  // cut into equal runs
  int32_t w_sum[kThreads / 32], start_b, start_off, total, workers;
};
constexpr size_t kSmemBytes = kOffBar + ((sizeof(Bars) + 15) / 16) * 16;
static_assert(kSmemBytes <= 232448, "shared memory of one CTA");

struct RingPos {
  int32_t slot;
  uint32_t phase;  // parity of the slot's current use
  __device__ __forceinline__ void advance(int32_t n) {
    slot += n;
    if (slot >= kSlots) {
      slot -= kSlots;
      phase ^= 1u;
    }
  }
  __device__ __forceinline__ RingPos after(int32_t n) const {
    RingPos r = *this;
    r.advance(n);
    return r;
  }
};

// Bounded wait of a converged warp; every thread gets the same answer. The flag that another role's
// timeout sets is read only while the phase is open.
__device__ __forceinline__ bool wait_or_fail(uint64_t* bar, uint32_t parity, volatile int32_t* fail) {
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *fail != 0)) return false;
  }
  msa_record_error(kErrTimeout);
  *fail = 1;
  return false;
}
// wait_or_fail for several barriers at once: each thread tests one (a completed wait takes 125 cycles).
__device__ __forceinline__ bool wait_all_or_fail(uint64_t* mine, uint32_t par, volatile int32_t* fail) {
  const uint32_t bar = smem_u32(mine);
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait_addr(bar, par))) return true;
    if (__any_sync(0xffffffffu, *fail != 0)) return false;
  }
  msa_record_error(kErrTimeout);
  *fail = 1;
  return false;
}
// A value that is the same in all threads of a converged warp, in a form that lets the compiler see
// it: operands of tensor-core and bulk-copy instructions that it cannot prove uniform cost a loop
// over the threads each.
__device__ __forceinline__ int32_t uniform(int32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Half of S = Q K^T: the four K-16 products of one channel half of 128-byte-swizzled tiles, issued
// by one elected lane of the converged warp.
__device__ __forceinline__ void issue_s(uint32_t d, uint64_t qd, uint64_t kd, uint32_t idesc, uint32_t accumulate) {
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
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// SELF: the CTAs cut the whole call into equal runs of steps among them, each for itself from the lengths;
// else they take the units that the plan kernel listed.
template <bool SELF>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_attention_kernel(const __grid_constant__ CUtensorMap qmap_t, const __grid_constant__ CUtensorMap qmap_h,
                           const __grid_constant__ CUtensorMap qmap_1,
                           const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                           const __grid_constant__ KParams p) {
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
    for (int i = 0; i < kSlots; ++i)
      for (int x = 0; x < 2; ++x) {
        mbar_init(&B.kv_full[x][i], 2);   // the producer twice, or the two late-row warps
        mbar_init(&B.kv_empty[x][i], 2);  // both issuers
      }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&B.o_free[x], 4);
      mbar_init(&B.drained[x], 1);
      for (int i = 0; i < 2; ++i) {
        mbar_init(&B.q_full[x][i], 1);
        mbar_init(&B.q_empty[x][i], 1);
        mbar_init(&B.s_full[x][i], 1);
        mbar_init(&B.o_full[x][i], 1);
        mbar_init(&B.p_full[x][i], 4);
      }
    }
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(&B.unit_full[i], 1);
      mbar_init(&B.unit_free[i], 13);  // readers: eight softmax warps, two issuers, the K, V and query loaders
    }
    for (int i = 0; i < kLate; ++i) mbar_init(&B.late_full[i], 1);
    mbar_init(&B.want, 1);
    mbar_init(&B.half_full, 4);
    mbar_init(&B.half_free, 4);
    B.fail = 0;
    B.odd[0] = B.odd[1] = 0;
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
    tma_prefetch_desc(&qmap_h);
    tma_prefetch_desc(&qmap_1);
  }
  tmem_fence_before();
  __syncthreads();
  tmem_fence_after();
  const uint32_t tmem = uniform((int32_t)B.tmem_base);
  const uint32_t sbase = smem_u32(smem);
  // The plan ends here, and with it what precedes it in the stream. The join may be scheduled as CTAs of
  // this kernel leave; it waits for all of their stores.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (SELF) {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
    // The layout holds the sums of token ranges in order below kMostCost. Ranges that overlap can pass it by far:
    // the sums stop there, and such a call has no work.
    uint32_t sum = 0;
    bool any_bad = false;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      bool bad;
      sum = min(sum + (uint32_t)request_cost(p, request_of(p, b, bad)), kMostCost);
      any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0) msa_record_error(kErrBadBlock);
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl = min(incl + y, kMostCost);
    }
    if (lane == 31) B.w_sum[warp] = (int32_t)incl;
    if (tid == 0) B.start_b = p.B;
    __syncthreads();
    uint32_t at = incl - sum;
    uint64_t all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      const uint32_t x = (uint32_t)B.w_sum[w];
      if (w < warp) at += x;  // means nothing where `all` is over
      all += x;
    }
    const int32_t total = all < kMostCost ? (int32_t)all : 0, before = (int32_t)at;
    const int32_t workers = max(1, min((int32_t)gridDim.x, total / kLeastRun));
    const int32_t x0 = (int32_t)((int64_t)total * min((int32_t)blockIdx.x, workers) / workers);
    if (total > 0 && before <= x0 && x0 - before < (int32_t)sum) {  // this CTA starts in one of the thread's requests
      int32_t off = x0 - before;
      int b = b0;
#pragma unroll 1
      for (; b < b1; ++b) {
        bool bad;
        const int32_t c = request_cost(p, request_of(p, b, bad));
        if (off < c) break;
        off -= c;
      }
      B.start_b = b;
      B.start_off = off;
    }
    if (tid == 0) {
      B.total = total;
      B.workers = workers;
    }
    __syncthreads();
  }
  // Tiles of at most 64 rows (a wider group's token of 128 rows is none).
  auto is_small = [&](const Unit& u) { return u.kind != kShared && u.tokens << p.gs <= 64; };
  // The k-th unit for one of its readers.
  auto take = [&](int32_t& k, Unit& u) {
    const int q = k & (kQueue - 1);
    if (!wait_or_fail(&B.unit_full[q], (k / kQueue) & 1, fail)) return false;
    const Unit& e = B.unit[q];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      u.n[x] = uniform(e.n[x]);
      u.key0[x] = uniform(e.key0[x]);
      u.g[x] = uniform(e.g[x]);
    }
    u.part = uniform(e.part);
    u.kind = uniform(e.kind);
    u.b = uniform(e.b);
    u.row = uniform(e.row);
    u.tokens = uniform(e.tokens);
    u.pos = uniform(e.pos);
    u.seq = uniform(e.seq);
    __syncwarp();
    mbar_arrive_if(&B.unit_free[q], lane == 0);
    ++k;
    return true;
  };
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == 0 || warp == 3) {
      // ============================================================== K, V
      // Warp 0 loads the units' keys and warp 3 their values, a unit's steps behind the other's; a slot takes
      // a producer some 700 cycles, so one for both was what bounded the kernel. A step of lanes with keys of
      // their own has a slot for each.
      const int V = warp == 3;
      const CUtensorMap* map = V ? &vmap : &kmap;
      uint8_t* ring = smem + (V ? kOffV : kOffK);
      RingPos r{0, 0};
      int32_t used = 0;     // slots begun
      int32_t late_n = 0;   // late entries
      // One slot: 64 rows from token row tok on. y, z: V's late rows and its end; lanes that read it.
      auto slot = [&](int32_t tok, int32_t g, int32_t y, int32_t z, int32_t lanes) {
        if (used >= kSlots && !wait_or_fail(&B.kv_empty[V][r.slot], r.phase ^ 1u, fail)) return false;
        const int32_t ut = uniform(tok), ug = uniform(g), us = uniform(r.slot);
        const bool late = V && y < kStep;
        if (lane == 0) {
          uint64_t* full = &B.kv_full[V][us];
          if (late) {
            const int32_t q = late_n & (kLate - 1);
            B.late[q] = {y, z, us, lanes};
            full = &B.late_full[q];
          } else {
            mbar_arrive(full);
          }
          mbar_expect_tx(full, kKvTile);
          tma_load_4d(ring + us * kKvTile, map, full, 0, ut, 0, ug);
        }
        __syncwarp();
        if (late) ++late_n;
        ++used;
        r.advance(1);
        return true;
      };
      int32_t k = 0, page[2] = {0, 0};
      // the pages of 32 steps from j on of a lane's run, one per thread
      auto look_up = [&](const Unit& u, int x, int32_t j) {
        const int32_t jj = j + lane, key = u.key0[x] + jj * kStep;
        const bool has = jj < u.n[x] && key < u.seq;
        int32_t at = has ? p.page_table[(int64_t)u.b * p.max_blocks + key / MSA_BLOCK_TOKENS] : 0;
        const bool bad = at < 0 || at >= p.num_pages;
        if (bad) at = 0;
        if (__any_sync(0xffffffffu, bad) && lane == 0) msa_record_error(kErrBadPage);
        return at;
      };
      Unit u;
      bool good = true;
#pragma unroll 1
      while (good && (good = take(k, u)) && u.n[0] > 0) {
        const int32_t steps = u.n[0];
#pragma unroll 1
        for (int32_t j = 0; j < steps; ++j) {
          if ((j & 31) == 0) {
            page[0] = look_up(u, 0, j);
            page[1] = u.kind == kHalves ? look_up(u, 1, j) : page[0];
          }
          auto one = [&](int x, int32_t lanes) {
            const int32_t key = u.key0[x] + j * kStep;
            const int32_t tok = __shfl_sync(0xffffffffu, page[x], j & 31) * MSA_BLOCK_TOKENS + key % MSA_BLOCK_TOKENS;
            return slot(tok, u.g[x], max(0, u.pos + 1 - key), max(0, min(u.seq - key, kStep)), lanes);
          };
          if (u.kind == kShared) good = one(0, 3);
          else good = one(0, 1) && (j >= u.n[1] || one(1, 2));
          if (!good) break;
          if (!SELF && !V) mbar_arrive_if(&B.want, lane == 0 && j == max(0, steps - 6));
        }
      }
      if (V && good && lane == 0) {  // the late-row warps' end
        B.late[late_n & (kLate - 1)] = {0, 0, -1, 0};
        mbar_arrive(&B.late_full[late_n & (kLate - 1)]);
      }
      if (!good) {  // let the copies in flight land before the CTA leaves
        for (int32_t q = max(0, used - kSlots); q < used; ++q)
          for (int x = 0; x < 1000 && !mbar_try_wait_hint(&B.kv_full[V][q % kSlots], (q / kSlots) & 1, 1000); ++x) {
          }
        for (int32_t q = max(0, late_n - kLate); q < late_n; ++q)
          for (int x = 0; x < 1000 && !mbar_try_wait_hint(&B.late_full[q % kLate], (q / kLate) & 1, 1000); ++x) {
          }
      }
    } else if (warp == 2) {
      // ============================================================== units
      int32_t ticket = blockIdx.x, total = 0;
      int32_t w_b = 0, w_i = 0, w_off = 0, w_left = 0;  // SELF: request, item, offset in it, what is left of the run
      Request w_q{};
      Shape w_h{};
      bool joins = false;
      if (SELF) {
        const int32_t c = blockIdx.x, W = B.workers;
        if (c < W) w_left = (int32_t)((int64_t)B.total * (c + 1) / W) - (int32_t)((int64_t)B.total * c / W);
        if (B.start_b >= p.B) w_left = 0;
        if (w_left > 0) {
          w_b = B.start_b;
          w_off = B.start_off;
          bool bad;
          w_q = request_of(p, w_b, bad);
          w_h = shape_of(p, w_q.n);
          if (w_h.ps > 0) {
            const int32_t group = pairs_cost(p, w_q, w_h), g = min(p.Hkv, w_off / group);
            w_off -= g * group;
            w_i = g * w_h.ps;
          }
#pragma unroll 1
          for (; w_i < w_h.items; ++w_i) {
            const int32_t cost = run_cost(item_of(p, w_b, w_q, w_h, w_i));
            if (w_off < cost) break;
            w_off -= cost;
          }
        }
      } else {
        total = p.head->units;
      }
      auto next_unit = [&]() {
        Unit u{};
        if constexpr (!SELF) {
          if (ticket < total) {
            const int4* src = reinterpret_cast<const int4*>(p.units + ticket);
            int4* dst = reinterpret_cast<int4*>(&u);
#pragma unroll
            for (int x = 0; x < 4; ++x) dst[x] = src[x];
            int32_t t = 0;
            if (lane == 0) t = atomicAdd(&p.head->ticket, 1);
            ticket = __shfl_sync(0xffffffffu, t, 0);
          }
          return u;
        } else {
#pragma unroll 1
          while (w_left > 0 && w_b < p.B) {
            if (w_i >= w_h.items) {
              w_i = 0;
              if (++w_b < p.B) {
                bool bad;
                w_q = request_of(p, w_b, bad);
                w_h = shape_of(p, w_q.n);
              }
              continue;
            }
            const Item t = item_of(p, w_b, w_q, w_h, w_i);
            const int32_t a0 = w_off, cost = run_cost(t), a1 = min(cost, a0 + w_left), per = step_cost(t.kind);
            const int32_t s0 = min(t.cost, (a0 + per - 1) / per), s1 = min(t.cost, (a1 + per - 1) / per);
            const int32_t c = blockIdx.x, C = gridDim.x, row = 2 * p.tile_rows;
            w_left -= a1 - a0;
            w_off = a1;
            if (a1 == cost) {
              ++w_i;
              w_off = 0;
            }
            if (s0 >= s1) continue;
            // a run has at most one piece that ends an item that it did not begin, and one that begins an item
            // without ending it
            if (s0 == 0 && s1 == t.cost) {
              u = unit_of(t, s0, s1, -1);
            } else {
              u = unit_of(t, s0, s1, (s0 == 0 ? C + c : c) * row);
              if (s0 > 0 && s1 == t.cost) {
                // the CTA in whose run the item begins
                const int64_t W = B.workers, all = B.total, begin = all * (c + 1) / W - w_left - a1;
                int32_t c0 = max(0, min((int32_t)(begin * W / all), c));
                while (c0 > 0 && all * c0 / W > begin) --c0;
                while (c0 < c && all * (c0 + 1) / W <= begin) ++c0;
                if (lane < 2)
                  store_join(p.joins + 2 * c + lane, join_of(p, t, lane, true, (C + c0) * row, (c0 + 1) * row, c - c0 + 1));
                joins = true;
              }
            }
            break;
          }
          return u;
        }
      };
      bool good = true;
#pragma unroll 1
      for (int32_t k = 0; good; ++k) {
        // a listed unit is taken no earlier than needed, so that it goes to the CTA that is free first
        if (!SELF && k > 0 && !(good = wait_or_fail(&B.want, (k - 1) & 1, fail))) break;
        const Unit u = next_unit();
        const int q = k & (kQueue - 1);
        if (k >= kQueue && !(good = wait_or_fail(&B.unit_free[q], (k / kQueue - 1) & 1, fail))) break;
        if (lane == 0) {
          B.unit[q] = u;
          mbar_arrive(&B.unit_full[q]);
        }
        __syncwarp();
        if (u.n[0] == 0) break;  // the end of the list
      }
      if (SELF && lane < 2 && !joins) store_join(p.joins + 2 * blockIdx.x + lane, JoinTile{});
    } else if (warp == 1) {
      // ============================================================== query tiles
      // Tiles of at most 64 rows alternate between the halves of the lane's area, so that the next one's rows
      // are there before the current one's last S.
      int32_t k = 0, done[2] = {0, 0};
      bool alone[2] = {true, true};  // the lane's last tile fills the area
      Unit u;
      bool good = true;
#pragma unroll 1
      while (good && take(k, u) && (u.n[0] | u.n[1]) != 0) {
        const bool small = is_small(u);
#pragma unroll
        for (int X = 0; X < 2; ++X) {
          if (u.n[X] == 0) continue;
          // the tile whose S must have completed before this one's rows may be overwritten
          const int32_t after = done[X] - (small && !alone[X] ? 2 : 1);
          if (after >= 0 && !(good = wait_or_fail(&B.q_empty[X][after & 1], (after >> 1) & 1, fail))) break;
          if (lane == 0) {
            // one token's rows for a decode row: the others of the tile may hold anything
            const bool single = u.tokens == 1;
            const CUtensorMap* map = single ? &qmap_1 : (small ? &qmap_h : &qmap_t);
            uint64_t* full = &B.q_full[X][done[X] & 1];
            uint8_t* dst = smem + X * kQTile + (small ? (done[X] & 1) * (kQHalf / 2) : 0);
            const int32_t row = u.row + (u.kind == kShared ? X * p.tpt : 0);
            mbar_expect_tx(full, (single ? p.G : (small ? 64 : 128)) * 256);
            tma_load_5d(dst, map, full, 0, 0, row, 0, u.g[X]);
            tma_load_5d(dst + kQHalf, map, full, 0, 0, row, 1, u.g[X]);
          }
          __syncwarp();
          ++done[X];
          alone[X] = !small;
        }
      }
      if (!good || *fail)  // let the copies in flight land before the CTA leaves
        for (int X = 0; X < 2; ++X)
          for (int32_t q = max(0, done[X] - 2); q < done[X]; ++q)
            for (int x = 0; x < 1000 && !mbar_try_wait_hint(&B.q_full[X][q & 1], (q >> 1) & 1, 1000); ++x) {
            }
    }
    __syncwarp();
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp < 14) {
      // ================================================================ MMA issuers, one per lane
      // For each step i of the CTA: O(i - 2), S(i). O needs P and V; S(i) needs K(i) and overwrites the
      // tensor memory from which O(i - 2) reads P, which it may as the tensor pipe runs one thread's MMAs
      // in issue order. The warp runs in lockstep, an elected lane issues. Either issuer waits for every
      // slot and gives it back, the other lane's too: a slot's users change with the units, and a barrier's
      // parity tells a use from the one before it only to a warp that has seen that one.
      const int X = warp - 12;
      const uint32_t s_tmem = tmem + X * 128, o_tmem = tmem + 256 + X * 128;
      const uint32_t idesc_s = umma_idesc_bf16(128, kStep, 0, 0);
      const uint32_t idesc_o = umma_idesc_bf16(128, 128, 0, 1);
      const uint64_t qd0 = umma_desc_sw128(sbase + X * kQTile, 16, 1024);
      uint64_t qd = qd0;
      const uint64_t kd0 = umma_desc_sw128(sbase + kOffK, 16, 1024);
      const uint64_t vd0 = umma_desc_sw128(sbase + kOffV, kKvHalf, 1024);
      constexpr uint32_t kMine = 1, kTwo = 2, kOpens = 4, kAny = 8;  // of a step
      uint32_t d1 = 0, d2 = 0;
      Unit u;
      u.n[0] = u.n[1] = u.kind = 0;
      int32_t k = 0, j = 0, steps = 0, n_s = 0, n_o = 0, opened = 0, tiles = 0;
      RingPos rk{0, 0}, rv{0, 0};
      bool good = true, more = true;
#pragma unroll 1
      while (more || d1 || d2) {
        if (d2) {  // O of the step before the last
          const bool mine = d2 & kMine, two = d2 & kTwo;
          const RingPos at = two && X ? rv.after(1) : rv, other = two ? (X ? rv : rv.after(1)) : at;
          const uint32_t buf = n_o & 1;
          if (mine && (d2 & kOpens) && opened++ > 0 && !(good = wait_or_fail(&B.o_free[X], opened & 1, fail))) break;
          // own V, the other lane's, P
          const int w = lane & 3;
          if (!(good = wait_all_or_fail(w == 0 && mine ? &B.p_full[X][buf] : &B.kv_full[1][w == 1 ? other.slot : at.slot],
                                        w == 0 && mine ? (n_o >> 1) & 1 : (w == 1 ? other.phase : at.phase), fail)))
            break;
          const int32_t us = uniform(at.slot);
          if (mine) {
            tmem_fence_after();
            issue_o(o_tmem, s_tmem + buf * 64, vd0 + us * (kKvTile >> 4), idesc_o, (d2 & kOpens) ? 0 : 1);
            umma_commit_elect(&B.o_full[X][buf]);
            umma_commit_elect(&B.kv_empty[1][us]);
            ++n_o;
          }
          mbar_arrive_if(&B.kv_empty[1][other.slot], lane == 0 && (two || !mine));
          rv.advance(two ? 2 : 1);
        }
        uint32_t d = 0;
        if (more) {
          if (j == steps) {
            if (!(good = take(k, u))) break;
            j = 0;
            steps = max(u.n[0], u.n[1]);
            more = steps > 0;
          }
          if (more) {
            const int32_t n_mine = X ? u.n[1] : u.n[0], n_other = X ? u.n[0] : u.n[1];
            d = kAny | (j < n_mine ? kMine : 0u) | (u.kind != kShared && j < n_mine && j < n_other ? kTwo : 0u) |
                (j == 0 && n_mine > 0 ? kOpens : 0u);
            const bool mine = d & kMine, two = d & kTwo;
            const RingPos at = two && X ? rk.after(1) : rk, other = two ? (X ? rk : rk.after(1)) : at;
            const bool q = mine && j == 0;  // own K, the other lane's, the tile's queries
            const int w = lane & 3;
            if (!(good = wait_all_or_fail(
                      w == 0 && q ? &B.q_full[X][tiles & 1] : &B.kv_full[0][w == 1 ? other.slot : at.slot],
                      w == 0 && q ? (tiles >> 1) & 1 : (w == 1 ? other.phase : at.phase), fail)))
              break;
            if (q) {
              qd = qd0 + (is_small(u) ? (tiles & 1) * (kQHalf / 2 >> 4) : 0);
              ++tiles;
            }
            if (mine) {
              const uint32_t buf = n_s & 1;
              tmem_fence_after();
              const int32_t us = uniform(at.slot);
              const uint64_t kd = kd0 + us * (kKvTile >> 4);
              issue_s(s_tmem + buf * 64, qd, kd, idesc_s, 0);
              issue_s(s_tmem + buf * 64, qd + (kQHalf >> 4), kd + (kKvHalf >> 4), idesc_s, 1);
              umma_commit_elect(&B.s_full[X][buf]);
              umma_commit_elect(&B.kv_empty[0][us]);
              if (j == n_mine - 1) umma_commit_elect(&B.q_empty[X][(tiles - 1) & 1]);
              ++n_s;
            }
            mbar_arrive_if(&B.kv_empty[0][other.slot], lane == 0 && (two || !mine));
            rk.advance(two ? 2 : 1);
            ++j;
          }
        }
        d2 = d1;
        d1 = d;
      }
      if (!good) {  // the MMAs in flight end before tensor memory is given back
        umma_commit_elect(&B.drained[X]);
        mbar_wait(&B.drained[X], 0);
      }
    } else {
      // ================================================================ late rows of V, a channel half each
      const int h = warp - 14;
#pragma unroll 1
      for (int32_t k = 0;; ++k) {
        const int q = k & (kLate - 1);
        if (!wait_or_fail(&B.late_full[q], (k / kLate) & 1, fail)) break;
        const Late e = B.late[q];
        if (e.slot < 0) break;  // no more
        const uint32_t at = sbase + kOffV + e.slot * kKvTile + h * kKvHalf + (lane & 7) * 16;
        bool odd = false;
        // lanes 8 i .. 8 i + 7: one row
#pragma unroll 1
        for (int32_t x = e.z + (lane >> 3); x < kStep; x += 4) st_shared_v4(at + x * 128, make_uint4(0, 0, 0, 0));
#pragma unroll 1
        for (int32_t x0 = e.y + (lane >> 3); x0 < e.z; x0 += 16) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (x0 + 4 * i < e.z) v[i] = ld_shared_v4(at + (x0 + 4 * i) * 128);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t x = x0 + 4 * i;
            if (x >= e.z) continue;
            const uint4 f = make_uint4(finite_bf16x2(v[i].x), finite_bf16x2(v[i].y), finite_bf16x2(v[i].z),
                                       finite_bf16x2(v[i].w));
            if (f.x != v[i].x || f.y != v[i].y || f.z != v[i].z || f.w != v[i].w) {
              odd = true;
              st_shared_v4(at + x * 128, f);
            }
          }
        }
        odd = __any_sync(0xffffffffu, odd);
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the MMAs read it by that proxy
        __syncwarp();
        if (lane == 0) {
          if (odd && (e.lanes & 1)) *(volatile int32_t*)&B.odd[0] = 1;
          if (odd && (e.lanes & 2)) *(volatile int32_t*)&B.odd[1] = 1;
          mbar_arrive(&B.kv_full[1][e.slot]);
        }
        __syncwarp();
      }
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ================================================================ softmax, outputs and partials
    const int X = (warp - 4) >> 2;
    const int row = (tid - 128) & 127;  // tile row = tensor memory lane
    const uint32_t lane_addr = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t s_tmem = tmem + lane_addr + X * 128;
    const uint32_t o_tmem = tmem + lane_addr + 256 + X * 128;
    const int32_t token = row >> p.gs;
    int32_t n = 0, k = 0, halved = 0;
    Unit u;
    bool good = true;
#pragma unroll 1
    while (good && take(k, u) && (u.n[0] | u.n[1]) != 0) {
      const int32_t steps = X ? u.n[1] : u.n[0];
      if (steps == 0) continue;
      const int32_t tile = u.kind == kShared ? X * p.tpt : 0;  // its first token within the unit's
      const int32_t rows = min(p.tpt, u.tokens - tile) << p.gs;
      const int32_t first_vis = u.pos + tile + 1;     // keys that the tile's first row sees
      const int32_t key0 = X ? u.key0[1] : u.key0[0], g = X ? u.g[1] : u.g[0];
      const int32_t part = u.part < 0 ? -1 : u.part + X * p.tile_rows;
      const bool halves = u.kind == kHalves && u.n[1] > 0;
      const bool act = 32 * (warp & 3) < rows;  // a warp of padding rows only keeps the barriers
      const bool mine = row < rows;  // the rows behind hold whatever the query area held before
      float m_run = -INFINITY, m_nat = 0.f, l = 0.f;  // running reference (log2 units; natural) and sum
      int32_t kb = key0;
#pragma unroll 1
      for (int32_t j = 0; j < steps; ++j, ++n, kb += kStep) {
        if (!(good = wait_or_fail(&B.s_full[X][n & 1], (n >> 1) & 1, fail))) break;
        tmem_fence_after();
        const uint32_t sb = s_tmem + (n & 1) * 64;
        if (act) {
          float l4[4];
          uint32_t pk[32];
          // Any reference near the row's maximum serves for m: P and its sums keep their relative
          // precision as long as nothing overflows. So P is taken against the reference there is, and
          // its sum, needed anyway, tells whether a score lies far above it; only then, and on a
          // unit's first step, a second pass takes the maximum.
#pragma unroll 1
          for (bool exact = j == 0;; exact = true) {
            float v[kStep];
            tmem_ld32(sb, v);
            tmem_ld32(sb + 32, v + 32);
            tmem_wait_ld();
            if (first_vis - kb < kStep) {  // uniform: the step holds a key some row does not see
              const int32_t vis = first_vis + token - kb;
#pragma unroll
              for (int x = 0; x < kStep; ++x)
                if (x >= vis) v[x] = -INFINITY;
            }
            if (exact) {
              float m4[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
              for (int x = 4; x < kStep; x += 2) m4[(x >> 1) & 3] = max3(m4[(x >> 1) & 3], v[x], v[x + 1]);
              const float mx = fmaxf(max3(m4[0], m4[1], m4[2]), m4[3]), m2 = mx * kLog2e;
              float factor = 1.f;
              if (m_run == -INFINITY) {
                m_run = m2;  // nothing in O yet
                m_nat = mx;
              } else if (mine && m2 > m_run) {
                factor = ex2(m_run - m2);
                m_run = m2;
                m_nat = mx;
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
            float off = m_run == -INFINITY ? 0.f : -m_run;
            if (__any_sync(0xffffffffu, mine && fabsf(off) > kFarRef)) {
              off = 0.f;
              if (m_run != -INFINITY)
#pragma unroll
                for (int x = 0; x < kStep; ++x) v[x] -= m_nat;
              __syncwarp();  // threads part here, and tensor memory is accessed by whole warps
            }
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
      // ---------------- the output, or the run's partial
      const int64_t out = ((int64_t)(u.row + tile + token)) * p.Hq + (g << p.gs) + (row & (p.G - 1));
      const int32_t cap = u.kind == kShared ? 128 : ((u.tokens << p.gs) + 7) / 8 * 8;
      if (!(good = wait_or_fail(&B.o_full[X][(n - 1) & 1], ((n - 1) >> 1) & 1, fail))) break;
      tmem_fence_after();
      float f0 = 1.f, f1 = 0.f;  // weights of the lanes' parts
      bool later = false;
      float4* half = nullptr;    // lane 1's part, for which lane 0 waits
      if (halves) {
        half = reinterpret_cast<float4*>(p.half_po) + (int64_t)blockIdx.x * 128 * 32 + row;
        if (X == 1) {
          if (halved > 0 && !(good = wait_or_fail(&B.half_free, (halved - 1) & 1, fail))) break;
          B.half_ml[row] = make_float2(m_run, l);
        } else {
          if (!(good = wait_or_fail(&B.half_full, halved & 1, fail))) break;
          const float2 o = B.half_ml[row];
          const float m = fmaxf(m_run, o.x);
          // whether the row sees keys of lane 1. Their weight may be 0 all the same, beside far larger scores
          // or where all that is left of them is a NaN: 0 times what is not finite then shows it
          later = o.x != -INFINITY || o.y != 0.f;
          if (later) f1 = ex2(o.x - m);
          if (m_run != m) f0 = ex2(m_run - m);
          m_run = m;
          l = l * f0 + (later ? o.y * f1 : 0.f);
        }
        ++halved;
      }
      float scale = 1.f;
      if (part < 0) {
        scale = l == 0.f ? 0.f : 1.0f / l;  // a row that sees no key: o = 0, lse = -inf
        if (mine && p.lse && !(halves && X == 1)) p.lse[out] = l == 0.f ? -INFINITY : (m_run + log2f(l)) * kLn2;
      } else if (mine && !(halves && X == 1)) {
        p.ml[part + row] = make_float2(m_run, l);
      }
      const bool odd = *(volatile int32_t*)&B.odd[X] != 0;
      // Sixteen channels at a time, not unrolled: a tile's end comes too rarely to keep long code in the
      // instruction caches.
#pragma unroll 1
      for (int c = 0; c < 8; ++c) {
        uint32_t raw[16];
        __syncwarp();  // threads of padding rows part from the others below, and tcgen05.ld takes a whole warp
        if (act) {
          tmem_ld16(o_tmem + c * 16, raw);
          tmem_wait_ld();
        }
        if (c == 7) {  // all of O is read: the next unit may overwrite it
          tmem_fence_before();
          __syncwarp();
          mbar_arrive_if(&B.o_free[X], lane == 0);
        }
        if (!mine) continue;
        float o[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __uint_as_float(raw[x]);
        if (odd) {
          // rare: what is not finite in V of the late keys that the row sees (their weights are above 0, so
          // it is added as it is)
          const int32_t end = min(first_vis + token, key0 + steps * kStep);
#pragma unroll 1
          for (int32_t key = max(key0, u.pos + 1); key < end; ++key) {
            int32_t page = p.page_table[(int64_t)u.b * p.max_blocks + key / MSA_BLOCK_TOKENS];
            if (page < 0 || page >= p.num_pages) page = 0;
            const int64_t cell = (int64_t)page * MSA_BLOCK_TOKENS + key % MSA_BLOCK_TOKENS;
            const uint2* v = reinterpret_cast<const uint2*>(p.v_cache + (cell * p.Hkv + g) * 128 + c * 16);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint2 w = v[x], f = make_uint2(finite_bf16x2(w.x), finite_bf16x2(w.y));
              if (f.x != w.x || f.y != w.y) {
                o[4 * x] += bf16_lo(w.x ^ f.x);
                o[4 * x + 1] += bf16_hi(w.x ^ f.x);
                o[4 * x + 2] += bf16_lo(w.y ^ f.y);
                o[4 * x + 3] += bf16_hi(w.y ^ f.y);
              }
            }
          }
        }
        if (halves) {
          if (X == 1) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              __stcg(half + (c * 4 + x) * 128, make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]));
            continue;
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 h = later ? __ldcg(half + (c * 4 + x) * 128) : make_float4(0.f, 0.f, 0.f, 0.f);
            o[4 * x] = fmaf(h.x, f1, o[4 * x] * f0);
            o[4 * x + 1] = fmaf(h.y, f1, o[4 * x + 1] * f0);
            o[4 * x + 2] = fmaf(h.z, f1, o[4 * x + 2] * f0);
            o[4 * x + 3] = fmaf(h.w, f1, o[4 * x + 3] * f0);
          }
        }
        if (part < 0) {
          uint4* dst = reinterpret_cast<uint4*>(p.o + out * 128 + c * 16);
#pragma unroll
          for (int x = 0; x < 2; ++x)
            dst[x] = make_uint4(pack_bf16x2(o[8 * x] * scale, o[8 * x + 1] * scale),
                                pack_bf16x2(o[8 * x + 2] * scale, o[8 * x + 3] * scale),
                                pack_bf16x2(o[8 * x + 4] * scale, o[8 * x + 5] * scale),
                                pack_bf16x2(o[8 * x + 6] * scale, o[8 * x + 7] * scale));
        } else {
          float4* dst = reinterpret_cast<float4*>(p.po + (int64_t)part * 128) + (int64_t)c * 4 * cap + row;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            dst[(int64_t)x * cap] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      }
      if (halves) {  // lane 1's part is written, or read
        __threadfence_block();
        __syncwarp();
        mbar_arrive_if(X == 1 ? &B.half_full : &B.half_free, lane == 0);
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
// A CTA joins rows of a tile: four groups of 256 threads take eight rows each, a thread four channels of one
// row, so a warp reads whole 128-byte lines of the partials' [channel quad][row][4] layout. Of more than four
// pieces the groups share them, for fewer rows at a time, four loads in flight each, and join through shared
// memory. A tile's slices of rows go to different CTAs, since the last tiles are cut into the most pieces
// (2048 tokens on 60032: 120 of them; a CTA per tile took 147 us).
constexpr int kJoinRows = 8;
constexpr int kJoinSplit = 4;
constexpr int kJoinThreads = kJoinRows * 32 * kJoinSplit;

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

__global__ void __launch_bounds__(kJoinThreads) chunk_join_kernel(const __grid_constant__ KParams p, int32_t tiles) {
  __shared__ float2 s_ml[kJoinSplit][kJoinRows * 32];
  __shared__ float4 s_o[kJoinSplit][kJoinRows * 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t = threadIdx.x % (kJoinRows * 32), group = threadIdx.x / (kJoinRows * 32), lane = threadIdx.x & 31;
  const int32_t quad = t / kJoinRows;
  // In the list the most pieces are behind. Of equal runs the first CTAs have what few there are, and the join's
  // first CTAs start first.
  const bool listed = tiles == 0;
  if (listed) tiles = p.head->joins;
  const int32_t slices = p.tile_rows / kJoinRows, step = 2 * p.tile_rows;
  const uint32_t units = (uint32_t)(tiles * slices);  // in 32 bits: tiles are a few thousand at most
#pragma unroll 1
  for (uint32_t u0 = blockIdx.x; u0 < units; u0 += 32 * gridDim.x) {
    // a lane reads one of the CTA's next 32 units
    const uint32_t unit = u0 + lane * gridDim.x;
    JoinTile mine{};
    int32_t my_split = 1;  // 1, 2 or 4
    int32_t my_r0 = 0;
    if (unit < units) {
      int32_t at = (int32_t)unit;
      if (slices > 1) {
        const int32_t slice = (int32_t)(unit / (uint32_t)tiles);
        at += slice * ((int32_t)((uint32_t)tiles / (uint32_t)slices) - tiles);
        if (at >= tiles) at -= tiles;
        my_r0 = slice * kJoinRows;
      }
      mine = p.joins[listed ? tiles - 1 - at : at];
      my_split = mine.pieces <= 4 ? 1 : (mine.pieces <= 8 ? 2 : 4);
    }
    uint32_t todo = __ballot_sync(0xffffffffu, my_r0 < mine.rows && (my_r0 & (kJoinRows * kJoinSplit / my_split - 1)) == 0);
#pragma unroll 1
    for (; todo; todo &= todo - 1) {
      const int src = __ffs(todo) - 1;
      auto get = [&](int32_t x) { return __shfl_sync(0xffffffffu, x, src); };
      const JoinTile e{get(mine.row), get(mine.rows), get(mine.g), get(mine.first), get(mine.rest),
                       get(mine.pieces), get(mine.cap), 0};
      const int32_t split = get(my_split), part = group & (split - 1);
      const int32_t r = get(my_r0) + (group >> (split >> 1)) * kJoinRows + (t & (kJoinRows - 1));
      const bool valid = r < e.rows;
      Joined j{-INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
      if (valid) {
#pragma unroll 1
        for (int32_t k = part; k < e.pieces; k += 4 * split) {
          float2 ml[4];
          float4 o[4];
          int have = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int32_t x = k + u * split;
            if (x < e.pieces) {
              const int64_t at = x == 0 ? e.first : e.rest + (int64_t)(x - 1) * step;
              ml[u] = __ldcs(p.ml + at + r);
              o[u] = __ldcs(reinterpret_cast<const float4*>(p.po) + at * 32 + (int64_t)quad * e.cap + r);
              ++have;
            }
          }
          join_four(j, ml, o, have);
        }
      }
      if (split > 1) {
        s_ml[group][t] = make_float2(j.m, j.l);
        s_o[group][t] = j.acc;
        __syncthreads();
        if (part == 0) {
          float2 ml[4];
          float4 o[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int x = group + (u + 1 < split ? u + 1 : 0);
            ml[u] = s_ml[x][t];
            o[u] = s_o[x][t];
          }
          join_four(j, ml, o, split - 1);
        }
        __syncthreads();  // the shared parts are read
      }
      if (valid && part == 0) {
        const float inv = j.l == 0.f ? 0.f : 1.0f / j.l;  // a row that sees no key: o = 0, lse = -inf
        const int64_t out = (int64_t)(e.row + (r >> p.gs)) * p.Hq + (e.g << p.gs) + (r & (p.G - 1));
        *reinterpret_cast<uint2*>(p.o + out * 128 + quad * 4) =
            make_uint2(pack_bf16x2(j.acc.x * inv, j.acc.y * inv), pack_bf16x2(j.acc.z * inv, j.acc.w * inv));
        if (quad == 0 && p.lse) p.lse[out] = j.l == 0.f ? -INFINITY : (j.m + log2f(j.l)) * kLn2;
      }
    }
  }
}

// ------------------------------------------------------------------------------ host
struct Layout {
  bool self;
  int32_t cap_units, cap_joins, cap_pieces, tile_rows;
  size_t units, joins, ml, po, half, total;
};

Layout layout_of(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t max_blocks, int ctas) {
  Layout y{};
  const int64_t G = Hq / Hkv, tpt = 128 / G, requests = B < T ? B : T;
  // pairs of tiles and single tiles
  const int64_t pairs = Hkv * (T / (2 * tpt)), items = pairs + Hkv * requests;
  const int64_t rows = (T * G + 7) / 8 * 8;
  y.tile_rows = (int32_t)(rows < 128 ? rows : 128);
  // Equal runs where tokens fill one tile per request on average, or there are few pairs: keys are then read
  // by few CTAs each, and what counts is that all CTAs have work, without the plan kernel's time.
  y.self = (T <= B * tpt || pairs <= 2 * ctas) &&
           items * ((2 * (int64_t)max_blocks + 1) * kOwnCost + kTileCost) <= kMostCost;
  if (y.self) {
    y.cap_joins = 2 * ctas;
    y.cap_pieces = 2 * ctas;  // of a run's first and last item
  } else {
    // Pieces of the items that are cut: an item of c steps with r still to come, itself included, has
    // ceil(c / max(16, 2 r / 3 ctas)) pieces, at most 2 c / that for more than one. r falls to 0 over the call,
    // so the sum is at most 2 * 1.5 ctas * (1 + log(most steps / 16)); with less than 16 steps per CTA pieces
    // are as short as these, and at most 2 * ctas.
    const double most = 2.0 * max_blocks / kMinPiece;
    const int64_t cut = (int64_t)(3.0 * ctas * (1.0 + (most > 1 ? log(most) : 0.0))) + 16;
    y.cap_units = (int32_t)(items + cut);
    y.cap_joins = (int32_t)(2 * cut);
    y.cap_pieces = (int32_t)cut;
  }
  size_t at = align_up(sizeof(Header), 256);
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(bytes, 256);
    return here;
  };
  y.units = take((size_t)y.cap_units * sizeof(Unit));
  y.joins = take((size_t)y.cap_joins * sizeof(JoinTile));
  y.ml = take((size_t)y.cap_pieces * 2 * y.tile_rows * sizeof(float2));
  y.po = take((size_t)y.cap_pieces * 2 * y.tile_rows * 128 * sizeof(float));
  y.half = take(Hkv == 1 ? (size_t)ctas * 128 * 128 * sizeof(float) : 0);
  y.total = at;
  return y;
}

template <bool SELF>
cudaError_t launch_kernels(const CUtensorMap& qt, const CUtensorMap& qh, const CUtensorMap& q1, const CUtensorMap& km,
                           const CUtensorMap& vm, const KParams& p, cudaStream_t stream) {
  cudaError_t e;
  static std::atomic<int> regs{0};  // of the kernel as built: the register split counts on it
  if (regs.load(std::memory_order_relaxed) == 0) {
    cudaFuncAttributes fa;
    e = cudaFuncGetAttributes(&fa, chunk_attention_kernel<SELF>);
    if (e != cudaSuccess) return e;
    regs.store(fa.numRegs, std::memory_order_relaxed);
  }
  if (regs.load(std::memory_order_relaxed) != kLaunchRegs) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  if (!SELF) {
    static std::atomic<size_t> raised[kMaxDevices];
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreads);
    cfg.dynamicSmemBytes = (size_t)(p.B + 1) * sizeof(int32_t);
    e = launch_with_smem(chunk_plan_kernel, (kMaxRequests + 1) * sizeof(int32_t), raised,
                         [&] { return cudaLaunchKernelEx(&cfg, chunk_plan_kernel, p); });
    if (e != cudaSuccess) return e;
  }
  static std::atomic<size_t> raised[kMaxDevices];
  cfg.gridDim = dim3((unsigned)p.ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  e = launch_with_smem(chunk_attention_kernel<SELF>, kSmemBytes, raised,
                       [&] { return cudaLaunchKernelEx(&cfg, chunk_attention_kernel<SELF>, qt, qh, q1, km, vm, p); });
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(2 * p.ctas));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, chunk_join_kernel, p, SELF ? 2 * p.ctas : 0);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace

size_t chunk_workspace_bytes(int32_t B, int32_t T, int32_t Hq, int32_t Hkv, int32_t max_blocks, int ctas) {
  return layout_of(B, T, Hq, Hkv, max_blocks, ctas).total;
}

cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t stream) {
  const int ctas = sm_count();
  const Layout y = layout_of(a.B, a.T, a.Hq, a.Hkv, a.max_blocks, ctas);
  const int32_t G = a.Hq / a.Hkv;
  KParams p{};
  p.page_table = a.page_table;
  p.seq_lens = a.seq_lens;
  p.cu_tokens = a.cu_tokens;
  p.B = a.B;
  p.T = a.T;
  p.G = G;
  p.Hq = a.Hq;
  p.Hkv = a.Hkv;
  p.max_blocks = a.max_blocks;
  p.num_pages = a.num_pages;
  while ((1 << p.gs) < G) ++p.gs;
  p.tpt = 128 / G;
  p.ctas = ctas;
  p.cap_units = y.cap_units;
  p.cap_joins = y.cap_joins;
  p.cap_pieces = y.cap_pieces;
  p.tile_rows = y.tile_rows;
  uint8_t* w = a.workspace;
  p.head = reinterpret_cast<Header*>(w);
  p.units = reinterpret_cast<Unit*>(w + y.units);
  p.joins = reinterpret_cast<JoinTile*>(w + y.joins);
  p.ml = reinterpret_cast<float2*>(w + y.ml);
  p.po = reinterpret_cast<float*>(w + y.po);
  p.half_po = reinterpret_cast<float*>(w + y.half);
  p.v_cache = a.v_cache;
  p.o = a.o;
  p.lse = a.lse;
  // query rows as (channel half, head of the group, token row, half, group): a box is G heads of
  // consecutive token rows, one 128-byte line each
  CUtensorMap qt, qh, q1, km, vm;
  const uint64_t qd[5] = {64, (uint64_t)G, (uint64_t)a.T, 2, (uint64_t)a.Hkv};
  const uint64_t qs[4] = {256, (uint64_t)a.q_stride * 2, 128, (uint64_t)G * 256};
  const uint32_t bt[5] = {64, (uint32_t)G, (uint32_t)p.tpt, 1, 1};
  const uint32_t bh[5] = {64, (uint32_t)G, (uint32_t)p.tpt / 2, 1, 1};
  const uint32_t b1[5] = {64, (uint32_t)G, 1, 1, 1};
  // cache cells as (channel half, token, half, group): a box is both halves of 64 tokens
  const uint64_t kd[4] = {64, (uint64_t)a.num_pages * 128, 2, (uint64_t)a.Hkv};
  const uint64_t ks[3] = {(uint64_t)a.Hkv * 256, 128, 256};
  const uint32_t bk[4] = {64, kStep, 2, 1};
  if (!encode_bf16_map(&qt, a.q, 5, qd, qs, bt, true) || !encode_bf16_map(&qh, a.q, 5, qd, qs, bh, true) ||
      !encode_bf16_map(&q1, a.q, 5, qd, qs, b1, true) ||
      !encode_bf16_map(&km, a.k_cache, 4, kd, ks, bk, true) || !encode_bf16_map(&vm, a.v_cache, 4, kd, ks, bk, true))
    return cudaErrorInvalidValue;
  return y.self ? launch_kernels<true>(qt, qh, q1, km, vm, p, stream) : launch_kernels<false>(qt, qh, q1, km, vm, p, stream);
}

}  // namespace msa
