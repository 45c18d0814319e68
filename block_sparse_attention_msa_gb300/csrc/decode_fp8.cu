// Paged sparse decode attention on the quantised K/V cache: the same flat page tables, rows and
// partial slots as the bf16 form (decode.cu), half its bytes.
//
// A key is k_n = 2^a_n k'_n and a value v_n = 2^b_n v'_n with k', v' rows of e4m3 numbers and one power of
// two per token and group. With t_n = (q . k'_n) 2^a_n log2(e),
//   m = max t_n,  l = sum 2^(t_n - m),  M = max (t_n + b_n),  O = sum 2^(t_n + b_n - M) v'_n
//   o = O 2^(M - m) / l,  lse = (m + log2 l) ln 2.
// The values' powers of two are part of the weights, so the products run on the stored numbers as they
// are. The weights have a maximum of their own, M: they stay in (0, 2^8] of it (see kFar) however the
// magnitudes of V differ from token to token, and l, without the powers, keeps m.
//
// e4m3 becomes fp16 in one instruction per pair, exactly, so both products are fp16 MMAs with fp32
// sums. The other operands are rounded to fp16: q after a power of two that brings its head's largest
// magnitude to [2^14, 2^15) (exact down to 2^-28 of that, then 2^-39 of it), the weights at 2^-11 of
// their value. fp16 keeps that to 2^-14, and a weight carries its value's power of two, so beside one token
// of far larger values the others' weights lie far below the largest. The weights are therefore taken times
// 2^7, to 2^15 at most, just within fp16: 2^-11 of their value down to 2^-21 of the largest, and 2^-32 of the
// largest below. bf16 weights, as beside bf16 values, would be at 2^-8.
//
// GB300 design. HBM-bound: 2 * 129 bytes per (row, group, token), so what counts is loads in flight and
// few instructions per byte.
//  * A page of a group is 16 KB in one piece in this cache ([page][group][token][channel]), so a warp
//    brings a step of 32 tokens (4 KB of K, 4 KB of V, 64 scales) with four bulk copies into its own
//    ring, a step ahead, and waits on its own barrier: no warp waits for another. (Two stages of 8 KB
//    in each of eight warps keep 64 KB a SM in flight beside what is worked on; three were slower, 55.9
//    instead of 53.2 us, and so were ten or twelve warps, 56.7.)
//  * The tokens are the M side of the MMAs (16 of them), the group's heads the N side (8, or two tiles
//    of 8): S^T = K Q^T and O^T = V^T P^T, so 8 heads fill their tile (as the 16-row side they would be
//    half of it: twice the MMAs, conversions alike). P^T goes from accumulator to operand layout by
//    an 8x8 transpose in registers (movmatrix).
//  * Which token is which row of a tile, and which channel which K index, is free as long as both
//    operands agree: a lane reads 16 channels of a token with one 16-byte load, and the choice of
//    rows below meets the 128-byte swizzle of the copies without bank conflicts. O^T then leaves a
//    lane 16 neighbouring channels of two heads.
//  * The batch's (row, page) units are split over the warps of a persistent grid in equal runs; a
//    warp leaves a row's partial in the slot of the first page it covered, and a second kernel joins
//    a row's slots in their order, launched beside it so that its start costs nothing. Few rows go to
//    clusters of four CTAs instead, which join through each other's shared memory in the same launch.
//
// Measured, Hq/Hkv/D = 64/8/128, top 16: 64 rows on 8k-128k 50 us (264 MB, 5.3 TB/s, 78 % of the
// copy rate; the bf16 form reads 528 MB), 4 rows on 1M 11.0 us, 1 row on 2048 8 us; 16 heads per group (Hq 128),
// 64 rows: 56 us. With two warps per scheduler the issue slots are 40 % used and DRAM 70 %: what is left is the
// latency from a step's arrival to its products' results, which more warps or stages do not hide (they were
// slower, above).
#include <cooperative_groups.h>

#include <algorithm>

#include "common.cuh"
#include "host_util.h"
#include "kernels.h"
#include "softmax_math.cuh"

MSA_DEFINE_ERROR_WORD(dec8)

namespace msa {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kTok = 32;                       // tokens per step
constexpr uint32_t kTile = kTok * 128;         // K or V of a step
constexpr uint32_t kStep = 2 * kTile;
constexpr uint32_t kRing = kStages * kStep;    // of one warp: 16 KB
constexpr uint32_t kScales = 2 * kTok;         // bytes per step
// A score may exceed the softmax's reference by this much (log2) before the reference moves, and weights are
// taken times 2^kLift: they stay at 2^15 at most, within fp16 (65504).
constexpr float kFar = 8.f;
constexpr float kLift = 7.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Bars {
  uint64_t full[kWarps][kStages];
  alignas(128) uint8_t scale[kWarps][kStages][kScales];  // K, V; 64-byte lines: 16-byte aligned bulk copies
};
static_assert(kTile % 1024 == 0 && kTok % 16 == 0, "alignment of the copies' targets");
constexpr size_t kSmemBytes = 1024 + kWarps * kRing + sizeof(Bars);

struct KParams {
  const uint16_t* q;
  const uint8_t* k_scale;
  const uint8_t* v_scale;
  const int32_t* fpt;
  const int32_t* lens;
  int32_t Hkv, hs, G, topk;
  int32_t rows, units;             // rows = R*Hkv, units = rows*topk
  int64_t num_pages;
  float* part_o;                   // [rows, topk, G, 128]
  float* part_lse;                 // [rows, topk, G]
};

// A warp-uniform, forward-moving view of a 32-bit array: lane l holds a[base + l].
struct RegWindow {
  int32_t base = INT32_MIN / 2, val = 0;
  __device__ __forceinline__ int32_t get(const int32_t* a, int32_t n, int32_t i, int lane) {
    if (i >= base + 32) {
      base = i;
      val = i + lane < n ? __ldg(a + i + lane) : 0;
    }
    return __shfl_sync(0xffffffffu, val, i - base);
  }
};

// A step of a warp's walk: row, page slot (row * topk + page), first token and the row's visible tokens.
struct Step {
  int32_t f, slot, n0, len;  // f < 0: the walk is over
};

// e4m3 pairs as fp16 pairs, exactly.
__device__ __forceinline__ uint32_t f16x2_lo(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, l;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.rn.f16x2.e4m3x2 %0, h;\n}" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// D(16x8, fp32) += A(16x16, fp16, row) * B(16x8, fp16, col)
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Walks a warp's unit range [u, u1): unit u = f*topk + pi is page pi of row f; pages past the row's
// visible length are skipped; each page is ceil(tokens/32) steps. next() brings the step's 32 tokens of K
// and V, and their scales, into a stage. An invalid page id is recorded and read as page 0, group 0.
struct Walk {
  int32_t u, u1, f, pi, len, npg, c, nc, row;
  RegWindow lens, pages;
  __device__ __forceinline__ void start(const KParams& p, int32_t u0, int32_t uend, int lane) {
    u = u0;
    u1 = uend;
    f = u0 / p.topk;
    pi = u0 - f * p.topk;
    c = nc = 0;
    if (u < u1) {  // both round trips at once
      (void)pages.get(p.fpt, p.units, u, lane);
      len = min(max(lens.get(p.lens, p.rows, f, lane), 0), p.topk * MSA_BLOCK_TOKENS);
    }
    npg = (len + MSA_BLOCK_TOKENS - 1) / MSA_BLOCK_TOKENS;
  }
  __device__ __forceinline__ Step next(const KParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                       uint8_t* dst, uint8_t* scales, uint64_t* full, int lane) {
    while (c >= nc) {
      if (u >= u1) return {-1, 0, 0, 0};
      if (pi == p.topk) {
        pi = 0;
        ++f;
        len = min(max(lens.get(p.lens, p.rows, f, lane), 0), p.topk * MSA_BLOCK_TOKENS);
        npg = (len + MSA_BLOCK_TOKENS - 1) / MSA_BLOCK_TOKENS;
      }
      if (pi >= npg) {  // the rest of this row has no visible tokens
        u += p.topk - pi;
        pi = p.topk;
        continue;
      }
      const int32_t v = pages.get(p.fpt, p.units, u, lane);
      int32_t page = v >> (7 + p.hs), g = v & ((MSA_BLOCK_TOKENS << p.hs) - 1);
      if (v < 0 || page >= p.num_pages || g >= p.Hkv) {
        if (lane == 0) msa_record_error(kErrBadPage);
        page = g = 0;
      }
      row = ((page << p.hs) + g) * MSA_BLOCK_TOKENS;
      c = 0;
      nc = (min(MSA_BLOCK_TOKENS, len - pi * MSA_BLOCK_TOKENS) + kTok - 1) / kTok;
      ++u;
      ++pi;
    }
    if (lane == 0) {
      const int32_t at = row + c * kTok;
      mbar_expect_tx(full, kStep + kScales);
      tma_load_2d(dst, &kmap, full, 0, at);
      tma_load_2d(dst + kTile, &vmap, full, 0, at);
      bulk_load(scales, p.k_scale + at, kTok, full);
      bulk_load(scales + kTok, p.v_scale + at, kTok, full);
    }
    return {f, u - 1, (pi - 1) * MSA_BLOCK_TOKENS + c++ * kTok, len};
  }
};

// What a row segment leaves in a lane, for HT tiles of 8 heads: heads 8 h + 2 tig + {0, 1}, channels
// 16 chunk + 0..15 (chunk: 4 (gid & 1) + gid / 2), O relative to 2^(M - kLift).
template <int HT>
struct Seg {
  float o[HT][8][4];  // [.][channel pair][channel 2x: heads 0, 1; channel 2x + 1: heads 0, 1]
  float m[HT][2], l[HT][2], M[HT][2];
};

// One warp's walk over the units [u0, u1) through its ring. At the end of each row segment it calls
// emit(f, slot_row, seg) with l summed over the warp. False after a wait that gave up.
template <int HT, class Emit>
__device__ __forceinline__ bool walk_units(const KParams& p, const CUtensorMap& kmap, const CUtensorMap& vmap,
                                           uint8_t* ring, Bars& bars, int warp, int32_t u0, int32_t u1, int lane,
                                           Emit&& emit) {
  const int gid = lane >> 2, tig = lane & 3, G = p.G;
  const uint32_t base = smem_u32(ring), sbase = smem_u32(bars.scale[warp]);
  // The rows of an 8-row tile are the tokens perm(0..7) = 0, 4, 1, 5, 2, 6, 3, 7, and lane gid reads
  // chunk perm(gid) of V: eight lanes of a load then meet eight different 16-byte columns.
  const uint32_t perm = ((gid & 1) << 2) | (gid >> 1);
  Walk walk;
  walk.start(p, u0, u1, lane);
  uint32_t issued = 0;
  auto prefetch = [&]() {
    const uint32_t s = issued % kStages;
    const Step x = walk.next(p, kmap, vmap, ring + s * kStep, bars.scale[warp][s], &bars.full[warp][s], lane);
    issued += x.f >= 0;
    return x;
  };
  Step ahead[kStages - 1];
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) ahead[k] = prefetch();

  uint32_t it = 0;
#pragma unroll 1
  while (ahead[0].f >= 0) {
    // ---- a row segment
    const int32_t f = ahead[0].f, slot_row = ahead[0].slot, len = ahead[0].len;
    // Q^T fragments (K index 16 x heads): k-step ks takes channels 64 (ks / 4) + 16 tig + 4 (ks % 4) + 0..3
    // of head 8 h + gid
    uint32_t qb[HT][8][2];
    // Of this lane's heads as columns of S^T: qf * qw = 2^eq * log2(e), qw the part of 2^eq above 1. A score is
    // (sc * (2^a * qf)) * qw: factors below 1 come together, so that nothing leaves fp32 but what the score does.
    float qf[HT][2], qw[HT][2];
#pragma unroll
    for (int h = 0; h < HT; ++h) {
      const int head = 8 * h + gid;
      uint32_t w[16];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (head < G)
          v = __ldg(reinterpret_cast<const uint4*>(p.q + ((int64_t)f * G + head) * 128 + (x >> 1) * 64 + tig * 16) + (x & 1));
        w[4 * x] = v.x;
        w[4 * x + 1] = v.y;
        w[4 * x + 2] = v.z;
        w[4 * x + 3] = v.w;
      }
      uint32_t m2 = 0;
#pragma unroll
      for (int x = 0; x < 16; ++x) m2 = __vmaxu2(m2, w[x] & 0x7fff7fffu);
      int32_t e = (int32_t)(max(m2 & 0xffffu, m2 >> 16) >> 7);
      e = max(e, __shfl_xor_sync(0xffffffffu, e, 1));
      e = max(e, __shfl_xor_sync(0xffffffffu, e, 2));
      // biased exponent of the head's largest magnitude; q * 2^(141 - e) lies below 2^15
      e = min(max(e, 15), 254);
      const float up = __int_as_float((268 - e) << 23);  // 2^(141 - e): exponent field 141 - e + 127
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        qb[h][ks][0] = pack_f16x2(bf16_lo(w[2 * ks]) * up, bf16_hi(w[2 * ks]) * up);
        qb[h][ks][1] = pack_f16x2(bf16_lo(w[2 * ks + 1]) * up, bf16_hi(w[2 * ks + 1]) * up);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int32_t ey = __shfl_sync(0xffffffffu, e, (2 * tig + y) * 4);
        // 2^(e - 141): exponent field e - 14 >= 1
        qf[h][y] = kLog2e * __int_as_float(min(ey - 14, 127) << 23);
        qw[h][y] = __int_as_float(max(ey - 14, 127) << 23);
      }
    }
    Seg<HT> s;
#pragma unroll
    for (int h = 0; h < HT; ++h) {
#pragma unroll
      for (int x = 0; x < 8; ++x) s.o[h][x][0] = s.o[h][x][1] = s.o[h][x][2] = s.o[h][x][3] = 0.f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        s.m[h][y] = s.M[h][y] = -INFINITY;
        s.l[h][y] = 0.f;
      }
    }

#pragma unroll 1
    do {
      const int n0 = ahead[0].n0;
      // the next step goes into the stage that the last one used
#pragma unroll
      for (int k = 0; k + 1 < kStages - 1; ++k) ahead[k] = ahead[k + 1];
      ahead[kStages - 2] = prefetch();
      const uint32_t st = it % kStages;
      // each thread waits for itself; the vote brings the warp together, as the products take it, with one answer
      if (!__all_sync(0xffffffffu, mbar_wait(&bars.full[warp][st], (it / kStages) & 1))) {
        if (lane == 0) msa_record_error(kErrTimeout);
        for (uint32_t k = it + 1; k < issued; ++k)  // the copies in flight land before the CTA leaves
          mbar_wait(&bars.full[warp][k % kStages], (k / kStages) & 1);
        return false;
      }
      const uint32_t kb = base + st * kStep, vb = kb + kTile, sb = sbase + st * kScales;
      // ---- S^T = K Q^T: two tiles of 16 tokens
      float sc[HT][2][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int h = 0; h < HT; ++h) sc[h][mt][0] = sc[h][mt][1] = sc[h][mt][2] = sc[h][mt][3] = 0.f;
        const uint32_t r0 = mt * 16 + perm, r1 = r0 + 8;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint4 a = lds128(kb + sw128(r0, tig + 4 * c)), b = lds128(kb + sw128(r1, tig + 4 * c));
          const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = f16x2_lo(aw[j]), a2 = f16x2_hi(aw[j]);
            const uint32_t a1 = f16x2_lo(bw[j]), a3 = f16x2_hi(bw[j]);
#pragma unroll
            for (int h = 0; h < HT; ++h)
              mma_f16(sc[h][mt], a0, a1, a2, a3, qb[h][4 * c + j][0], qb[h][4 * c + j][1]);
          }
        }
      }
      // ---- softmax statistics: token 16 mt + 8 r + perm, heads 2 tig + y
      float ks[2][2], vs[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const uint32_t tok = mt * 16 + r * 8 + perm;
          const uint32_t b = lds8(sb + tok);
          ks[mt][r] = __int_as_float(b ? b << 23 : 0x400000);  // 2^(b - 127)
          vs[mt][r] = (float)((int32_t)lds8(sb + kTok + tok) - 127);
        }
      uint32_t pb[HT][2][2];
#pragma unroll
      for (int h = 0; h < HT; ++h) {
        float w[2][4];
        float mx[2] = {-INFINITY, -INFINITY}, Mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int r = c >> 1, y = c & 1;
            float t = sc[h][mt][c] * (ks[mt][r] * qf[h][y]) * qw[h][y];
            if (n0 + mt * 16 + r * 8 + (int)perm >= len) t = -INFINITY;
            sc[h][mt][c] = t;
            w[mt][c] = t + vs[mt][r];
            mx[y] = fmaxf(mx[y], t);
            Mx[y] = fmaxf(Mx[y], w[mt][c]);
          }
        // Any references near the maxima serve, so they move only when a score lies far above them.
        bool far = false;
#pragma unroll
        for (int y = 0; y < 2; ++y) far |= mx[y] > s.m[h][y] + kFar || Mx[y] > s.M[h][y] + kFar;
        if (__any_sync(0xffffffffu, far)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xffffffffu, mx[y], o));
              Mx[y] = fmaxf(Mx[y], __shfl_xor_sync(0xffffffffu, Mx[y], o));
            }
          float fo[2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const float mn = fmaxf(s.m[h][y], mx[y]), Mn = fmaxf(s.M[h][y], Mx[y]);
            s.l[h][y] *= mn == -INFINITY ? 1.f : ex2(s.m[h][y] - mn);
            fo[y] = Mn == -INFINITY ? 1.f : ex2(s.M[h][y] - Mn);
            s.m[h][y] = mn;
            s.M[h][y] = Mn;
          }
#pragma unroll
          for (int x = 0; x < 8; ++x)
#pragma unroll
            for (int c = 0; c < 4; ++c) s.o[h][x][c] *= fo[c & 1];
        }
        float mref[2], Mref[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          mref[y] = s.m[h][y] == -INFINITY ? 0.f : s.m[h][y];
          Mref[y] = (s.M[h][y] == -INFINITY ? 0.f : s.M[h][y]) - kLift;
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            s.l[h][c & 1] += ex2(sc[h][mt][c] - mref[c & 1]);
            w[mt][c] = ex2(w[mt][c] - Mref[c & 1]);
          }
          // tokens as rows, heads as columns -> the other way round, as P^T's operand wants them
          pb[h][mt][0] = transpose8x8(pack_f16x2(w[mt][0], w[mt][1]));
          pb[h][mt][1] = transpose8x8(pack_f16x2(w[mt][2], w[mt][3]));
        }
      }
      // ---- O^T += V^T P^T: per 16 tokens this lane reads 16 channels of tokens tig, tig + 4, + 8, + 12
      const bool cut = n0 + kTok > len;  // cells behind the row's last token may hold NaN, and 0 * NaN is NaN
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t r = mt * 16 + tig + 4 * i;
          v[i] = lds128(vb + sw128(r, perm));
          if (cut && n0 + (int)r >= len) v[i] = make_uint4(0, 0, 0, 0);
        }
        const uint32_t vw4[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                    {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t lo01 = __byte_perm(vw4[0][i], vw4[1][i], 0x5140), hi01 = __byte_perm(vw4[0][i], vw4[1][i], 0x7362);
          const uint32_t lo23 = __byte_perm(vw4[2][i], vw4[3][i], 0x5140), hi23 = __byte_perm(vw4[2][i], vw4[3][i], 0x7362);
          const uint32_t a[2][4] = {{f16x2_lo(lo01), f16x2_hi(lo01), f16x2_lo(lo23), f16x2_hi(lo23)},
                                    {f16x2_lo(hi01), f16x2_hi(hi01), f16x2_lo(hi23), f16x2_hi(hi23)}};
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int h = 0; h < HT; ++h)
              mma_f16(s.o[h][2 * i + x], a[x][0], a[x][1], a[x][2], a[x][3], pb[h][mt][0], pb[h][mt][1]);
        }
      }
      __syncwarp();  // every lane is done with the stage before it is refilled
      ++it;
    } while (ahead[0].f == f);

    // ---- the segment's sums over the lanes that hold the same heads
#pragma unroll
    for (int h = 0; h < HT; ++h)
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) s.l[h][y] += __shfl_xor_sync(0xffffffffu, s.l[h][y], o);
    emit(f, slot_row, s);
  }
  return true;
}

// Writes a segment's partial as normalised fp32 rows dst[head][128] and its LSE per head.
template <int HT>
__device__ __forceinline__ void store_partial(float* dst, float* lse_dst, const Seg<HT>& s, int G, int lane) {
  const int gid = lane >> 2, tig = lane & 3;
  const int chunk = ((gid & 1) << 2) | (gid >> 1);
#pragma unroll
  for (int h = 0; h < HT; ++h)
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int head = 8 * h + 2 * tig + y;
      if (head >= G) continue;
      const float l = s.l[h][y];
      // O 2^(M - kLift - m) / l, the power in two halves: it may leave fp32's range where O's product does not
      const float half = l == 0.f ? 0.f : ex2(0.5f * (s.M[h][y] - kLift - s.m[h][y])), inv = l == 0.f ? 0.f : 1.0f / l;
      float4* d = reinterpret_cast<float4*>(dst + head * 128 + chunk * 16);
#pragma unroll
      for (int x = 0; x < 4; ++x)
        d[x] = make_float4(s.o[h][2 * x][y] * half * inv * half, s.o[h][2 * x][y + 2] * half * inv * half,
                           s.o[h][2 * x + 1][y] * half * inv * half, s.o[h][2 * x + 1][y + 2] * half * inv * half);
      if (gid == 0) lse_dst[head] = l == 0.f ? -INFINITY : (s.m[h][y] + log2f(l)) * kLn2;
    }
}

__device__ __forceinline__ uint8_t* init_smem(uint8_t* raw, Bars*& bars) {
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  bars = reinterpret_cast<Bars*>(smem + kWarps * kRing);
  if (threadIdx.x < kWarps * kStages) mbar_init(&bars->full[0][0] + threadIdx.x, 1);
  mbar_fence_init();
  __syncthreads();
  return smem;
}

template <int HT>
__global__ void __launch_bounds__(kThreads, 1)
    paged_decode_fp8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                            const __grid_constant__ KParams p) {
  extern __shared__ uint8_t smem_raw[];
  Bars* bars;
  uint8_t* smem = init_smem(smem_raw, bars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;
  const int64_t nw = (int64_t)gridDim.x * kWarps, wg = (int64_t)blockIdx.x * kWarps + warp;
  const int32_t u0 = (int32_t)(p.units * wg / nw), u1 = (int32_t)(p.units * (wg + 1) / nw);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // every slot of the range starts empty; a row segment's partial overwrites its first slot
  for (int64_t i = (int64_t)u0 * G + lane; i < (int64_t)u1 * G; i += 32) p.part_lse[i] = -INFINITY;
  __syncwarp();
  walk_units<HT>(p, kmap, vmap, smem + warp * kRing, *bars, warp, u0, u1, lane,
                 [&](int32_t, int32_t slot_row, const Seg<HT>& s) {
                   store_partial<HT>(p.part_o + (int64_t)slot_row * G * 128, p.part_lse + (int64_t)slot_row * G, s, G, lane);
                 });
}

// Few rows (a small batch at long context): a cluster of kClusterCtas CTAs per flattened row, as in the
// bf16 form: its warps split the row's pages, leave their partials in their own ring, and the
// cluster's CTAs merge a share of the row's outputs each through distributed shared memory.
constexpr int kClusterCtas = 4, kClusterWarps = 8, kClusterThreads = kClusterWarps * 32;
static_assert(kClusterWarps <= kWarps, "their rings fit");

template <int HT>
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads, 1)
    paged_decode_fp8_cluster_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                                    const __grid_constant__ KParams p, uint16_t* __restrict__ o_out,
                                    float* __restrict__ lse_out) {
  namespace cg = cooperative_groups;
  extern __shared__ uint8_t smem_raw[];
  Bars* bars;
  uint8_t* smem = init_smem(smem_raw, bars);
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster.block_rank();
  const int64_t f = blockIdx.x / kClusterCtas;  // flattened row (request, group)
  const int G = p.G;
  constexpr int kParts = kClusterCtas * kClusterWarps;
  const int wi = rank * kClusterWarps + warp;
  const int32_t u0 = (int32_t)(f * p.topk) + p.topk * wi / kParts;
  const int32_t u1 = (int32_t)(f * p.topk) + p.topk * (wi + 1) / kParts;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // a warp's partial, once its walk is over: O [G][128] fp32, then its G LSEs
  float* part = reinterpret_cast<float*>(smem + warp * kRing);
  float* part_lse = part + 16 * 128;
  bool emitted = false;
  const bool good = walk_units<HT>(p, kmap, vmap, smem + warp * kRing, *bars, warp, u0, u1, lane,
                                   [&](int32_t, int32_t, const Seg<HT>& s) {
                                     __syncwarp();  // the ring's last step is read: it becomes the partial's space
                                     store_partial<HT>(part, part_lse, s, G, lane);
                                     emitted = true;
                                   });
  if (!emitted && good) {  // no visible page in the range: O = 0, LSE -inf
    for (int i = lane; i < G * 128; i += 32) part[i] = 0.f;
    for (int h = lane; h < G; h += 32) part_lse[h] = -INFINITY;
  }
  cluster.sync();  // every warp's partial is in its CTA's shared memory
  // the row's merge weights, one warp per head, lane j = partial j: w[h][j] = e^(lse_j - lse) (0 for an
  // empty range), kept in this CTA (behind warp 0's partial, which stays readable)
  float* wts = reinterpret_cast<float*>(smem + 12 * 1024);
  static_assert(kParts == 32, "one lane per partial");
  for (int h = warp; h < G; h += kClusterWarps) {
    const float* pl = cluster.map_shared_rank(
        reinterpret_cast<float*>(smem + (lane % kClusterWarps) * kRing) + 16 * 128, lane / kClusterWarps);
    const float l = pl[h];
    const float m = warp_max(l);
    // the lane's own part alone says whether it is empty: a NaN, which the maximum passes over, stays one
    const float e = l == -INFINITY ? 0.f : __expf(l - m);
    const float total = warp_sum(e);
    wts[h * 32 + lane] = total == 0.f ? 0.f : e / total;
    if (lane == 0 && lse_out && rank == (h % kClusterCtas))
      lse_out[f * G + h] = total == 0.f ? -INFINITY : m + __logf(total);
  }
  __syncthreads();
  // (head, channel) outputs of the row, dealt over the cluster's threads: 32 independent remote loads each
  for (int item = rank * kClusterThreads + (int)threadIdx.x; item < G * 128; item += kClusterCtas * kClusterThreads) {
    const int h = item >> 7, ch = item & 127;
    float acc = 0.f;
#pragma unroll
    for (int j = 0; j < kParts; ++j) {
      const float* pj =
          cluster.map_shared_rank(reinterpret_cast<float*>(smem + (j % kClusterWarps) * kRing), j / kClusterWarps);
      acc = fmaf(wts[h * 32 + j], pj[h * 128 + ch], acc);
    }
    o_out[(f * G + h) * 128 + ch] = __bfloat16_as_ushort(__float2bfloat16_rn(acc));
  }
  cluster.sync();  // no CTA leaves while another still reads its shared memory
}

// Joins the partials of a flattened row's slots, in their order: a warp per (row, head). Lane j weighs
// slots j and j + 32 (at most 64 of them); the partials that carry weight then stream four at a time, all
// their loads in flight, four channels a lane. Few registers, so that its CTAs stand beside the attention
// kernel's and wait there.
constexpr int kMergeWarps = 4;
__global__ void __launch_bounds__(kMergeWarps * 32, 12) decode_fp8_merge_kernel(const __grid_constant__ KParams p,
                                                                                uint16_t* __restrict__ o_out,
                                                                                float* __restrict__ lse_out) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t item = (int64_t)blockIdx.x * kMergeWarps + warp;  // row * G + head
  const bool mine = item < (int64_t)p.rows * p.G;
  const int64_t f = item / p.G;
  const int e = (int)(item - f * p.G);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!mine) return;
  const float* lse = p.part_lse + f * p.topk * p.G + e;
  const float4* part = reinterpret_cast<const float4*>(p.part_o + (f * p.topk * p.G + e) * 128) + lane;
  float l[2], w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int s = lane + 32 * h;
    l[h] = s < p.topk ? __ldcs(lse + s * p.G) : -INFINITY;
  }
  const float m = warp_max(fmaxf(l[0], l[1]));
#pragma unroll
  for (int h = 0; h < 2; ++h) w[h] = l[h] == -INFINITY ? 0.f : ex2((l[h] - m) * kLog2e);
  // slots with a partial; a NaN among them reaches the output
  uint64_t rest = (uint64_t)__ballot_sync(0xffffffffu, l[0] != -INFINITY) |
                  ((uint64_t)__ballot_sync(0xffffffffu, l[1] != -INFINITY) << 32);
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  while (rest) {
    constexpr int kBatch = 4;
    float wk[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int s = rest ? __ffsll((long long)rest) - 1 : -1;
      rest &= rest - 1;
      wk[k] = __shfl_sync(0xffffffffu, s >= 32 ? w[1] : w[0], s & 31);
      v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s >= 0) v[k] = __ldcs(part + (int64_t)s * p.G * 32);
      else wk[k] = 0.f;
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      acc[0] = fmaf(wk[k], v[k].x, acc[0]);
      acc[1] = fmaf(wk[k], v[k].y, acc[1]);
      acc[2] = fmaf(wk[k], v[k].z, acc[2]);
      acc[3] = fmaf(wk[k], v[k].w, acc[3]);
    }
  }
  const float total = warp_sum(w[0] + w[1]);
  const float inv = total == 0.f ? 0.f : 1.0f / total;
  *reinterpret_cast<uint2*>(o_out + item * 128 + lane * 4) =
      make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (lane == 0 && lse_out) lse_out[item] = total == 0.f ? -INFINITY : m + log2f(total) * kLn2;
}

template <int HT>
cudaError_t launch(const CUtensorMap& kmap, const CUtensorMap& vmap, const KParams& p, const DecodeFp8Args& a,
                   cudaStream_t stream) {
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const int sms = sm_count();
  if ((int64_t)p.rows * kClusterCtas <= sms) {  // few rows: one cluster per row, no partial in HBM, no merge kernel
    static std::atomic<size_t> raised[kMaxDevices];
    cfg.gridDim = dim3((unsigned)(p.rows * kClusterCtas));
    cfg.blockDim = dim3(kClusterThreads);
    return launch_with_smem(paged_decode_fp8_cluster_kernel<HT>, kSmemBytes, raised, [&] {
      return cudaLaunchKernelEx(&cfg, paged_decode_fp8_cluster_kernel<HT>, kmap, vmap, p, a.o, a.lse);
    });
  }
  static std::atomic<size_t> raised[kMaxDevices];
  cfg.gridDim = dim3((unsigned)std::min<int64_t>(((int64_t)p.units + kWarps - 1) / kWarps, sms));
  cudaError_t e = launch_with_smem(paged_decode_fp8_kernel<HT>, kSmemBytes, raised, [&] {
    return cudaLaunchKernelEx(&cfg, paged_decode_fp8_kernel<HT>, kmap, vmap, p);
  });
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(((int64_t)p.rows * p.G + kMergeWarps - 1) / kMergeWarps));
  cfg.blockDim = dim3(kMergeWarps * 32);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, decode_fp8_merge_kernel, p, a.o, a.lse);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace

cudaError_t launch_paged_decode_fp8(const DecodeFp8Args& a, cudaStream_t stream) {
  KParams p{};
  p.q = a.q;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.fpt = a.fpt;
  p.lens = a.lens;
  p.Hkv = a.Hkv;
  while ((1 << p.hs) < a.Hkv) ++p.hs;
  p.G = a.Hq / a.Hkv;
  p.topk = a.topk;
  p.rows = a.R * a.Hkv;
  p.units = p.rows * a.topk;
  p.num_pages = a.num_pages;
  p.part_o = a.part_o;
  p.part_lse = a.part_lse;
  if (p.units <= 0) return cudaSuccess;
  CUtensorMap kmap, vmap;
  const int64_t rows = a.num_pages * a.Hkv * MSA_BLOCK_TOKENS;
  if (!encode_u8_rows_map(&kmap, a.k_cache, rows, kTok) || !encode_u8_rows_map(&vmap, a.v_cache, rows, kTok))
    return cudaErrorInvalidValue;
  return p.G > 8 ? launch<2>(kmap, vmap, p, a, stream) : launch<1>(kmap, vmap, p, a, stream);
}

}  // namespace msa
