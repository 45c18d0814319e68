// The quantised K/V cache: rows quantised as they are written, and read back.
//
// A row is one token of one KV group: 128 channels of K or of V. It is held as 128 e4m3 numbers and
// one power of two, 2^e with e the smallest integer for which every |x| <= 448 * 2^e (448: the largest
// e4m3 number): x is stored as the nearest e4m3 number to x * 2^-e, ties to even. A power of two costs
// e4m3, a floating-point format, next to nothing against any other scale (the relative error is 2^-4
// of a value at most either way) and makes every step but that one rounding exact: x * 2^-e is exact in
// fp32, and the value read back, e4m3 * 2^e, has four significant bits and is exact in bf16. So a row
// that was read back is held exactly when it is written again. e is held as a byte, e + 127: 129 bytes a
// row instead of 256.
//
// Both kernels copy: 385 bytes a row move either way, so HBM bounds long runs and the launch bounds
// decode steps. Eight threads own a row, 16 channels each (two 16-byte loads of bf16, one 16-byte
// store of e4m3, or the reverse); a row's largest magnitude takes three shuffles on packed bit patterns.
// The 32 bytes of bf16 move in one access where they are aligned: two 16-byte stores half a sector each
// cost the read-back a fifth of its rate (4.5 instead of 5.2 TB/s). Measured, replayed from a graph, Hkv 8:
// 60032 rows read back in 56.5 us (370 MB, 6.5 TB/s, 96% of a copy), 32768 rows written and read back in
// 64 us (404 MB, 6.3 TB/s), 8 rows in 4.1 us. Two rows of a thread: one 62.8 and 67.8 us, four 57.6 and
// 64.7 us; a persistent grid 70.5 us for the first.
#include "common.cuh"
#include "host_util.h"
#include "kernels.h"

MSA_DEFINE_ERROR_WORD(kvq)

namespace msa {

namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 2;  // rows of a thread, all requested before the first store

struct QuantParams {
  const uint16_t* src[2];  // K, V rows
  int64_t src_stride[2];   // elements between token rows
  uint8_t* cache[2];       // [num_pages, Hkv, 128, 128] e4m3
  uint8_t* scale[2];       // [num_pages, Hkv, 128]
  const int32_t* slots;
  int32_t T, hs;           // hs: log2 of Hkv
  int64_t cells;
};

// Larger of the magnitudes of packed bf16 pairs, as bit patterns.
__device__ __forceinline__ uint32_t max_mag2(uint32_t a, uint32_t b) { return __vmaxu2(a, b & 0x7fff7fffu); }

// Two floats as e4m3 bytes (lo in the low byte), nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 bytes as fp16 pairs (exact).
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint16_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(x));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t x) {
  float r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, l;\n}" : "=f"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float f16_hi(uint32_t x) {
  float r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n cvt.f32.f16 %0, h;\n}" : "=f"(r) : "r"(x));
  return r;
}
// NaN in the place of what is not finite, which e4m3 holds as NaN (it has no infinity).
__device__ __forceinline__ float nan_or(float x) { return fabsf(x) <= 3.4028235e38f ? x : __int_as_float(0x7fffffff); }

// 32 bytes in one access where the address allows it (WIDE), else in two.
template <bool WIDE>
__device__ __forceinline__ void load32(const uint4* at, uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(at)
                 : "memory");
  } else {
    const uint4 a = __ldcs(at), b = __ldcs(at + 1);
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store32(uint4* at, const uint32_t (&w)[8]) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    __stcs(at, make_uint4(w[0], w[1], w[2], w[3]));
    __stcs(at + 1, make_uint4(w[4], w[5], w[6], w[7]));
  }
}

// (token, group) row `i` of a tensor of T << hs rows; eight lanes per row, c = channels 16 c .. + 15.
template <bool WIDE>
__global__ void __launch_bounds__(kThreads) append_kv_fp8_kernel(const __grid_constant__ QuantParams p) {
  const int x = blockIdx.y, c = threadIdx.x & 7;
  const int64_t rows = (int64_t)p.T << p.hs;
  const int64_t base = (int64_t)blockIdx.x * (kThreads / 8 * kUnroll) + (threadIdx.x >> 3);
  const uint16_t* src = p.src[x];
  uint32_t v[kUnroll][8];
  int32_t slot[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = base + u * (kThreads / 8), t = i >> p.hs;
    slot[u] = -1;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = 0;
    if (i < rows) {
      slot[u] = p.slots[t];
      load32<WIDE>(reinterpret_cast<const uint4*>(src + t * p.src_stride[x] + (i - (t << p.hs)) * 128) + 2 * c, v[u]);
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = base + u * (kThreads / 8);
    const uint32_t(&w)[8] = v[u];
    uint32_t m2 = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m2 = max_mag2(m2, w[k]);
    uint32_t m = max(m2 & 0xffffu, m2 >> 16);
    const bool odd = m >= 0x7f80u;  // an infinity or a NaN: it does not count
    if (odd) {
      m = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
        if (lo < 0x7f80u) m = max(m, lo);
        if (hi < 0x7f80u) m = max(m, hi);
      }
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    // |x| = f * 2^(E - 127), f in [1, 2), and 448 = 1.75 * 2^8: e + 127 = E - 8, one more if f > 1.75.
    // 246: rows beyond 1.75 * 2^127 are held at it, since 448 * 2^120 is no finite bf16.
    const int32_t b = min(max((int32_t)(m >> 7) - 8 + ((m & 0x7fu) > 0x60u ? 1 : 0), 0), 246);
    const float inv = __int_as_float((254 - b) << 23);
    uint32_t q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float f[4] = {bf16_lo(w[2 * k]) * inv, bf16_hi(w[2 * k]) * inv, bf16_lo(w[2 * k + 1]) * inv,
                    bf16_hi(w[2 * k + 1]) * inv};
      if (odd)
#pragma unroll
        for (int y = 0; y < 4; ++y) f[y] = nan_or(f[y]);
      q[k] = e4m3x2(f[0], f[1]) | (e4m3x2(f[2], f[3]) << 16);
    }
    if (slot[u] < 0) continue;
    if (slot[u] >= p.cells) {
      if (c == 0) msa_record_error(kErrBadPage);
      continue;
    }
    const int64_t g = i & (((int64_t)1 << p.hs) - 1);
    const int64_t cell = ((((int64_t)(slot[u] >> 7) << p.hs) + g) << 7) + (slot[u] & 127);
    reinterpret_cast<uint4*>(p.cache[x] + cell * 128)[c] = make_uint4(q[0], q[1], q[2], q[3]);
    if (c == 0) p.scale[x][cell] = (uint8_t)b;
  }
}

struct GatherParams {
  const uint8_t* cache[2];
  const uint8_t* scale[2];
  uint16_t* dst[2];  // [T, Hkv, 128] bf16
  const int32_t* slots;
  int32_t T, hs;
  int64_t cells;
};

template <bool WIDE>
__global__ void __launch_bounds__(kThreads) gather_kv_fp8_kernel(const __grid_constant__ GatherParams p) {
  const int x = blockIdx.y, c = threadIdx.x & 7;
  const int64_t rows = (int64_t)p.T << p.hs;
  const int64_t base = (int64_t)blockIdx.x * (kThreads / 8 * kUnroll) + (threadIdx.x >> 3);
  int32_t slot[kUnroll];
  uint4 v[kUnroll];
  uint32_t b[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = base + u * (kThreads / 8);
    slot[u] = i < rows ? p.slots[i >> p.hs] : -1;
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t i = base + u * (kThreads / 8);
    if (slot[u] >= p.cells) {
      if (c == 0) msa_record_error(kErrBadPage);
      slot[u] = -1;
    }
    if (slot[u] < 0) continue;
    const int64_t g = i & (((int64_t)1 << p.hs) - 1);
    const int64_t cell = ((((int64_t)(slot[u] >> 7) << p.hs) + g) << 7) + (slot[u] & 127);
    v[u] = __ldcs(reinterpret_cast<const uint4*>(p.cache[x] + cell * 128) + c);
    b[u] = p.scale[x][cell];
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    if (slot[u] < 0) continue;
    const int64_t i = base + u * (kThreads / 8);
    const float f = __int_as_float(b[u] ? b[u] << 23 : 0x400000);  // 2^(b - 127)
    const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
    uint32_t r[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t lo = f16x2_of_e4m3x2((uint16_t)w[k]), hi = f16x2_of_e4m3x2((uint16_t)(w[k] >> 16));
      r[2 * k] = pack_bf16x2(f16_lo(lo) * f, f16_hi(lo) * f);
      r[2 * k + 1] = pack_bf16x2(f16_lo(hi) * f, f16_hi(hi) * f);
    }
    store32<WIDE>(reinterpret_cast<uint4*>(p.dst[x] + i * 128) + 2 * c, r);
  }
}

int32_t log2_of(int32_t x) {
  int32_t s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

// K and V side by side.
template <class P>
cudaError_t launch_rows(void (*kernel)(P), const P& p, int64_t rows, cudaStream_t stream) {
  constexpr int64_t per = kThreads / 8 * kUnroll;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((rows + per - 1) / per), 2);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  // the launch's own status: the thread's last error may be an older call's
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace

cudaError_t launch_append_kv_fp8(const AppendFp8Args& a, cudaStream_t stream) {
  QuantParams p{};
  p.src[0] = a.k;
  p.src[1] = a.v;
  p.src_stride[0] = a.k_stride;
  p.src_stride[1] = a.v_stride;
  p.cache[0] = a.k_cache;
  p.cache[1] = a.v_cache;
  p.scale[0] = a.k_scale;
  p.scale[1] = a.v_scale;
  p.slots = a.slot_map;
  p.T = a.T;
  p.hs = log2_of(a.Hkv);
  p.cells = a.num_pages * MSA_BLOCK_TOKENS;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                         (uintptr_t)(a.k_stride * 2) | (uintptr_t)(a.v_stride * 2);
  return launch_rows((bits & 31) == 0 ? append_kv_fp8_kernel<true> : append_kv_fp8_kernel<false>, p,
                     (int64_t)a.T * a.Hkv, stream);
}

cudaError_t launch_gather_kv_fp8(const GatherFp8Args& a, cudaStream_t stream) {
  GatherParams p{};
  p.cache[0] = a.k_cache;
  p.cache[1] = a.v_cache;
  p.scale[0] = a.k_scale;
  p.scale[1] = a.v_scale;
  p.dst[0] = a.k;
  p.dst[1] = a.v;
  p.slots = a.slots;
  p.T = a.T;
  p.hs = log2_of(a.Hkv);
  p.cells = a.num_pages * MSA_BLOCK_TOKENS;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
  return launch_rows((bits & 31) == 0 ? gather_kv_fp8_kernel<true> : gather_kv_fp8_kernel<false>, p,
                     (int64_t)a.T * a.Hkv, stream);
}

}  // namespace msa
