// Host-side helpers shared by the launchers: TMA tensor-map encoding and SM count.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <mutex>

namespace msa {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, fetched once through the runtime (no libcuda link).
inline EncodeTiledFn encode_tiled_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// bf16 tensor map of `rank` dims (dims[0] innermost, strides in bytes for dims 1..rank-1),
// box `box` elements, 128-byte swizzle (box[0] * 2 must be 128) or none.
inline bool encode_bf16_map(CUtensorMap* map, const void* base, int rank, const uint64_t* dims,
                            const uint64_t* strides_bytes, const uint32_t* box, bool swizzle128) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t gdim[5], gstr[4];
  cuuint32_t bdim[5], estr[5];
  for (int i = 0; i < rank; ++i) {
    gdim[i] = dims[i];
    bdim[i] = box[i];
    estr[i] = 1;
  }
  for (int i = 0; i + 1 < rank; ++i) gstr[i] = strides_bytes[i];
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void*>(base),
                  gdim, gstr, bdim, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Map of `rows` rows of 128 bytes, box of `box_rows` of them, 128-byte swizzle.
inline bool encode_u8_rows_map(CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  const cuuint64_t gdim[2] = {128, rows}, gstr[1] = {128};
  const cuuint32_t bdim[2] = {128, box_rows}, estr[2] = {1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), gdim, gstr, bdim, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

inline int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0)
    return 148;
  return n;
}

// Raises a kernel's dynamic shared memory limit on the current device, once per device (the call
// takes several microseconds; `raised` is the kernel's own, zero-initialised, and `bytes` the same
// in every call for it).
constexpr int kMaxDevices = 64;
template <class K>
inline cudaError_t raise_smem_limit(K kernel, size_t bytes, std::atomic<size_t> (&raised)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < kMaxDevices && raised[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev < kMaxDevices) raised[dev].store(bytes, std::memory_order_relaxed);
  return e;
}
// Launches a kernel that takes up to `bytes` of dynamic shared memory: `launch` returns the launch's own
// status. A device reset unloads the kernel and its limit, which the record of it outlives; so a
// launch that fails with cudaErrorInvalidValue is made once more with the limit raised again, and
// only once: whatever it then returns is the answer. The error of a failed launch is taken off the
// thread, since the caller gets it as a status.
template <class K, class L>
inline cudaError_t launch_with_smem(K kernel, size_t bytes, std::atomic<size_t> (&raised)[kMaxDevices],
                                    L launch) {
  for (int attempt = 0;; ++attempt) {
    cudaError_t e = raise_smem_limit(kernel, bytes, raised);
    if (e == cudaSuccess) e = launch();
    if (e == cudaSuccess) return e;
    cudaGetLastError();
    int dev = 0;
    if (e != cudaErrorInvalidValue || attempt > 0 || cudaGetDevice(&dev) != cudaSuccess || dev >= kMaxDevices)
      return e;
    raised[dev].store(0, std::memory_order_relaxed);
  }
}

inline size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

}  // namespace msa
