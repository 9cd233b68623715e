// Shared host/device plumbing for the attention kernels: the device error
// word, TMA descriptor encoding and a small per-device property cache.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/fa.h"

namespace fa {

// One error word per translation unit (no relocatable device code).  A kernel
// that gives up a bounded wait stores the site id of that wait here; the host
// code of the same unit reads and clears it.
static __device__ unsigned int g_fa_err;

__device__ __forceinline__ unsigned int* fwd_error_word() { return &g_fa_err; }
__device__ __forceinline__ unsigned int* device_error_word() { return &g_fa_err; }

// Read and clear this unit's error word (synchronises the stream).
inline unsigned int read_and_clear_error(cudaStream_t s) {
  unsigned int v = 0, z = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess) return 0xFFFFFFFFu;
  if (cudaMemcpyFromSymbol(&v, g_fa_err, sizeof(v)) != cudaSuccess) return 0xFFFFFFFFu;
  if (v) cudaMemcpyToSymbol(g_fa_err, &z, sizeof(z));
  return v;
}

// ------------------------------------------------------------------ host side

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry point, so the
// library needs no link against libcuda.
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

// 4-D BSHD view [B, L, heads, D] of a contiguous 16-bit tensor, loaded as
// boxes of 64 head-dim elements x 128 sequence rows with 128-byte swizzle.
inline bool make_bshd_map(CUtensorMap* map, const void* ptr, int B, int L, int heads, int D,
                          bool bf16, int box_rows = 128) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)heads * D * 2,
                           (cuuint64_t)L * heads * D * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<void*>(ptr), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Same view for 8-bit E4M3 codes: dims {D, heads, L, B}, box {128, 1,
// box_rows, 1} (one 128-byte row per sequence position when D = 128).
inline bool make_bshd_map_e4m3(CUtensorMap* map, const void* ptr, int B, int L, int heads, int D,
                               int box_rows = 128) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)L, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)heads * D, (cuuint64_t)L * heads * D};
  cuuint32_t box[4] = {128, 1, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Packed-Q tensor map: dims {D, H, Lq, B}, box {64, g, Lq, 1}, so one load
// brings a K/V head's g query heads for all Lq queries, row = query * g + head.
inline bool make_group_map(CUtensorMap* map, const void* Q, int B, int Lq, int H, int g, int D, bool bf16) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)Lq, (cuuint64_t)B};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)Lq * H * D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)g, (cuuint32_t)Lq, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  4, const_cast<void*>(Q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// Launch with the programmatic-dependency attribute: the kernel may be placed
// while its predecessor still runs and waits for it with griddepcontrol.wait.
template <typename... A, typename... P>
inline bool launch_after_smem(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                              const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess;
}
template <typename... A, typename... P>
inline bool launch_after(void (*kern)(P...), dim3 grid, dim3 block, cudaStream_t s, const A&... args) {
  return launch_after_smem(kern, grid, block, 0, s, args...);
}

inline int sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

}  // namespace fa
