// Host side of the eviction: the two launches.
#include "common.cuh"
#include "evict.cuh"
#include "internal.h"

namespace fa {

fa_status run_paged_evict(const PagedEvictArgs& a, cudaStream_t s) {
  EvictParams p;
  p.lens = a.lens;
  p.weights = a.weights;
  p.table = a.table;
  p.dst_table = a.dst_table;
  p.kept = a.kept;
  p.new_lens = a.new_lens;
  p.new_weights = a.new_weights;
  p.K = static_cast<uint4*>(a.K);
  p.V = static_cast<uint4*>(a.V);
  p.wstride = a.weights_stride;
  p.k_page = a.k_page_stride / 8;
  p.v_page = a.v_page_stride / 8;
  p.B = a.B;
  p.Hkv = a.Hkv;
  p.units = a.D / 8;
  p.page = a.page;
  p.max_pages = a.max_pages;
  p.dst_pages = a.dst_pages;
  p.num_pages = a.num_pages;
  p.keep = a.keep;
  p.sinks = a.sinks;
  p.recent = a.recent;
  // Keys kept in shared memory (200 KB of them at most; longer sequences read
  // their weights again in every pass).
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  p.smem_keys = static_cast<int>(cap < 51200 ? cap : 51200);
  const size_t smem = static_cast<size_t>(p.smem_keys) * 4;
  if (cudaFuncSetAttribute(fa_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           51200 * 4) != cudaSuccess)
    return FA_ERR_CUDA;
  fa_evict_select_kernel<<<a.B * a.Hkv, kEvictThreads, smem, s>>>(p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  const int rows = 4 * 256 / p.units;  // tokens per block of the move
  const int dst = a.dst_pages * a.page;
  const dim3 grid((dst + rows - 1) / rows, a.B * a.Hkv);
  const bool ok = p.units == 16 ? launch_after(fa_evict_move_kernel<16>, grid, dim3(256), s, p)
                                : launch_after(fa_evict_move_kernel<8>, grid, dim3(256), s, p);
  return ok ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
