// Host side of the eviction: the two launches.
#include "common.cuh"
#include "evict.cuh"
#include "internal.h"

namespace fa {

namespace {

template <int CS>
bool launch_select(const EvictParams& p, int pairs, cudaStream_t s) {
  auto kern = fa_evict_select_kernel<CS>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 51200 * 4) != cudaSuccess)
    return false;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(pairs * CS);
  cfg.blockDim = dim3(evict_threads(CS));
  cfg.dynamicSmemBytes = static_cast<size_t>(p.smem_keys) * 4;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CS;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, p) == cudaSuccess;
}

}  // namespace

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
  // CTAs per (sequence, head): one per 4,096 keys of the longest sequence that
  // the table allows (the lengths are not known here), up to the portable cluster
  // size, as long as there are no more CTAs than SMs.  Measured (cold): 32,768 keys, 8 pairs, one CTA
  // 29 us, eight 16; 12,032 keys, 128 pairs, one CTA 18 us, four 25.
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  int cs = 1;
  while (cs < kEvictCluster && cs * 4096ll < cap && 2ll * cs * a.B * a.Hkv <= sm_count())
    cs *= 2;
  // Keys of a CTA kept in shared memory (200 KB of them at most; longer shares
  // read their weights again in every pass).
  const long long share = ((cap + cs - 1) / cs + 31) / 32 * 32;
  p.smem_keys = static_cast<int>(share < 51200 ? share : 51200);
  const bool selected = cs == 1   ? launch_select<1>(p, a.B * a.Hkv, s)
                        : cs == 2 ? launch_select<2>(p, a.B * a.Hkv, s)
                        : cs == 4 ? launch_select<4>(p, a.B * a.Hkv, s)
                                  : launch_select<8>(p, a.B * a.Hkv, s);
  if (!selected) return FA_ERR_CUDA;
  const int rows = 4 * 256 / p.units;  // tokens per block of the move
  const int dst = a.dst_pages * a.page;
  const dim3 grid((dst + rows - 1) / rows, a.B * a.Hkv);
  const bool ok = p.units == 16 ? launch_after(fa_evict_move_kernel<16>, grid, dim3(256), s, p)
                                : launch_after(fa_evict_move_kernel<8>, grid, dim3(256), s, p);
  return ok ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
