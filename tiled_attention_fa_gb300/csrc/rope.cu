// Host side of the rotary positions and of the append to the paged cache.
#include "common.cuh"
#include "internal.h"
#include "rope.cuh"

namespace fa {

namespace {

template <typename T, int UN, bool APPEND>
fa_status launch(RopeParams& p, bool neighbours, cudaStream_t s) {
  constexpr int ROWS = 256 / UN;
  const int all = p.H + (APPEND ? 2 : 1) * p.Hkv;
  const long long tokens = static_cast<long long>(p.B) * p.L;
  // Threads that share a token's unit: as few as leave each at most 12 heads (B4
  // L4096 H32/8 D128 both directions 108 us, with at most 6 heads 116), more while
  // the GPU is not full.
  const long long full = 1024ll * sm_count();
  int hs_log = 0;
  while ((2 << hs_log) <= ROWS && (1 << hs_log) < all &&
         ((all >> hs_log) > 12 || (tokens * UN << hs_log) < full))
    ++hs_log;
  p.hs_log = hs_log;
  const unsigned grid = static_cast<unsigned>((tokens + (ROWS >> hs_log) - 1) / (ROWS >> hs_log));
  return launch_after(neighbours ? fa_rope_kernel<T, UN, true, APPEND> : fa_rope_kernel<T, UN, false, APPEND>,
                      dim3(grid), dim3(256), s, p)
             ? FA_OK
             : FA_ERR_CUDA;
}

template <bool APPEND>
fa_status pick(RopeParams& p, const RopeArgs& a, cudaStream_t s) {
  const bool nb = a.neighbours != 0;
  if (a.dtype == FA_BF16)
    return a.D == 64 ? launch<__nv_bfloat16, 4, APPEND>(p, nb, s) : launch<__nv_bfloat16, 8, APPEND>(p, nb, s);
  return a.D == 64 ? launch<__half, 4, APPEND>(p, nb, s) : launch<__half, 8, APPEND>(p, nb, s);
}

RopeTensor tensor(const RopeView& x, const RopeView& y) {
  return {static_cast<const uint4*>(x.p), static_cast<uint4*>(const_cast<void*>(y.p)), x.batch / 8, x.token / 8,
          y.batch / 8, y.token / 8};
}

RopeParams params(const RopeArgs& a) {
  RopeParams p = {};
  p.q = tensor(a.q, a.qy);
  p.k = tensor(a.k, a.ky);
  p.table = static_cast<const longlong2*>(a.table);
  p.pos = a.positions;
  p.axes = a.axes;
  p.B = a.B;
  p.L = a.L;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.nrot = a.rotary / 16;
  p.back = a.back;
  return p;
}

}  // namespace

fa_status run_rope(const RopeArgs& a, cudaStream_t s) {
  RopeParams p = params(a);
  return pick<false>(p, a, s);
}

fa_status run_paged_append(const RopeArgs& a, const PagedAppendArgs& c, cudaStream_t s) {
  RopeParams p = params(a);
  p.k.y = static_cast<uint4*>(c.K_pool);
  p.v = {static_cast<const uint4*>(c.v.p), static_cast<uint4*>(c.V_pool), c.v.batch / 8, c.v.token / 8, 0, 0};
  p.block_table = c.table;
  p.start = c.start;
  p.counts = c.counts;
  p.k_page = c.k_page_stride / 8;
  p.v_page = c.v_page_stride / 8;
  p.weights = c.weights;
  p.new_w = c.new_weights;
  p.wstride = c.weights_stride;
  p.page_log = 31 - __builtin_clz(static_cast<unsigned>(c.page));
  p.max_pages = c.max_pages;
  p.num_pages = c.num_pages;
  return pick<true>(p, a, s);
}

}  // namespace fa
