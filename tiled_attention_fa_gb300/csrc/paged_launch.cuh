// Launches of the paged decode kernel, for the two units that hold its forms.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace fa {

// The launch's parameters and its number of CTAs (paged.cu).
fa_status paged_setup(const PagedDecodeArgs& a, PagedParams& p, int& G);

// Query rows a thread processes for `rows` packed ones.
inline int rows_class(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

// K or V pool [pages, page, Hkv, D] with a free page stride, loaded as boxes
// of 64 head-dim elements x min(page, 128) rows of one page and head.
inline bool make_pool_map(CUtensorMap* map, const void* ptr, int pages, int page, int Hkv, int D,
                   long long page_stride, bool bf16) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)page, (cuuint64_t)pages};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)page_stride * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)(page < 128 ? page : 128), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, int R, bool OWN>
fa_status launch_decode(const PagedDecodeArgs& a, PagedParams& p, int G, cudaStream_t s) {
  using Ly = PagedLayout<D, R>;
  CUtensorMap tq, tk, tv;
  if (!make_group_map(&tq, a.Q, a.B, a.Lq, a.H, p.g, D, BF16) ||
      !make_pool_map(&tk, a.K, a.num_pages, a.page, a.Hkv, D, a.k_page_stride, BF16) ||
      !make_pool_map(&tv, a.V, a.num_pages, a.page, a.Hkv, D, a.v_page_stride, BF16))
    return FA_ERR_CUDA;
  auto kern = fa_paged_decode_kernel<D, BF16, R, OWN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM_ALLOC) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  if (!launch_after_smem(kern, dim3(G), dim3(Ly::NTHREADS), Ly::SMEM_ALLOC, s, tq, tk, tv, p))
    return FA_ERR_CUDA;
  if (OWN || a.weights == nullptr) return FA_OK;
  return launch_after(fa_paged_weights_kernel, dim3((p.max_tiles + 7) / 8, a.B * a.Hkv), dim3(256), s, p, a.weights,
                      static_cast<long long>(a.weights_stride))
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool BF16, bool OWN>
fa_status pick_rows(const PagedDecodeArgs& a, PagedParams& p, int G, cudaStream_t s) {
  switch (rows_class(p.rows)) {
    case 8: return launch_decode<D, BF16, 8, OWN>(a, p, G, s);
    case 16: return launch_decode<D, BF16, 16, OWN>(a, p, G, s);
    case 32: return launch_decode<D, BF16, 32, OWN>(a, p, G, s);
    case 64: return launch_decode<D, BF16, 64, OWN>(a, p, G, s);
    default: return launch_decode<D, BF16, 128, OWN>(a, p, G, s);
  }
}

template <bool OWN>
fa_status launch_paged(const PagedDecodeArgs& a, PagedParams& p, int G, cudaStream_t s) {
  const bool bf16 = a.dtype == FA_BF16;
  if (a.D == 64)
    return bf16 ? pick_rows<64, true, OWN>(a, p, G, s) : pick_rows<64, false, OWN>(a, p, G, s);
  return bf16 ? pick_rows<128, true, OWN>(a, p, G, s) : pick_rows<128, false, OWN>(a, p, G, s);
}

}  // namespace fa
