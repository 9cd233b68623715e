// Host side of the attention behind shared prefixes: workspace and launches.
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged_launch.cuh"  // make_pool_map
#include "prefix.cuh"

namespace fa {

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

struct PrefixPlan {
  int mt;            // tiles of an item
  int tok;           // tokens of a tile
  long long items, units;  // at most
  int G;             // CTAs
  size_t own, own_o, own_lse, base, part_o, part_lse, bytes;
};

PrefixPlan prefix_plan_of(const PrefixDecodeArgs& a) {
  PrefixPlan w;
  const int g = a.H / a.Hkv;
  int sms = sm_count();
  if (sms < 1) sms = 1;
  w.tok = 128 / g;
  const long long tokens = static_cast<long long>(a.B) * a.Lq;
  // Groups of one tile (in the mean) have a CTA's two softmax groups share it.
  w.mt = tokens <= static_cast<long long>(w.tok) * a.groups ? 1 : 2;
  const long long per = static_cast<long long>(w.tok) * w.mt;
  const long long cap = static_cast<long long>(a.prefix_pages) * a.page;
  w.items = a.Hkv * (tokens / per + a.groups);
  w.units = w.items * ((cap + 127) / 128);
  w.G = w.units < sms ? static_cast<int>(w.units) : sms;
  const size_t rows = static_cast<size_t>(tokens) * a.H, chunks = static_cast<size_t>(w.items + w.G) * w.mt;
  size_t at = 0;
  w.own = at;
  at += align256(paged_decode_workspace_size(a.B, a.Lq, static_cast<long long>(a.max_pages) * a.page, a.H, a.Hkv,
                                             a.D, false));
  w.own_o = at;
  at += align256(rows * a.D * sizeof(float));
  w.own_lse = at;
  at += align256(rows * sizeof(float));
  w.base = at;
  at += align256((2 * static_cast<size_t>(a.groups) + 1) * sizeof(int));
  w.part_o = at;
  at += chunks * 128 * a.D * sizeof(float);
  w.part_lse = at;
  at += chunks * 128 * sizeof(float);
  w.bytes = at;
  return w;
}

// Q as [B * Lq, H, D], loaded as boxes of 64 head-dim elements x g heads x the
// tokens of a tile: row = token * g + head.
bool make_rows_map(CUtensorMap* map, const void* Q, long long tokens, int H, int g, int tok, int D, bool bf16) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)tokens, 1};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)H * D * 2, (cuuint64_t)tokens * H * D * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)g, (cuuint32_t)tok, 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(Q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool BF16, int MT>
fa_status launch_prefix(const PrefixDecodeArgs& a, const PrefixPlan& w, cudaStream_t s) {
  using Ly = PrefixLayout<D, MT>;
  char* ws = static_cast<char*>(a.workspace);
  PrefixJoinParams j;
  PrefixParams& p = j.p;
  p.table = a.prefix_table;
  p.lens = a.prefix_lens;
  p.starts = a.group_starts;
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  p.base = reinterpret_cast<int*>(ws + w.base);
  p.B = a.B;
  p.Lq = a.Lq;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.g = a.H / a.Hkv;
  p.groups = a.groups;
  p.tok = w.tok;
  p.max_items = static_cast<int>(w.items);
  p.ginv = 65536 / p.g + 1;
  p.page = a.page;
  p.max_pages = a.prefix_pages;
  p.cap = a.prefix_pages * a.page;
  p.sl2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  CUtensorMap tq, tk, tv;
  if (!make_rows_map(&tq, a.Q, static_cast<long long>(a.B) * a.Lq, a.H, p.g, p.tok, D, BF16) ||
      !make_pool_map(&tk, a.K, a.num_pages, a.page, a.Hkv, D, a.k_page_stride, BF16) ||
      !make_pool_map(&tv, a.V, a.num_pages, a.page, a.Hkv, D, a.v_page_stride, BF16))
    return FA_ERR_CUDA;
  auto kern = fa_prefix_kernel<D, BF16, MT>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM_ALLOC) != cudaSuccess)
    return FA_ERR_CUDA;
  if (!launch_after_smem(kern, dim3(w.G), dim3(Ly::NTHREADS), Ly::SMEM_ALLOC, s, tq, tk, tv, p))
    return FA_ERR_CUDA;
  // The sequences' own keys, in fp32.
  PagedDecodeArgs o;
  o.Q = a.Q;
  o.K = a.K;
  o.V = a.V;
  o.table = a.table;
  o.lens = a.lens;
  o.O = ws + w.own_o;
  o.LSE = reinterpret_cast<float*>(ws + w.own_lse);
  o.weights = nullptr;
  o.weights_stride = 0;
  o.k_page_stride = a.k_page_stride;
  o.v_page_stride = a.v_page_stride;
  o.workspace = ws + w.own;
  o.workspace_bytes = w.own_o - w.own;
  o.B = a.B;
  o.Lq = a.Lq;
  o.H = a.H;
  o.Hkv = a.Hkv;
  o.D = a.D;
  o.page = a.page;
  o.max_pages = a.max_pages;
  o.num_pages = a.num_pages;
  o.window = 0;
  o.sinks = 0;
  o.dtype = a.dtype;
  const fa_status st = run_paged_own(o, s);
  if (st != FA_OK) return st;
  j.own_lens = a.lens;
  j.own_o = static_cast<const float*>(o.O);
  j.own_lse = o.LSE;
  j.O = a.O;
  j.LSE = a.LSE;
  j.own_cap = a.max_pages * a.page;
  j.G = w.G;
  const int per = p.g * (D / 8), ppb = per <= 256 ? 256 / per : 1;
  const long long pairs = static_cast<long long>(a.B) * a.Lq * a.Hkv;
  return launch_after(fa_prefix_join_kernel<D, BF16, MT>, dim3(static_cast<unsigned>((pairs + ppb - 1) / ppb)),
                      dim3(256), s, j)
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool BF16>
fa_status pick_tiles(const PrefixDecodeArgs& a, const PrefixPlan& w, cudaStream_t s) {
  return w.mt == 1 ? launch_prefix<D, BF16, 1>(a, w, s) : launch_prefix<D, BF16, 2>(a, w, s);
}

}  // namespace

size_t paged_prefix_workspace_size(const PrefixDecodeArgs& a) { return prefix_plan_of(a).bytes; }

fa_status run_paged_prefix(const PrefixDecodeArgs& a, cudaStream_t s) {
  const PrefixPlan w = prefix_plan_of(a);
  if (w.units >= (1ll << 31) || w.items >= (1ll << 30)) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(a.B) * a.Hkv * ((static_cast<long long>(a.max_pages) * a.page + 127) / 128) >= (1ll << 31))
    return FA_ERR_UNSUPPORTED;
  if (a.workspace_bytes < w.bytes) return FA_ERR_SCRATCH_TOO_SMALL;
  const bool bf16 = a.dtype == FA_BF16;
  if (a.D == 64) return bf16 ? pick_tiles<64, true>(a, w, s) : pick_tiles<64, false>(a, w, s);
  return bf16 ? pick_tiles<128, true>(a, w, s) : pick_tiles<128, false>(a, w, s);
}

unsigned int prefix_read_error(cudaStream_t s) { return read_and_clear_error(s); }

}  // namespace fa
