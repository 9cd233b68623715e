// Host side of the attention behind shared prefixes: workspace and launches.
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "prefix.cuh"

namespace fa {

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// launch_after_smem in clusters of two along x, of which grid.x is a multiple.
template <typename... A, typename... P>
bool launch_pairs_after(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, static_cast<P>(args)...) == cudaSuccess;
}

struct PrefixPlan {
  int tok, rows;          // tokens of a prefix's tile, rows of a sequence's
  long long items, own;   // at most: items of prefixes, of sequences
  long long most;         // at most: the weight of all items' units
  int G;                  // CTAs
  size_t part_o, part_lse, own_o, own_lse, ends, bytes;
};

PrefixPlan prefix_plan_of(const PrefixDecodeArgs& a) {
  PrefixPlan w;
  const int g = a.H / a.Hkv;
  int sms = sm_count();
  if (sms < 1) sms = 1;
  w.tok = 128 / g;
  w.rows = g * a.Lq;
  const long long tokens = static_cast<long long>(a.B) * a.Lq;
  w.items = a.Hkv * (tokens / (2 * w.tok) + a.groups);
  w.own = static_cast<long long>(a.B) * a.Hkv;
  const long long prefix_units = w.items * ((static_cast<long long>(a.prefix_pages) * a.page + 127) / 128);
  const long long own_units = w.own * ((static_cast<long long>(a.max_pages) * a.page + 127) / 128);
  w.most = prefix_units * prefix_pair_weight(a.D) + own_units * kOneWeight;
  // (in pairs: prefixes and own keys may have CTAs of their own)
  w.G = prefix_units + own_units < sms ? static_cast<int>(prefix_units + own_units) : sms;
  w.G = w.G < 2 ? 2 : (w.G + 1) / 2 * 2;
  // Prefix partials: every query row once, and an item's 256 for every part.
  const size_t rows = static_cast<size_t>(tokens) * a.H + 256 * static_cast<size_t>(w.G);
  size_t at = 0;
  w.part_o = at;
  at += align256(rows * a.D * sizeof(float));
  w.part_lse = at;
  at += align256(rows * sizeof(float));
  w.own_o = at;
  at += align256(static_cast<size_t>(w.own + w.G) * w.rows * a.D * sizeof(float));
  w.own_lse = at;
  at += align256(static_cast<size_t>(w.own + w.G) * w.rows * sizeof(float));
  w.ends = at;
  at += static_cast<size_t>(w.items + w.own) * 2 * sizeof(int);
  w.bytes = at;
  return w;
}

// K or V pool [pages, page, Hkv, D] with a free page stride, loaded as boxes of
// 64 head-dim elements x min(page, 64) rows of one page and head.  The L2 fetches
// what a head's row holds: 128 bytes at D = 64, where 256 would bring its
// neighbour's row too, which another CTA reads at another time.
bool make_pool_map(CUtensorMap* map, const void* ptr, int pages, int page, int Hkv, int D, long long page_stride,
                   bool bf16) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hkv, (cuuint64_t)page, (cuuint64_t)pages};
  cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)Hkv * D * 2, (cuuint64_t)page_stride * 2};
  cuuint32_t box[4] = {64, 1, (cuuint32_t)(page < 1 << kOwnBoxLog ? page : 1 << kOwnBoxLog), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
            const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
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

template <int D, bool BF16, int R>
fa_status launch_prefix(const PrefixDecodeArgs& a, const PrefixPlan& w, PrefixJoinParams& j, cudaStream_t s) {
  using Sh = PrefixShared<D, R>;
  PrefixParams& p = j.p;
  p.entries = R == 0 ? a.groups + a.B : a.groups;
  PagedOwnParams o = {};
  o.table = a.table;
  o.lens = a.lens;
  o.part_o = p.own_o;
  o.part_lse = p.own_lse;
  o.ends = p.ends + 2 * w.items;
  o.B = a.B;
  o.Lq = a.Lq;
  o.H = a.H;
  o.Hkv = a.Hkv;
  o.g = p.g;
  o.rows = p.rows;
  o.ginv = p.ginv;
  o.page = a.page;
  o.max_pages = a.max_pages;
  o.cap = p.cap;
  o.max_tiles = (p.cap + 127) / 128;
  o.sl2 = p.sl2;
  CUtensorMap tq, to, tk, tv;
  if (!make_rows_map(&tq, a.Q, static_cast<long long>(a.B) * a.Lq, a.H, p.g, p.tok, D, BF16) ||
      !make_group_map(&to, a.Q, a.B, a.Lq, a.H, p.g, D, BF16) ||
      !make_pool_map(&tk, a.K, a.num_pages, a.page, a.Hkv, D, a.k_page_stride, BF16) ||
      !make_pool_map(&tv, a.V, a.num_pages, a.page, a.Hkv, D, a.v_page_stride, BF16))
    return FA_ERR_CUDA;
  auto kern = fa_prefix_kernel<D, BF16, R>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::ALLOC) != cudaSuccess)
    return FA_ERR_CUDA;
  // The kernel moves registers between its warpgroups; the budgets add up only when
  // every thread starts with REGS.  Any other allocation would leave an increase
  // waiting for registers that never come back, so refuse to launch instead.
  static int num_regs = -1;
  static std::once_flag once;
  std::call_once(once, [&] {
    cudaFuncAttributes at;
    if (cudaFuncGetAttributes(&at, kern) == cudaSuccess) num_regs = at.numRegs;
  });
  if (num_regs != PrefixLayout<D>::REGS) return FA_ERR_UNSUPPORTED;
  // Clusters of two, whose CTAs lie on one TPC and have the same role.  Placed one by one
  // as SMs fall free, 256 sequences behind 16,384 keys took 123 us instead of 97 (why two
  // roles on a TPC slow one another down was not measured); launched when all before is
  // done, the CTAs lie in order by themselves, but a call starts 2 to 3 us later.
  if (!launch_pairs_after(kern, dim3(w.G), dim3(Sh::NTHREADS), Sh::ALLOC, s, tq, to, tk, tv, p, o)) return FA_ERR_CUDA;
  // Parts of a prefix's item in the mean: with more than 8, four threads share them.
  const int cells = p.g * (D / 4), sp = w.G > 8 * w.items ? 4 : 1;
  const dim3 grid(static_cast<unsigned>(a.B) * a.Lq * a.Hkv, (cells * sp + 127) / 128);
  return (sp == 1 ? launch_after(fa_prefix_join_kernel<D, BF16, 1>, grid, dim3(128), s, j)
                  : launch_after(fa_prefix_join_kernel<D, BF16, 4>, grid, dim3(128), s, j))
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool BF16>
fa_status pick_rows(const PrefixDecodeArgs& a, const PrefixPlan& w, cudaStream_t s) {
  char* ws = static_cast<char*>(a.workspace);
  PrefixJoinParams j;
  PrefixParams& p = j.p;
  p.ptable = a.prefix_table;
  p.plens = a.prefix_lens;
  p.starts = a.group_starts;
  p.table = a.table;
  p.lens = a.lens;
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  p.own_o = reinterpret_cast<float*>(ws + w.own_o);
  p.own_lse = reinterpret_cast<float*>(ws + w.own_lse);
  p.ends = reinterpret_cast<int*>(ws + w.ends);
  p.most = static_cast<uint32_t>(w.most);
  p.B = a.B;
  p.Lq = a.Lq;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.g = a.H / a.Hkv;
  p.groups = a.groups;
  p.rows = w.rows;
  p.tok = w.tok;
  p.items = static_cast<int>(w.items);
  p.ginv = 65536 / p.g + 1;
  p.page = a.page;
  p.prefix_pages = a.prefix_pages;
  p.max_pages = a.max_pages;
  p.pcap = a.prefix_pages * a.page;
  p.cap = a.max_pages * a.page;
  p.sl2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  p.pair_weight = prefix_pair_weight(a.D);
  p.own_weight = prefix_own_weight(a.D);
  j.O = a.O;
  j.LSE = a.LSE;
  j.G = w.G;
  if (w.rows <= 8) return launch_prefix<D, BF16, 8>(a, w, j, s);
  if (w.rows <= 16) return launch_prefix<D, BF16, 16>(a, w, j, s);
  if (w.rows <= 32) return launch_prefix<D, BF16, 32>(a, w, j, s);
  return launch_prefix<D, BF16, 0>(a, w, j, s);
}

}  // namespace

size_t paged_prefix_workspace_size(const PrefixDecodeArgs& a) { return prefix_plan_of(a).bytes; }

fa_status run_paged_prefix(const PrefixDecodeArgs& a, cudaStream_t s) {
  const PrefixPlan w = prefix_plan_of(a);
  if (w.most >= (1ll << 32) || w.items + w.own >= (1ll << 29)) return FA_ERR_UNSUPPORTED;
  if (a.workspace_bytes < w.bytes) return FA_ERR_SCRATCH_TOO_SMALL;
  const bool bf16 = a.dtype == FA_BF16;
  if (a.D == 64) return bf16 ? pick_rows<64, true>(a, w, s) : pick_rows<64, false>(a, w, s);
  return bf16 ? pick_rows<128, true>(a, w, s) : pick_rows<128, false>(a, w, s);
}

unsigned int prefix_read_error(cudaStream_t s) { return read_and_clear_error(s); }

}  // namespace fa
