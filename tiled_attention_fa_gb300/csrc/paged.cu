// Host side of the paged cache: the decode launches (parts, join, weights)
// and the write of new tokens.
#include <atomic>
#include <chrono>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "paged.cuh"

namespace fa {

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

// Query rows a thread processes for `rows` packed ones.
int rows_class(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128; }

struct WsPlan {
  size_t count, part_o, part_lse, scores, bytes;
};

WsPlan ws_plan(int B, int Lq, long long cap, int H, int Hkv, int D, bool weights, int sms) {
  const size_t rows = static_cast<size_t>(H / Hkv) * Lq;
  WsPlan w;
  if (sms < 1) sms = 1;
  w.count = 0;
  size_t at = align256(sizeof(unsigned long long) * sms);
  w.part_o = at;
  at += align256(2 * static_cast<size_t>(sms) * rows * D * sizeof(float));
  w.part_lse = at;
  at += align256(2 * static_cast<size_t>(sms) * rows * sizeof(float));
  w.scores = at;
  if (weights)
    at += static_cast<size_t>(B) * Hkv * ((cap + 127) / 128) * rows * 128 * sizeof(float);
  w.bytes = at;
  return w;
}

// A number no other call of this process has, and no memory is likely to hold:
// it marks the join's counters as this call's, so the workspace needs no
// initialisation (48 bits, not 0).
unsigned long long call_nonce() {
  static std::atomic<unsigned long long> next{[] {
    const unsigned long long t = std::chrono::steady_clock::now().time_since_epoch().count() ^
                                 std::chrono::system_clock::now().time_since_epoch().count() << 7 ^
                                 reinterpret_cast<uintptr_t>(&t) << 20;  // where this process's stack lies
    return t * 0x9E3779B97F4A7C15ull;
  }()};
  const unsigned long long n = next.fetch_add(1) & 0xFFFFFFFFFFFFull;
  return n ? n : next.fetch_add(1) & 0xFFFFFFFFFFFFull;
}

// K or V pool [pages, page, Hkv, D] with a free page stride, loaded as boxes
// of 64 head-dim elements x min(page, 128) rows of one page and head.
bool make_pool_map(CUtensorMap* map, const void* ptr, int pages, int page, int Hkv, int D,
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

template <int D, bool BF16, int R>
fa_status launch_decode(const PagedDecodeArgs& a, PagedParams& p, int G, cudaStream_t s) {
  using Ly = PagedLayout<D, R>;
  CUtensorMap tq, tk, tv;
  if (!make_group_map(&tq, a.Q, a.B, a.Lq, a.H, p.g, D, BF16) ||
      !make_pool_map(&tk, a.K, a.num_pages, a.page, a.Hkv, D, a.k_page_stride, BF16) ||
      !make_pool_map(&tv, a.V, a.num_pages, a.page, a.Hkv, D, a.v_page_stride, BF16))
    return FA_ERR_CUDA;
  auto kern = fa_paged_decode_kernel<D, BF16, R>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM_ALLOC) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  if (!launch_after_smem(kern, dim3(G), dim3(Ly::NTHREADS), Ly::SMEM_ALLOC, s, tq, tk, tv, p))
    return FA_ERR_CUDA;
  if (a.weights == nullptr) return FA_OK;
  return launch_after(fa_paged_weights_kernel, dim3((p.max_tiles + 7) / 8, a.B * a.Hkv), dim3(256), s, p, a.weights,
                      static_cast<long long>(a.weights_stride))
             ? FA_OK
             : FA_ERR_CUDA;
}

template <int D, bool BF16>
fa_status pick_rows(const PagedDecodeArgs& a, PagedParams& p, int G, cudaStream_t s) {
  switch (rows_class(p.rows)) {
    case 8: return launch_decode<D, BF16, 8>(a, p, G, s);
    case 16: return launch_decode<D, BF16, 16>(a, p, G, s);
    case 32: return launch_decode<D, BF16, 32>(a, p, G, s);
    case 64: return launch_decode<D, BF16, 64>(a, p, G, s);
    default: return launch_decode<D, BF16, 128>(a, p, G, s);
  }
}

}  // namespace

size_t paged_decode_workspace_size(int B, int Lq, long long cap, int H, int Hkv, int D, bool weights) {
  return ws_plan(B, Lq, cap, H, Hkv, D, weights, sm_count()).bytes;
}

fa_status run_paged_decode(const PagedDecodeArgs& a, cudaStream_t s) {
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const int sms = sm_count();
  const WsPlan w = ws_plan(a.B, a.Lq, cap, a.H, a.Hkv, a.D, a.weights != nullptr, sms);
  if (a.workspace_bytes < w.bytes) return FA_ERR_SCRATCH_TOO_SMALL;
  char* ws = static_cast<char*>(a.workspace);
  PagedParams p;
  p.table = a.table;
  p.lens = a.lens;
  p.O = a.O;
  p.LSE = a.LSE;
  p.count = reinterpret_cast<unsigned long long*>(ws + w.count);
  p.nonce = call_nonce();
  p.part_o = reinterpret_cast<float*>(ws + w.part_o);
  p.part_lse = reinterpret_cast<float*>(ws + w.part_lse);
  p.scores = a.weights != nullptr ? reinterpret_cast<float*>(ws + w.scores) : nullptr;
  p.B = a.B;
  p.Lq = a.Lq;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.g = a.H / a.Hkv;
  p.rows = p.g * a.Lq;
  p.ginv = 65536 / p.g + 1;
  p.page = a.page;
  p.max_pages = a.max_pages;
  p.cap = static_cast<int>(cap);
  p.max_tiles = static_cast<int>((cap + 127) / 128);
  p.window = a.window < p.cap ? a.window : 0;  // wider than the cache: every key
  p.sinks = p.window ? (a.sinks < p.cap ? a.sinks : p.cap) : 0;
  p.sl2 = 1.4426950408889634f / sqrtf(static_cast<float>(a.D));
  // Tiles an item visits at most: all of the table's, or with a window those that
  // Lq - 1 + window keys in a row touch and the sinks'.
  long long visit = p.max_tiles;
  if (p.window) {
    const long long reach = (static_cast<long long>(p.window) + a.Lq + 125) / 128 + 1 + (p.sinks + 127) / 128;
    if (reach < visit) visit = reach;
  }
  // One CTA per SM, fewer when even full sequences have fewer tiles.
  const long long most = static_cast<long long>(a.B) * a.Hkv * p.max_tiles;
  if (most >= (1ll << 31) || sms >= 65536) return FA_ERR_UNSUPPORTED;
  if (a.weights != nullptr && static_cast<long long>(a.B) * a.Hkv > 65535) return FA_ERR_UNSUPPORTED;
  int G = most < sms ? static_cast<int>(most) : sms;
  // Few items cut into many parts: whoever joins an item reads all its partials,
  // rows * D floats each at some 40 GB/s, while a tile takes some 2 us.  So at
  // most as many parts an item as make the sum of both smallest for an item of
  // `visit` tiles; a shorter one under a wide table is still cut into too many
  // (the host does not know the lengths).  All SMs and so, tables as wide as the
  // sequence: B1 H8/1 D128, 16 tokens, 20,000 keys 295 and 96 us; B2 H16/2, 4
  // tokens, 8,000 keys 64 and 39; B1 H4/1, a token, 30,000 keys 30 and 22.
  const double parts = std::ceil(std::sqrt(visit * 2.0 / (p.rows * a.D * 4 / 40e3)));
  const double limit = parts * a.B * a.Hkv;
  if (limit < G) G = static_cast<int>(limit);
  const bool bf16 = a.dtype == FA_BF16;
  if (a.D == 64) return bf16 ? pick_rows<64, true>(a, p, G, s) : pick_rows<64, false>(a, p, G, s);
  return bf16 ? pick_rows<128, true>(a, p, G, s) : pick_rows<128, false>(a, p, G, s);
}

fa_status run_paged_write(const void* K, const void* V, void* Kc, void* Vc, long long k_page,
                          long long v_page, const int* table, const int* start, const int* counts,
                          float* weights, long long wstride, const float* new_w, int B, int L,
                          int Hkv, int D, int page, int max_pages, int num_pages, cudaStream_t s) {
  const long long units = static_cast<long long>(B) * L * Hkv * (D / 8);
  const long long blocks = (units + 255) / 256;
  const long long most = 16ll * sm_count();
  fa_paged_write_kernel<<<static_cast<unsigned>(blocks < most ? blocks : most), 256, 0, s>>>(
      static_cast<const uint4*>(K), static_cast<const uint4*>(V), static_cast<uint4*>(Kc),
      static_cast<uint4*>(Vc), k_page / 8, v_page / 8, table, start, counts, weights, wstride, new_w,
      B, L, Hkv, D / 8, page, max_pages, num_pages);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

unsigned int paged_read_error(cudaStream_t s) { return read_and_clear_error(s); }

}  // namespace fa
