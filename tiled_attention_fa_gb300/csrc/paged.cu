// Host side of the paged cache: the decode launches (parts, join, weights)
// and the write of new tokens.
#include <atomic>
#include <chrono>
#include <cmath>

#include "common.cuh"
#include "internal.h"
#include "paged_launch.cuh"

namespace fa {

namespace {

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

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

}  // namespace

size_t paged_decode_workspace_size(int B, int Lq, long long cap, int H, int Hkv, int D, bool weights) {
  return ws_plan(B, Lq, cap, H, Hkv, D, weights, sm_count()).bytes;
}

fa_status paged_setup(const PagedDecodeArgs& a, PagedParams& p, int& G) {
  const long long cap = static_cast<long long>(a.max_pages) * a.page;
  const int sms = sm_count();
  const WsPlan w = ws_plan(a.B, a.Lq, cap, a.H, a.Hkv, a.D, a.weights != nullptr, sms);
  if (a.workspace_bytes < w.bytes) return FA_ERR_SCRATCH_TOO_SMALL;
  char* ws = static_cast<char*>(a.workspace);
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
  G = most < sms ? static_cast<int>(most) : sms;
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
  return FA_OK;
}

fa_status run_paged_decode(const PagedDecodeArgs& a, cudaStream_t s) {
  PagedParams p;
  int G = 0;
  const fa_status st = paged_setup(a, p, G);
  return st == FA_OK ? launch_paged<false>(a, p, G, s) : st;
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
