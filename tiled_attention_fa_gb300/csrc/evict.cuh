// Eviction from a paged cache by accumulated attention weight.
//
// Per sequence and K/V head: of n keys keep the first `sinks`, the last
// `recent`, and of those between the `need` = keep - sinks - recent heaviest,
// ties to the lower index; then move the survivors, in their order, into other
// pages.  Two kernels:
//   fa_evict_select_kernel  one CTA per (sequence, head).  The weights become
//     32-bit keys that order like the floats; a radix select over 11 + 11 + 10
//     bits (histogram, then a suffix scan for the bin that holds the need-th
//     largest) finds the threshold T and how many keys equal to T are taken;
//     then each warp counts and writes its contiguous share, so survivors come
//     out in ascending order with no sort.  Whole numbers only: exact.
//   fa_evict_move_kernel    bound by the read and write of the survivors' K
//     and V: 16 bytes per thread and access, several rows in flight.
#pragma once

#include <cstdint>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

struct EvictParams {
  const int* lens;        // [B]
  const float* weights;   // [B, Hkv, wstride]
  const int* table;       // [B, max_pages]
  const int* dst_table;   // [B, dst_pages]
  int* kept;              // [B, Hkv, keep]
  int* new_lens;          // [B]
  float* new_weights;     // [B, Hkv, dst_pages * page]
  uint4 *K, *V;           // pools
  long long wstride, k_page, v_page;  // page strides in 16-byte units
  int B, Hkv, units;      // units = D / 8 per row and head
  int page, max_pages, dst_pages, num_pages;
  int keep, sinks, recent;
  int smem_keys;          // keys that fit in shared memory
};

// Unsigned order of the floats: NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kEvictThreads = 1024, kEvictBins = 2048;

__global__ void __launch_bounds__(kEvictThreads) fa_evict_select_kernel(const EvictParams p) {
  constexpr int NT = kEvictThreads, NW = NT / 32;
  extern __shared__ uint32_t keys[];  // [smem_keys]
  __shared__ uint32_t hist[kEvictBins];
  __shared__ uint32_t wsum[NW], wsum2[NW];
  __shared__ uint32_t found[3];  // bin, count above it, count in it
  pdl_launch_dependents();
  const int bh = blockIdx.x, b = bh / p.Hkv;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int n = static_cast<int>(
      min(static_cast<long long>(max(p.lens[b], 0)), static_cast<long long>(p.max_pages) * p.page));
  int* kept = p.kept + static_cast<long long>(bh) * p.keep;
  if (t == 0 && bh - b * p.Hkv == 0) p.new_lens[b] = min(n, p.keep);
  if (n <= p.keep) {
    for (int i = t; i < p.keep; i += NT) kept[i] = i < n ? i : -1;
    return;
  }
  const float* w = p.weights + bh * p.wstride;
  const int lo = p.sinks, hi = n - p.recent;  // the contested keys (more of them than `need`)
  const bool fits = n <= p.smem_keys;
  auto key_at = [&](int j) -> uint32_t { return fits ? keys[j] : evict_key(w[j]); };
  if (fits)
    for (int j = t; j < n; j += NT) keys[j] = evict_key(w[j]);
  uint32_t need = p.keep - p.sinks - p.recent;
  uint32_t prefix = 0, mask = 0;  // bits fixed so far
  const uint32_t want = need;
  if (want > 0) {
    constexpr int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = t; i < kEvictBins; i += NT) hist[i] = 0;
      __syncthreads();
      const uint32_t bm = (1u << bits[pass]) - 1u;
      for (int j = lo + t; j < hi; j += NT) {
        const uint32_t k = key_at(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shifts[pass]) & bm], 1u);
      }
      __syncthreads();
      // Thread t owns bins top - 2t, top - 2t - 1 (from the heaviest down):
      // the bin in which the running count reaches `need`.
      const int b1 = kEvictBins - 1 - 2 * t, b0 = b1 - 1;
      const uint32_t c1 = hist[b1], c0 = hist[b0];
      uint32_t incl = c1 + c0;
#pragma unroll
      for (int h = 1; h < 32; h <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, h);
        if (lane >= h) incl += o;
      }
      if (lane == 31) wsum[warp] = incl;
      __syncthreads();
      uint32_t before = incl - c1 - c0;
      for (int x = 0; x < warp; ++x) before += wsum[x];
      if (before < need && before + c1 >= need) {
        found[0] = b1;
        found[1] = before;
      } else if (before + c1 < need && before + c1 + c0 >= need) {
        found[0] = b0;
        found[1] = before + c1;
      }
      __syncthreads();
      prefix |= found[0] << shifts[pass];
      mask |= bm << shifts[pass];
      need -= found[1];
      __syncthreads();
    }
  } else {
    __syncthreads();
  }
  // Now prefix is the need-th largest key's value, and `need` of the keys
  // equal to it are taken (the first ones); want == 0 takes none.
  const int per = (n + NW * 32 - 1) / (NW * 32) * 32;
  const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
  // 2: always taken, 1: equal to the threshold, 0: not taken
  auto cls = [&](int j) -> int {
    if (j < lo || j >= hi) return 2;
    if (want == 0) return 0;
    const uint32_t k = key_at(j);
    return k > prefix ? 2 : (k == prefix ? 1 : 0);
  };
  uint32_t sure = 0, tied = 0;
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int c = j0 + lane < w1 ? cls(j0 + lane) : 0;
    sure += __popc(__ballot_sync(0xffffffffu, c == 2));
    tied += __popc(__ballot_sync(0xffffffffu, c == 1));
  }
  if (lane == 0) {
    wsum[warp] = sure;
    wsum2[warp] = tied;
  }
  __syncthreads();
  uint32_t at = 0, ties = 0;  // survivors, tied keys of the warps before
  for (int x = 0; x < warp; ++x) {
    at += wsum[x];
    ties += wsum2[x];
  }
  at += min(ties, need);
  for (int j0 = w0; j0 < w1; j0 += 32) {
    const int j = j0 + lane;
    const int c = j < w1 ? cls(j) : 0;
    const uint32_t eq = __ballot_sync(0xffffffffu, c == 1), below = (1u << lane) - 1u;
    const bool take = c == 2 || (c == 1 && ties + __popc(eq & below) < need);
    const uint32_t all = __ballot_sync(0xffffffffu, take);
    if (take) kept[at + __popc(all & below)] = j;
    at += __popc(all);
    ties += __popc(eq);
  }
}

// Block (x, bh): rows of K and V of tokens [x * T, x * T + T) of the survivors,
// one 16-byte unit per thread and row; then their weights, and zeros behind.
template <int UNITS>
__global__ void __launch_bounds__(256) fa_evict_move_kernel(const EvictParams p) {
  constexpr int RPP = 256 / UNITS;  // rows a pass
  constexpr int PASSES = 4;
  pdl_wait();
  const int bh = blockIdx.y, b = bh / p.Hkv, h = bh - b * p.Hkv;
  const int m = p.new_lens[b];
  const int* kept = p.kept + static_cast<long long>(bh) * p.keep;
  const int u = threadIdx.x % UNITS, r0 = threadIdx.x / UNITS;
  const int t0 = blockIdx.x * RPP * PASSES;
  const long long row_units = static_cast<long long>(p.Hkv) * UNITS;
  uint4 kv[PASSES], vv[PASSES];
  long long kd[PASSES], vd[PASSES];
#pragma unroll
  for (int x = 0; x < PASSES; ++x) {
    const int t = t0 + x * RPP + r0;
    kd[x] = -1;
    kv[x] = vv[x] = make_uint4(0, 0, 0, 0);
    if (t < m) {
      const int src = kept[t];
      const int sp = p.table[static_cast<size_t>(b) * p.max_pages + src / p.page];
      const int dp = p.dst_table[static_cast<size_t>(b) * p.dst_pages + t / p.page];
      const long long so = static_cast<long long>(src % p.page) * row_units + h * UNITS + u;
      if (sp >= 0 && sp < p.num_pages) {
        kv[x] = __ldcs(p.K + sp * p.k_page + so);
        vv[x] = __ldcs(p.V + sp * p.v_page + so);
      }
      if (dp >= 0 && dp < p.num_pages) {
        const long long to = static_cast<long long>(t % p.page) * row_units + h * UNITS + u;
        kd[x] = dp * p.k_page + to;
        vd[x] = dp * p.v_page + to;
      }
    }
  }
#pragma unroll
  for (int x = 0; x < PASSES; ++x)
    if (kd[x] >= 0) {
      p.K[kd[x]] = kv[x];
      p.V[vd[x]] = vv[x];
    }
  const int cap = p.dst_pages * p.page;
  const float* w = p.weights + bh * p.wstride;
  for (int t = t0 + threadIdx.x; t < min(cap, t0 + RPP * PASSES); t += 256)
    p.new_weights[static_cast<long long>(bh) * cap + t] = t < m ? w[kept[t]] : 0.f;
}

}  // namespace fa
