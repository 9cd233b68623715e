// Eviction from a paged cache by accumulated attention weight.
//
// Per sequence and K/V head: of n keys keep the first `sinks`, the last
// `recent`, and of those between the `need` = keep - sinks - recent heaviest,
// ties to the lower index; then move the survivors, in their order, into other
// pages.  Two kernels:
//   fa_evict_select_kernel  one cluster of 1 to 8 CTAs per (sequence, head), each
//     holding a contiguous share of the keys in shared memory.  The weights
//     become 32-bit keys that order like the floats; a radix select over
//     11 + 11 + 10 bits (each CTA's histogram, added up a slice per CTA through
//     the cluster's shared memory, then a scan for the bin that holds the
//     need-th largest) finds the threshold T and how many keys equal to T are
//     taken; then each warp counts and writes its contiguous share, so survivors
//     come out in ascending order with no sort.  Whole numbers only: exact.
//     Bound by latency: ten cluster barriers and the atomics of a few hot bins
//     (32,768 keys, 8 pairs: 16 us).
//   fa_evict_move_kernel    bound by the read and write of the survivors' K
//     and V: 16 bytes per thread and access, several rows in flight.
// Measured, both: 16 sequences of 3,000 to 12,000 keys, 8 heads of D 128, cut to
// 4,096: 114 us, 4.8 TB/s; one of 32,768 cut to 2,048: 19 us.
#pragma once

#include <cooperative_groups.h>

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
  int smem_keys;          // keys of a CTA that fit in shared memory
};

// Unsigned order of the floats: NaN above everything, -0 equal to 0.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (w != w) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Keys of sequence b.  new_lens may be lens itself: the selection, whose CTAs
// all read the length, leaves it alone; the move writes it, whose blocks need
// min(n, keep) only, which is the same before and after that write.
__device__ __forceinline__ int evict_len(const EvictParams& p, int b) {
  return static_cast<int>(
      min(static_cast<long long>(max(p.lens[b], 0)), static_cast<long long>(p.max_pages) * p.page));
}

constexpr int kEvictBins = 2048, kEvictCluster = 8;
constexpr int evict_threads(int cs) { return cs == 1 ? 1024 : 512; }

// Exclusive sum of v over the block's threads; the block's total in `total`.
template <int NT>
__device__ __forceinline__ uint32_t evict_scan(uint32_t v, uint32_t* warps, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t incl = v;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, h);
    if (lane >= h) incl += o;
  }
  __syncthreads();  // (warps may still be read from the last scan)
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  uint32_t before = incl - v;
  total = 0;
#pragma unroll
  for (int x = 0; x < NT / 32; ++x) {
    const uint32_t c = warps[x];
    if (x < warp) before += c;
    total += c;
  }
  return before;
}

template <int CS>
__global__ void __launch_bounds__(evict_threads(CS)) fa_evict_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  constexpr int NT = evict_threads(CS), NW = NT / 32;
  extern __shared__ uint32_t keys[];  // [smem_keys]
  __shared__ uint32_t hist[kEvictBins];
  __shared__ uint32_t warps[NW];
  __shared__ uint32_t slice[kEvictCluster];  // totals of the ranks' slices of bins
  __shared__ uint32_t found[2];              // bin, keys above it
  __shared__ uint32_t counts[kEvictCluster][2];  // sure, tied keys of each rank
  const int rank = CS == 1 ? 0 : static_cast<int>(cg::this_cluster().block_rank());
  auto sync = [&]() {
    if constexpr (CS == 1)
      __syncthreads();
    else
      cg::this_cluster().sync();
  };
  auto of_rank = [&](uint32_t* x, int r) -> uint32_t* {
    if constexpr (CS == 1)
      return x;
    else
      return cg::this_cluster().map_shared_rank(x, r);
  };
  pdl_launch_dependents();
  const int bh = blockIdx.x / CS, b = bh / p.Hkv;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int n = evict_len(p, b);
  int* kept = p.kept + static_cast<long long>(bh) * p.keep;
  if (n <= p.keep) {  // (the whole cluster)
    for (int i = rank * NT + t; i < p.keep; i += CS * NT) kept[i] = i < n ? i : -1;
    return;
  }
  const float* w = p.weights + bh * p.wstride;
  // This rank's keys [s0, s1), and the contested ones of them [lo, hi).
  const int share = ((n + CS - 1) / CS + 31) / 32 * 32;
  const int s0 = min(n, rank * share), s1 = min(n, s0 + share);
  const int lo = max(s0, p.sinks), hi = min(s1, n - p.recent);
  const bool fits = share <= p.smem_keys;
  auto key_at = [&](int j) -> uint32_t { return fits ? keys[j - s0] : evict_key(w[j]); };
  if (fits) {
    int j = s0 + t;
    for (; j + 3 * NT < s1; j += 4 * NT) {  // four reads under way
      const float a = w[j], b4 = w[j + NT], c = w[j + 2 * NT], d = w[j + 3 * NT];
      keys[j - s0] = evict_key(a);
      keys[j - s0 + NT] = evict_key(b4);
      keys[j - s0 + 2 * NT] = evict_key(c);
      keys[j - s0 + 3 * NT] = evict_key(d);
    }
    for (; j < s1; j += NT) keys[j - s0] = evict_key(w[j]);
  }
  uint32_t need = p.keep - p.sinks - p.recent;
  uint32_t prefix = 0, mask = 0;  // bits fixed so far
  const uint32_t want = need;
  constexpr int per_rank = kEvictBins / CS;  // bins of a slice; rank r sums bins from the top
  if (want > 0) {
    constexpr int shifts[3] = {21, 10, 0}, bits[3] = {11, 11, 10};
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      for (int i = t; i < kEvictBins; i += NT) hist[i] = 0;
      __syncthreads();
      const uint32_t bm = (1u << bits[pass]) - 1u;
      const int sh = shifts[pass];
      for (int j = lo + t; j < hi; j += NT) {
        const uint32_t k = key_at(j);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> sh) & bm], 1u);
      }
      sync();
      // Rank r owns the bins top - r * per_rank downwards; thread t owns `each`
      // consecutive ones of them, summed over the ranks' histograms.
      constexpr int each = per_rank > NT ? per_rank / NT : 1;
      const int first = kEvictBins - 1 - rank * per_rank - t * each;
      uint32_t c[each], mine = 0;
#pragma unroll
      for (int y = 0; y < each; ++y) c[y] = 0;
      if (t * each < per_rank) {
#pragma unroll
        for (int r = 0; r < CS; ++r)
#pragma unroll
          for (int y = 0; y < each; ++y) c[y] += of_rank(hist, r)[first - y];
#pragma unroll
        for (int y = 0; y < each; ++y) mine += c[y];
      }
      uint32_t total;
      uint32_t before = evict_scan<NT>(mine, warps, total);
      if (CS > 1) {
        if (t < CS) of_rank(slice, t)[rank] = total;
        sync();
      }
      // The slice, then the bin, in which the running count reaches `need`.
      for (int r = 0; r < rank; ++r) before += slice[r];
      if (t * each < per_rank && before < need && before + mine >= need) {
        int at = first;
#pragma unroll
        for (int y = 0; y + 1 < each; ++y)
          if (at == first - y && before + c[y] < need) {
            before += c[y];
            --at;
          }
        for (int r = 0; r < CS; ++r) {
          uint32_t* f = of_rank(found, r);
          f[0] = at;
          f[1] = before;
        }
      }
      sync();
      prefix |= found[0] << sh;
      mask |= bm << sh;
      need -= found[1];
    }
  } else {
    // (The counts below go to the other ranks' shared memory: all must have
    // begun.  Above, the first pass's barrier sees to that.)
    sync();
  }
  // Now prefix is the need-th largest key's value, and `need` of the keys
  // equal to it are taken (the first ones); want == 0 takes none.
  const int per = (s1 - s0 + NW * 32 - 1) / (NW * 32) * 32;
  const int w0 = min(s1, s0 + warp * per), w1 = min(s1, w0 + per);
  // 2: always taken, 1: equal to the threshold, 0: not taken
  auto cls = [&](int j) -> int {
    if (j < p.sinks || j >= n - p.recent) return 2;
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
  // Survivors and tied keys before this warp's: in the ranks before, in the
  // warps before (one scan for both: 16 bits would not do, so two).
  uint32_t all_sure, all_tied;
  uint32_t at = evict_scan<NT>(lane == 0 ? sure : 0u, warps, all_sure);
  uint32_t ties = evict_scan<NT>(lane == 0 ? tied : 0u, warps, all_tied);
  at = __shfl_sync(0xffffffffu, at, 0);
  ties = __shfl_sync(0xffffffffu, ties, 0);
  if (CS > 1) {
    if (t < CS) {
      of_rank(&counts[0][0], t)[2 * rank] = all_sure;
      of_rank(&counts[0][0], t)[2 * rank + 1] = all_tied;
    }
    sync();  // (the last access to another rank's shared memory is before it)
  }
  for (int r = 0; r < rank; ++r) {
    at += counts[r][0];
    ties += counts[r][1];
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
  const int m = min(evict_len(p, b), p.keep);
  if (blockIdx.x == 0 && h == 0 && threadIdx.x == 0) p.new_lens[b] = m;
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
