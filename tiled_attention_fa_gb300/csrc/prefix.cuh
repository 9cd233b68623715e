// Attention of a batch's new tokens over key/value prefixes that several of its
// sequences share, and the join with their attention over their own keys.
//
// Mathematics: softmax over the union of two sets of keys from the softmaxes of
// both: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.  Every new
// token behind a prefix sees all of it, so the prefix's part is one product
// chain of all rows (tokens x query heads of a K/V head) with the prefix's keys
// and values, which are read once, not once per sequence.
//
// Three launches.  fa_prefix_kernel: the prefixes' part, cut into partials.  The
// paged decode kernel (its OWN form) over the sequences' own keys: it may start
// as soon as SMs are free of the first.  fa_prefix_join_kernel: each row's
// partials of both.
//
// fa_prefix_kernel.  A tile is up to 128 rows: 128 / g tokens (g query heads a
// K/V head) of one group, row = token * g + head.  An item is one K/V head of a
// group and MT tiles (2, or 1 where a group has few rows); its units are the
// prefix's 128-key tiles.  The units of all items form one list and each CTA
// takes one of G equal contiguous parts of it, so all SMs work whatever the
// lengths and groups are.  A part's share of an item (a chunk) gives one
// normalised fp32 partial and its LSE.  Chunks number item + part, which no two
// share: the next chunk in the list is of the next item, the next part, or both.
//   warps 0-3, 4-7  softmax, a thread per row.  MT = 2: of tile 0 and tile 1.
//                   MT = 1: of the one tile's even and odd steps, each with a
//                   maximum, a sum and an O of its own, joined at the end.
//   warp 8          TMA: Q, then K_0, V_0, K_1, V_1, ... through one ring across
//                   chunks; lane i loads the i-th page of a tile
//   warp 9          TMEM, MMAs: S_t = Q_t K_j^T, P over S as 16 bits, O_t += P V_j
// Per 64 KB of K and V (D = 128) a CTA with 256 rows needs the tensor cores for
// 2,150 cycles and the exponentials for 2,050; its share of the memory bandwidth
// takes 2,790.  So up to 256 rows the read of the prefix bounds the kernel,
// above it the products do and the other row tiles' reads hit the L2.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "fwd.cuh"  // pack2
#include "ptx.cuh"

namespace fa {

struct PrefixParams {
  const int* table;   // [groups, max_pages]
  const int* lens;    // [groups]
  const int* starts;  // [groups + 1] first sequence of each group, or NULL: one group of all
  float* part_o;      // [chunks][MT][D / 4][128][4]: a warp's rows lie together
  float* part_lse;    // [chunks][MT][128], log2 units
  int* base;          // [2 groups + 1] first unit and first item of each group; all units
  int B, Lq, H, Hkv, g, groups;
  int tok;            // tokens of a tile: 128 / g
  int max_items;      // the workspace's
  int ginv;           // 65536 / g + 1: row / g = row * ginv >> 16
  int page, max_pages, cap;  // cap = max_pages * page
  float sl2;          // log2(e) / sqrt(D)
};

// One group: its tokens [t0, t1) of the batch's B * Lq, its items per K/V head
// and its units per item.
struct PrefixGroup {
  int n;  // prefix length
  int t0, t1, items, cnt;
};

template <int MT>
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixParams& p, int i) {
  PrefixGroup s;
  int b0 = 0, b1 = p.B;
  if (p.starts != nullptr) {
    b0 = min(max(p.starts[i], 0), p.B);
    b1 = min(max(p.starts[i + 1], b0), p.B);
  }
  s.n = min(max(p.lens[i], 0), p.cap);
  s.t0 = b0 * p.Lq;
  s.t1 = b1 * p.Lq;
  s.cnt = (s.n + 127) >> 7;
  s.items = s.cnt > 0 ? (s.t1 - s.t0 + MT * p.tok - 1) / (MT * p.tok) : 0;
  return s;
}

// Part c of G of `total` units begins at unit:
__device__ __forceinline__ int prefix_part(int total, int G, int c) {
  const int q = total / G, r = total - q * G;
  return c * q + (c < r ? c : r);
}
// The part that holds unit t.
__device__ __forceinline__ int prefix_part_of(int total, int G, int t) {
  const int q = total / G, r = total - q * G, big = r * (q + 1);
  return t < big ? t / (q + 1) : r + (t - big) / q;
}

// Walk over the chunks of one part.
template <int MT>
struct PrefixWalk {
  int grp, hkv, it, k;  // group, K/V head, item of it, first unit of the chunk
  int left;             // units of the chunk
  int rem;              // units left in the part, the chunk's included
  int chunk;            // its number
  int done;             // chunks before it in the part
  PrefixGroup s;

  __device__ __forceinline__ void next(const PrefixParams& p) {
    rem -= left;
    if (rem <= 0) return;
    k = 0;
    ++chunk;
    ++done;
    if (++it == s.items) {
      it = 0;
      if (++hkv == p.Hkv) {
        hkv = 0;
        do {
          if (++grp >= p.groups) {
            rem = 0;
            return;
          }
          s = prefix_group<MT>(p, grp);
        } while (s.items == 0);
      }
    }
    left = min(s.cnt, rem);
  }
  // First token of tile t of the item.
  __device__ __forceinline__ int token(const PrefixParams& p, int t) const { return s.t0 + (it * MT + t) * p.tok; }
};

template <int D, int MT>
struct PrefixLayout {
  static constexpr int KCH = D / 64;
  static constexpr uint32_t CHUNK = 128u * 128u;  // 128 rows x 64 columns
  static constexpr uint32_t TILE = KCH * CHUNK;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr uint32_t Q_OFF = 0;
  static constexpr uint32_t RING_OFF = MT * TILE;
  static constexpr uint32_t BAR_OFF = RING_OFF + STAGES * TILE;
  static constexpr int B_QFULL = 0, B_QEMPTY = 1, B_KVFULL = 2, B_KVEMPTY = B_KVFULL + STAGES,
                       B_SFULL = B_KVEMPTY + STAGES, B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 4,
                       B_OEMPTY = B_OFULL + 2, B_MATE = B_OEMPTY + 2, B_DONE = B_MATE + 1, NBAR = B_DONE + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;  // tmem slot, abort flag, plan, sums
  static constexpr uint32_t MATE_OFF = (MISC_OFF + 192 + 15) / 16 * 16;  // MT = 1: [2 chunks][2 groups][m, l][128]
  static constexpr uint32_t SMEM_USED = MATE_OFF + (MT == 1 ? 4096 : 0);
  static constexpr uint32_t SMEM_ALLOC = SMEM_USED + 1024;
  static constexpr uint32_t TM_S = 0, TM_O = 256, TMEM_COLS = 512;
  static constexpr int NTHREADS = 320;
  static_assert(SMEM_ALLOC <= 232448, "shared memory");
};

// This CTA's part: the walk's start in plan {grp, hkv, it, k, n, first chunk}.
// Called by the whole CTA; CTA 0 leaves the groups' bases for the join.
template <int MT, int NT>
__device__ __forceinline__ void prefix_plan(const PrefixParams& p, long long* sums, int* plan) {
  const int lane = lane_id(), G = gridDim.x, c = blockIdx.x;
  const int per = (p.groups + NT - 1) / NT;
  const int i0 = min(p.groups, static_cast<int>(threadIdx.x) * per), i1 = min(p.groups, i0 + per);
  // (64 bits: starts that fall make groups overlap, and any sum possible)
  long long units = 0, items = 0;
  for (int i = i0; i < i1; ++i) {
    const PrefixGroup s = prefix_group<MT>(p, i);
    units += static_cast<long long>(s.items) * s.cnt * p.Hkv;
    items += static_cast<long long>(s.items) * p.Hkv;
  }
  long long iu = units, ii = items;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, iu, h), b = __shfl_up_sync(0xffffffffu, ii, h);
    if (lane >= h) {
      iu += a;
      ii += b;
    }
  }
  if (lane == 31) {
    sums[2 * warp_id()] = iu;
    sums[2 * warp_id() + 1] = ii;
  }
  __syncthreads();
  long long before_u = iu - units, before_i = ii - items, all_u = 0, all_i = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < static_cast<int>(warp_id())) {
      before_u += sums[2 * w];
      before_i += sums[2 * w + 1];
    }
    all_u += sums[2 * w];
    all_i += sums[2 * w + 1];
  }
  // More items than the workspace has room for: starts that fall.  No prefix then.
  const int total = all_i <= p.max_items && all_u < (1ll << 31) ? static_cast<int>(all_u) : 0;
  int ub = static_cast<int>(before_u), ib = static_cast<int>(before_i);
  const int t0 = prefix_part(total, G, c), n = prefix_part(total, G, c + 1) - t0;
  if (threadIdx.x == 0) {
    plan[4] = n;
    if (c == 0) p.base[2 * p.groups] = total;
  }
  for (int i = i0; i < i1; ++i) {
    const PrefixGroup s = prefix_group<MT>(p, i);
    const int here = s.items * s.cnt * p.Hkv;
    if (c == 0) {
      p.base[2 * i] = ub;
      p.base[2 * i + 1] = ib;
    }
    if (n > 0 && t0 >= ub && t0 < ub + here) {
      const int item = (t0 - ub) / s.cnt;
      plan[0] = i;
      plan[1] = item / s.items;
      plan[2] = item - plan[1] * s.items;
      plan[3] = t0 - ub - item * s.cnt;
      plan[5] = ib + item + c;
    }
    ub += here;
    ib += s.items * p.Hkv;
  }
  __syncthreads();
}

template <int MT>
__device__ __forceinline__ PrefixWalk<MT> prefix_walk(const PrefixParams& p, const int* plan) {
  PrefixWalk<MT> w;
  w.rem = plan[4];
  w.left = 0;
  w.done = 0;
  if (w.rem > 0) {
    w.grp = plan[0];
    w.hkv = plan[1];
    w.it = plan[2];
    w.k = plan[3];
    w.chunk = plan[5];
    w.s = prefix_group<MT>(p, w.grp);
    w.left = min(w.s.cnt - w.k, w.rem);
  }
  return w;
}

template <int D, bool BF16, int MT>
__global__ void __launch_bounds__(320, 1)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const PrefixParams p) {
  using Ly = PrefixLayout<D, MT>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  using Walk = PrefixWalk<MT>;
  constexpr uint32_t IDESC_S = idesc_f16(BF16, 128, 128, false, false);
  constexpr uint32_t IDESC_PV = idesc_f16(BF16, 128, D, false, true);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + Ly::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Ly::MISC_OFF);
  AbortState* ab = reinterpret_cast<AbortState*>(gbase + Ly::MISC_OFF + 4);
  int* plan = reinterpret_cast<int*>(gbase + Ly::MISC_OFF + 8);   // 6
  long long* sums = reinterpret_cast<long long*>(gbase + Ly::MISC_OFF + 32);  // 2 x 10 warps
  unsigned int* err = device_error_word();
  const uint32_t warp = warp_id(), lane = lane_id();

  // Rows of a tile that no head fills (g not a power of two) are zero.
  const int rows = p.tok * p.g;
  if (rows < 128) {
    for (uint32_t i = threadIdx.x; i < MT * Ly::TILE / 16u; i += Ly::NTHREADS)
      reinterpret_cast<uint4*>(gbase + Ly::Q_OFF)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < Ly::NBAR; ++i) {
      const bool p_full = i >= Ly::B_PFULL && i < Ly::B_OFULL, o_empty = i >= Ly::B_OEMPTY && i < Ly::B_MATE;
      // (MT = 1: both groups read both O)
      mbar_init(bar(i), p_full ? 4 : o_empty ? (MT == 1 ? 8 : 4) : i == Ly::B_MATE ? 8 : 1);
    }
    ab->flag = 0;
    fence_barrier_init();
  }
  if (warp == 8 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(base + Ly::MISC_OFF, Ly::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  // What was before is done when the next kernel in the stream may start.
  pdl_wait();
  pdl_launch_dependents();
  prefix_plan<MT, Ly::NTHREADS>(p, sums, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ------------------------------------------------------------ producer
    const int page_log = 31 - __clz(p.page);  // (a page is a power of two)
    const int box = min(p.page, 128), nbox = 128 >> min(page_log, 7), per_batch = 32 >> (7 - min(page_log, 7));
    uint32_t stage = 0, phase = 0, used = 0, q_uses = 0;
    bool ok = true;
    for (Walk w = prefix_walk<MT>(p, plan); ok && w.rem > 0; w.next(p)) {
      if (q_uses > 0 && !mbar_wait_warp(bar(Ly::B_QEMPTY), (q_uses - 1) & 1, ab, err, 1101)) {
        ok = false;
        break;
      }
      const int tiles = MT == 2 && w.token(p, 1) < w.s.t1 ? 2 : 1;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(Ly::B_QFULL), static_cast<uint32_t>(tiles * Ly::KCH * rows) * 128u);
        for (int t = 0; t < tiles; ++t)
          for (int c = 0; c < Ly::KCH; ++c)
            tma_load_4d(base + Ly::Q_OFF + t * Ly::TILE + c * Ly::CHUNK, &tmQ, bar(Ly::B_QFULL), c * 64,
                        w.hkv * p.g, w.token(p, t), 0);
      }
      __syncwarp();
      ++q_uses;
      // Page ids of the next tiles, one box per lane, a batch ahead.
      const int* table = p.table + static_cast<size_t>(w.grp) * p.max_pages;
      auto pages = [&](int j) -> int {
        const int at = ((w.k + j) * 128 + static_cast<int>(lane) * box) >> page_log;
        return at < p.max_pages ? table[at] : -1;
      };
      int ids = pages(0), ahead = per_batch < w.left ? pages(per_batch) : -1;
      for (int j = 0; ok && j < w.left; ++j) {
        const int x = j % per_batch;
        if (x == 0 && j > 0) {
          ids = ahead;
          if (j + per_batch < w.left) ahead = pages(j + per_batch);
        }
        const int pid = __shfl_sync(0xffffffffu, ids, (x * nbox + static_cast<int>(lane)) & 31);
        const int k0 = (w.k + j) * 128 + static_cast<int>(lane) * box;
        const bool go = static_cast<int>(lane) < nbox && k0 < w.s.n;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, go));
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          if (!mbar_wait_warp(bar(Ly::B_KVEMPTY + stage), phase ^ 1u, ab, err, 1102)) {
            ok = false;
            break;
          }
          if (lane == 0)
            mbar_arrive_expect_tx(bar(Ly::B_KVFULL + stage), boxes * box * static_cast<uint32_t>(D) * 2u);
          __syncwarp();
          if (go) {
#pragma unroll
            for (int c = 0; c < Ly::KCH; ++c)
              tma_load_4d(base + Ly::RING_OFF + stage * Ly::TILE + c * Ly::CHUNK + lane * box * 128u,
                          kv ? &tmV : &tmK, bar(Ly::B_KVFULL + stage), c * 64, w.hkv, k0 & (p.page - 1), pid);
          }
          used |= 1u << stage;
          if (++stage == Ly::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    }
    if (!ok && lane == 0) {
      // Unwinding: let copies in flight land.  The newest use of a stage before
      // the write position has this round's parity, the others the last round's.
      if (q_uses > 0) mbar_wait_drain(bar(Ly::B_QFULL), (q_uses - 1) & 1);
      for (int s = 0; s < Ly::STAGES; ++s)
        if (used >> s & 1u)
          mbar_wait_drain(bar(Ly::B_KVFULL + s), s < static_cast<int>(stage) ? phase : phase ^ 1u);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0, q_cnt = 0;
    uint32_t p_cnt0 = 0, p_cnt1 = 0, o_uses0 = 0, o_uses1 = 0;  // (scalars: they stay in registers)
    bool ok = true;
    auto tS = [&](int t) { return tmem + Ly::TM_S + 128u * t; };
    auto tO = [&](int t) { return tmem + Ly::TM_O + static_cast<uint32_t>(D) * t; };
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
      __syncwarp();
    };
    auto issue_s = [&](int t, uint32_t ks) {
      const uint64_t qd = sdesc_sw128(base + Ly::Q_OFF + (MT == 2 ? t : 0) * Ly::TILE, 16, 1024);
      const uint64_t kd = sdesc_sw128(base + Ly::RING_OFF + ks * Ly::TILE, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint64_t off = ((k >> 2) * Ly::CHUNK + (k & 3) * 32u) >> 4;
          mma_ss(tS(t), qd + off, kd + off, IDESC_S, k > 0 ? 1u : 0u);
        }
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, uint32_t vs, bool acc, int k_lo, int k_hi) {
      const uint64_t vd = sdesc_sw128(base + Ly::RING_OFF + vs * Ly::TILE, Ly::CHUNK, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = k_lo; k < k_hi; ++k)
          mma_ts(tO(t), tS(t) + 8u * k, vd + ((2048u * k) >> 4), IDESC_PV, (acc || k > 0) ? 1u : 0u);
      }
      __syncwarp();
    };
    auto take = [&](uint32_t& slot, unsigned int site) -> bool {
      slot = stage;
      if (!mbar_wait_warp(bar(Ly::B_KVFULL + stage), phase, ab, err, site)) return false;
      if (++stage == Ly::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      tc_fence_after();
      return true;
    };
    for (Walk w = prefix_walk<MT>(p, plan); ok && w.rem > 0; w.next(p)) {
      const int n = w.left;
      const int tiles = MT == 2 && w.token(p, 1) < w.s.t1 ? 2 : 1;
      if (!mbar_wait_warp(bar(Ly::B_QFULL), q_cnt & 1, ab, err, 1103)) { ok = false; break; }
      ++q_cnt;
      tc_fence_after();
      uint32_t ks, vs;
      if (!take(ks, 1104)) { ok = false; break; }
      for (int t = 0; t < tiles; ++t) {
        issue_s(t, ks);
        commit(Ly::B_SFULL + t);
      }
      commit(Ly::B_KVEMPTY + ks);
      for (int j = 0; ok && j < n; ++j) {
        if (!take(vs, 1105)) { ok = false; break; }
        const bool more = j + 1 < n;
        if (more && !take(ks, 1106)) { ok = false; break; }
        if (MT == 1 && more) {
          // The other group's next step, ahead of this one's P.
          issue_s((j + 1) & 1, ks);
          commit(Ly::B_SFULL + ((j + 1) & 1));
          commit(Ly::B_KVEMPTY + ks);
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (MT == 1 ? (j & 1) != t : t >= tiles) continue;
          uint32_t& p_cnt = t ? p_cnt1 : p_cnt0;
          uint32_t& o_uses = t ? o_uses1 : o_uses0;
          const bool first = MT == 1 ? j < 2 : j == 0;
          if (first && o_uses > 0 &&
              !mbar_wait_warp(bar(Ly::B_OEMPTY + t), (o_uses - 1) & 1, ab, err, 1107)) {
            ok = false;
            break;
          }
          if (!mbar_wait_warp(bar(Ly::B_PFULL + 2 * t), p_cnt & 1, ab, err, 1108)) { ok = false; break; }
          tc_fence_after();
          issue_pv(t, vs, !first, 0, 4);
          if (!mbar_wait_warp(bar(Ly::B_PFULL + 2 * t + 1), p_cnt & 1, ab, err, 1109)) { ok = false; break; }
          ++p_cnt;
          tc_fence_after();
          issue_pv(t, vs, true, 4, 8);
          if (MT == 1 ? j + 2 >= n : !more) {  // the tile's (or the group's) last step
            commit(Ly::B_OFULL + t);
            ++o_uses;
          }
          if (MT == 2 && more) {
            issue_s(t, ks);
            commit(Ly::B_SFULL + t);
          }
        }
        if (!ok) break;
        commit(Ly::B_KVEMPTY + vs);
        if (MT == 2 && more) commit(Ly::B_KVEMPTY + ks);
      }
      if (!ok) break;
      commit(Ly::B_QEMPTY);
    }
    commit(Ly::B_DONE);
    mbar_wait_drain(bar(Ly::B_DONE), 0);
  } else {
    // ------------------------------------------------------------ softmax
    const int t = warp >> 2;          // MT = 2: the tile; MT = 1: steps j % 2 = t
    const int r = threadIdx.x & 127;  // row of the tile == TMEM lane
    const uint32_t lane_off = ((warp & 3u) * 32u) << 16;
    const uint32_t tS = tmem + lane_off + Ly::TM_S + 128u * t;
    const uint32_t tO = tmem + lane_off + Ly::TM_O + static_cast<uint32_t>(D) * t;
    const float sl2 = p.sl2;
    uint32_t s_cnt = 0, o_cnt = 0, o1_cnt = 0, mates = 0;
    uint32_t ring = 0;  // ring position of the chunk's first K
    bool ok = true;
    for (Walk w = prefix_walk<MT>(p, plan); ok && w.rem > 0; ring += 2 * w.left, w.next(p)) {
      const int tile = MT == 2 ? t : 0;
      const int tok0 = w.token(p, tile);
      if (MT == 2 && tok0 >= w.s.t1) continue;
      const bool live = r < rows && tok0 + (r * p.ginv >> 16) < w.s.t1;
      float m = -INFINITY, l = 0.f;
      for (int j = MT == 2 ? 0 : t; j < w.left; j += MT == 2 ? 1 : 2) {
        if (!mbar_wait_warp(bar(Ly::B_SFULL + t), s_cnt & 1, ab, err, 1110)) { ok = false; break; }
        ++s_cnt;
        tc_fence_after();
        uint32_t sr[128];
        tmem_ld32(tS + 0, sr);
        tmem_ld32(tS + 32, sr + 32);
        tmem_ld32(tS + 64, sr + 64);
        tmem_ld32(tS + 96, sr + 96);
        tmem_ld_wait32(sr);
        tmem_ld_wait32(sr + 32);
        tmem_ld_wait32(sr + 64);
        tmem_ld_wait32(sr + 96);
        const int valid = w.s.n - (w.k + j) * 128;  // keys of the tile, >= 1
        if (valid < 128) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= valid) sr[c] = __float_as_uint(-INFINITY);
        }
        float mx8[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          mx8[u] = fmax3(__uint_as_float(sr[u]), __uint_as_float(sr[8 + u]), __uint_as_float(sr[16 + u]));
#pragma unroll
          for (int x = 3; x < 15; x += 2)
            mx8[u] = fmax3(mx8[u], __uint_as_float(sr[8 * x + u]), __uint_as_float(sr[8 * x + 8 + u]));
          mx8[u] = fmaxf(mx8[u], __uint_as_float(sr[120 + u]));
        }
        const float mx = fmax3(fmax3(mx8[0], mx8[1], mx8[2]), fmax3(mx8[3], mx8[4], mx8[5]),
                               fmaxf(mx8[6], mx8[7]));
        const float m_new = fmaxf(m, mx);
        float alpha = 1.f;
        bool rescale = false;
        if (j == (MT == 2 ? 0 : t)) {
          m = m_new;
        } else if (__any_sync(0xffffffffu, (m_new - m) * sl2 > 8.0f)) {
          // Some row's maximum grew by more than 2^8: this warp's rows move theirs.
          // (A row whose scores were all -inf so far has O = l = 0.)
          if (m_new != -INFINITY) alpha = ex2((m - m_new) * sl2);
          m = m_new;
          rescale = true;
        }
        // Half h of P is in TMEM.  Before the first, O is scaled if the maximum
        // moved (the commit behind this S covers the tile's, or group's, last PV),
        // and V's rows behind the prefix's end, whatever their slots hold, are zero.
        auto p_ready = [&](int h) {
          if (h == 0 && rescale) {
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * cc, o);
              tmem_ld_wait32(o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st32(tO + 32 * cc, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Ly::B_PFULL + 2 * t + h));
        };
        if (valid < 128 && tile == 0) {
          // (V's stage held, before it, a tile that S of this step or an earlier
          // product has used, so the parity cannot be the fill before's.)
          const uint32_t pos = ring + 2 * j + 1;
          if (!mbar_wait_warp(bar(Ly::B_KVFULL + pos % Ly::STAGES), (pos / Ly::STAGES) & 1, ab, err, 1111)) {
            ok = false;
            break;
          }
          if (r >= valid) {
            uint4* v = reinterpret_cast<uint4*>(gbase + Ly::RING_OFF + (pos % Ly::STAGES) * Ly::TILE + r * 128);
#pragma unroll
            for (int c = 0; c < Ly::KCH; ++c)
#pragma unroll
              for (int u = 0; u < 8; ++u) v[c * (Ly::CHUNK / 16) + u] = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        const float mb = m == -INFINITY ? 0.f : m * sl2;
        const uint64_t sl2x2 = f2_pack(sl2, sl2), nmb2 = f2_pack(-mb, -mb);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        // P = exp2(s c - m c), rounded to the 16-bit type that the MMA reads; the
        // row sum takes the unrounded values.
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c = 32 * q4 + 2 * i;
            float a0, a1;
            f2_unpack(ffma2(f2_pack(__uint_as_float(sr[c]), __uint_as_float(sr[c + 1])), sl2x2, nmb2), a0, a1);
            const float p0 = ex2(a0), p1 = ex2(a1);
            acc[i & 3] = fadd2(acc[i & 3], f2_pack(p0, p1));
            pk[i] = pack2<T>(p0, p1);
          }
          tmem_st16(tS + 16 * q4, pk);
          if (q4 & 1) p_ready(q4 >> 1);
        }
        float rs4[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float lo, hi;
          f2_unpack(acc[u], lo, hi);
          rs4[u] = lo + hi;
        }
        l = l * alpha + ((rs4[0] + rs4[1]) + (rs4[2] + rs4[3]));
      }
      if (!ok) break;
      // ---- the chunk's partial: O / l and its LSE
      float f0 = 1.f, f1 = 0.f;  // factors of O_0 and O_1 (MT = 1)
      bool both = false;
      if constexpr (MT == 1) {
        // Both groups leave their maxima and sums; each stores half of the columns.
        float* mate = reinterpret_cast<float*>(gbase + Ly::MATE_OFF) + (mates & 1) * 512;  // [2][m, l][128]
        mate[256 * t + r] = m;
        mate[256 * t + 128 + r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_MATE));
        if (!mbar_wait_warp(bar(Ly::B_MATE), mates & 1, ab, err, 1112)) { ok = false; break; }
        ++mates;
        const float m0 = mate[r], m1 = mate[256 + r];
        const float top = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.f : ex2((m0 - top) * sl2);
        f1 = m1 == -INFINITY ? 0.f : ex2((m1 - top) * sl2);
        l = mate[128 + r] * f0 + mate[384 + r] * f1;
        m = top;
        both = w.left > 1;
        if (!mbar_wait_warp(bar(Ly::B_OFULL), o_cnt & 1, ab, err, 1113)) { ok = false; break; }
        ++o_cnt;
        if (both) {
          if (!mbar_wait_warp(bar(Ly::B_OFULL + 1), o1_cnt & 1, ab, err, 1114)) { ok = false; break; }
          ++o1_cnt;
        }
      } else {
        if (!mbar_wait_warp(bar(Ly::B_OFULL + t), o_cnt & 1, ab, err, 1115)) { ok = false; break; }
        ++o_cnt;
      }
      tc_fence_after();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      f0 *= inv;
      f1 *= inv;
      const size_t at = static_cast<size_t>(w.chunk) * MT + tile;
      float4* dst = reinterpret_cast<float4*>(p.part_o) + at * (D / 4) * 128 + r;
      const int c0 = MT == 1 ? t * (D / 64) : 0, c1 = MT == 1 ? c0 + D / 64 : D / 32;
#pragma unroll 1
      for (int cc = c0; cc < c1; ++cc) {
        uint32_t o[32];
        tmem_ld32(tmem + lane_off + Ly::TM_O + (MT == 2 ? D * t : 0) + 32 * cc, o);
        tmem_ld_wait32(o);
        float v[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f0;
        if (MT == 1 && both) {
          tmem_ld32(tmem + lane_off + Ly::TM_O + D + 32 * cc, o);
          tmem_ld_wait32(o);
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), f1, v[i]);
        }
        if (live) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[(8 * cc + i) * 128] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      if (live && (MT == 2 || t == 0))
        p.part_lse[at * 128 + r] = l == 0.f ? -INFINITY : m * sl2 + __log2f(l);  // (NaN stays NaN)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (MT == 2) {
          mbar_arrive(bar(Ly::B_OEMPTY + t));
        } else {
          mbar_arrive(bar(Ly::B_OEMPTY));
          if (both) mbar_arrive(bar(Ly::B_OEMPTY + 1));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Ly::TMEM_COLS);
  }
}

struct PrefixJoinParams {
  PrefixParams p;
  const int* own_lens;   // [B]
  const float* own_o;    // [B, Lq, H, D]
  const float* own_lse;  // [B, H, Lq], natural log
  void* O;               // [B, Lq, H, D]
  float* LSE;            // [B, H, Lq], natural log
  int own_cap;
  int G;                 // CTAs of fa_prefix_kernel
};

// Join each row's partials: those of its prefix's chunks and that of its own
// keys.  A thread joins 8 dims of one row; the lanes run over the g heads of a
// K/V head, whose rows lie together in a partial, then over the dims.
template <int D, bool BF16, int MT>
__global__ void __launch_bounds__(256) fa_prefix_join_kernel(const PrefixJoinParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  const PrefixParams& p = a.p;
  pdl_launch_dependents();
  pdl_wait();
  const int per = p.g * (D / 8), ppb = per <= 256 ? 256 / per : 1;
  const int pl = static_cast<int>(threadIdx.x) / per;  // pair (token, K/V head) of the block
  const long long pair = static_cast<long long>(blockIdx.x) * ppb + pl;
  if (pl >= ppb || pair >= static_cast<long long>(p.B) * p.Lq * p.Hkv) return;
  const int tk = static_cast<int>(pair / p.Hkv), hkv = static_cast<int>(pair - static_cast<long long>(tk) * p.Hkv);
  const int b = tk / p.Lq, ql = tk - b * p.Lq;
  const bool pad = min(max(a.own_lens[b], 0), a.own_cap) - p.Lq + ql < 0;
  // The sequence's group, and the chunks of its tile.
  int grp = 0;
  if (p.starts != nullptr) {
    int lo = 0, hi = p.groups;  // the last group that starts at or before b
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.starts[mid] <= b) lo = mid;
      else hi = mid;
    }
    grp = lo;
  }
  const PrefixGroup s = prefix_group<MT>(p, grp);
  int n = 0, chunk0 = 0, row0 = 0, tile = 0;
  const int total = p.base[2 * p.groups];
  if (!pad && total > 0 && s.items > 0 && tk >= s.t0 && tk < s.t1) {
    tile = (tk - s.t0) / p.tok;
    row0 = (tk - s.t0 - tile * p.tok) * p.g;
    const int it = hkv * s.items + tile / MT;
    const int first = p.base[2 * grp] + it * s.cnt;
    const int c0 = prefix_part_of(total, a.G, first), c1 = prefix_part_of(total, a.G, first + s.cnt - 1);
    chunk0 = p.base[2 * grp + 1] + it + c0;
    n = c1 - c0 + 1;
    tile %= MT;
  }
  for (int x = static_cast<int>(threadIdx.x) - pl * per; x < per; x += 256) {
    const int d8 = x / p.g, hg = x - d8 * p.g, h = hkv * p.g + hg;
    const size_t out = (static_cast<size_t>(tk) * p.H + h) * D + 8 * d8;
    const size_t lse_at = (static_cast<size_t>(b) * p.H + h) * p.Lq + ql;
    float mx = -INFINITY, den = 0.f, acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    if (!pad) {
      auto add = [&](float lse, const float4& u, const float4& v) {
        const float m = fmaxf(mx, lse);
        // (each for itself: a NaN LSE has no part in m, but its weight is NaN)
        const float old = mx == -INFINITY ? 0.f : ex2(mx - m), w = lse == -INFINITY ? 0.f : ex2(lse - m);
        const float o[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
        den = fmaf(den, old, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(acc[i], old, lse == -INFINITY ? 0.f : w * o[i]);
        mx = m;
      };
      const float4* own = reinterpret_cast<const float4*>(a.own_o + out);
      const float4 ou = own[0], ov = own[1];
      const float ol = a.own_lse[lse_at] * 1.4426950408889634f;
      constexpr int C = 4;
#pragma unroll 1
      for (int q0 = 0; q0 < n; q0 += C) {
        float ls[C];
        float4 u[C], v[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const size_t at = static_cast<size_t>(chunk0 + min(q0 + c, n - 1)) * MT + tile;
          const float4* src = reinterpret_cast<const float4*>(p.part_o) + (at * (D / 4) + 2 * d8) * 128 + row0 + hg;
          ls[c] = q0 + c < n ? p.part_lse[at * 128 + row0 + hg] : -INFINITY;
          u[c] = src[0];
          v[c] = src[128];
        }
#pragma unroll
        for (int c = 0; c < C; ++c) add(ls[c], u[c], v[c]);
      }
      add(ol, ou, ov);
    }
    const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);  // (NaN stays NaN)
    *reinterpret_cast<uint4*>(reinterpret_cast<T*>(a.O) + out) =
        make_uint4(pack2<T>(acc[0] * inv, acc[1] * inv), pack2<T>(acc[2] * inv, acc[3] * inv),
                   pack2<T>(acc[4] * inv, acc[5] * inv), pack2<T>(acc[6] * inv, acc[7] * inv));
    if (d8 == 0) a.LSE[lse_at] = den == 0.f ? -INFINITY : (mx + __log2f(den)) * 0.6931471805599453f;
  }
}

}  // namespace fa
