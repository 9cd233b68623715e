// Attention of a batch's new tokens over key/value prefixes that several of its
// sequences share and over each sequence's own keys, both in a paged cache.
//
// Mathematics: softmax over the union of sets of keys from the softmaxes of
// each: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.  Every new
// token behind a prefix sees all of it, so the prefix's part is one product
// chain of all rows (tokens x query heads of a K/V head) with the prefix's keys
// and values, which are read once for 256 rows, not once per sequence.
//
// Two launches: fa_prefix_kernel cuts both parts into chunks and leaves each
// chunk's partial O and LSE in fp32; fa_prefix_join_kernel joins each row's.
//
// fa_prefix_kernel, a persistent CTA per SM, of one of two kinds.
//   Prefixes (prefix_body).  A tile is up to 128 rows: 128 / g tokens of a group (g
//   query heads a K/V head), row = token * g + head.  An item is one K/V head of a
//   group and two neighbouring tiles (the last may have one); its units are the
//   prefix's 128-key tiles.  The units of all items form one list, in which a unit
//   weighs about what it takes, and each CTA takes an equal part of it, so all work
//   alike whatever the lengths and groups are.
//   Own keys (paged_body, R > 0): the paged decode's roles, whose products are
//   transposed and waste no rows on a sequence's few.  Sequences of more than 32
//   rows (R = 0) fill a tile well enough: their items are in the prefixes' list, of
//   one tile each.
// How many CTAs are of each kind follows on the device from the lengths: the first
// are bound by the products, the others by the read, so the two overlap on the
// chip and one launch's start serves both.  A part's share of an item is a chunk.
// Own keys' chunks are stored at item + part, which no two share: the next chunk in a
// list is of a later item, a later part, or both.  Prefixes' are stored at the rows
// before the item + 256 part (an item has 256 rows at most), for the same reason.
// The join finds an item's first and last part in a table.
//
// prefix_body:
//   warps 0-3, 4-7  softmax, a thread per row.  Two tiles: one each.  One tile:
//                   its even and its odd steps, each group with a maximum, a sum
//                   and an O of its own; warps 4-7 join them at the chunk's end
//                   while warps 0-3 begin the next
//   warp 9          TMEM, MMAs: S_t = Q_t K_j^T, P over S as 16 bits, O_t += P V_j
//   warp 10         TMA: Q, then K_0, V_0, K_1, V_1, ... through one ring across
//                   chunks; lane i loads the i-th page of a tile
// Registers: 200 a softmax thread, 104 the others.  With fewer for the warp that
// issues the products its descriptors are spilled, and a unit of two tiles took
// 4,400 cycles instead of 2,950.
// What bounds it: per 64 KB of K and V (D = 128) two tiles take 2,950 cycles, of
// which the tensor cores work 2,200 (each tile's chain S, softmax, PV, S is in the
// way, as in the dense forward); a CTA's share of the memory bandwidth brings 64 KB
// in 2,790.  A launch's first 5 us go until the first scores are there (2 to the plan:
// code, lengths; then page ids, the first tiles), its last 5 to the join.
// P goes to its product in the inputs' 16-bit type, like all of this library's: the
// outputs' distance from 64 bits is 1.3 to 1.4 times that of one rounding at the end.
// Measured (H32/8 D128): 64 sequences of 100 to 1,000 own keys behind 32,768: 59.5 us
// (the paged decode over tables that repeat the prefix reads it 64 times from the L2);
// 256 of 64 to 512 behind 16,384: 95.6 us, with pages of 16 137; 20 of four tokens, 50
// to 800 behind 6,001: 31 us, of 8 tokens (32 rows) 46, of 16 (64 rows) 58; 8 of 1 to
// 100 behind 2,001: 14 us.  H16/16 D64: 40 of 16 to 500 in five groups behind 1,000 to
// 9,000: 36.5 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "fwd.cuh"  // pack2
#include "paged.cuh"
#include "ptx.cuh"

namespace fa {

struct PrefixParams {
  const int *ptable, *plens;  // [groups, prefix_pages], [groups]
  const int* starts;          // [groups + 1] first sequence of each group, or NULL: one group of all
  const int *table, *lens;    // [B, max_pages], [B]: own keys
  float* part_o;              // prefix partials: a tile's [D / 4][its rows][4], so that a warp's rows lie together
  float* part_lse;            // a row's, log2 units; where a chunk's rows begin: prefix_first_row
  float* own_o;               // [B * Hkv + G][rows][D]
  float* own_lse;             // [B * Hkv + G][rows], log2 units
  int* ends;                  // [prefix items][2], then [B * Hkv][2]: an item's first and last part
  uint32_t most;              // the list's weight can be no more (all sums fit 32 bits)
  int B, Lq, H, Hkv, g, groups, rows;  // rows = g * Lq
  int tok;                    // tokens of a prefix's tile: 128 / g
  int items;                  // prefix items there may be
  int entries;                // of the list: groups, or groups + B
  int ginv;                   // 65536 / g + 1: row / g = row * ginv >> 16
  int page, prefix_pages, max_pages, pcap, cap;  // caps: pages * page
  float sl2;                  // log2(e) / sqrt(D)
  int pair_weight;            // of a unit of two tiles
  float own_weight;           // of own keys in CTAs of their own
};

// mbar_wait_warp in less code, inlined: a call, as the paged decode's waits are,
// does not go with the register split (its callee could not be allocated).
__device__ __forceinline__ bool prefix_wait(uint32_t bar, uint32_t parity, AbortState* ab, unsigned int* err,
                                            unsigned int site) {
  bool ok = false;
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) {
      ok = true;
      break;
    }
    if ((it & 31u) == 0u) {
      if (*reinterpret_cast<volatile int*>(&ab->flag)) break;
      const unsigned long long now = globaltimer_ns();
      if (t0 == 0) t0 = now;
      if (now - t0 > kWaitTimeoutNs) {
        *reinterpret_cast<volatile int*>(&ab->flag) = 1;
        atomicCAS(err, 0u, site);
        break;
      }
    }
  }
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

// Arrive n times.
__device__ __forceinline__ void prefix_arrive(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

// What a unit weighs: of one tile, and of two; and in the same measure the own keys
// that have CTAs of their own, a tile and as much again an item.  At D = 128 a unit of
// one tile is bound by the read and gets more than its share while others compute: own
// keys 1.5 (256 sequences behind 16,384 keys 98 us, behind 32,768 65; with 1.3 103 and
// 68, with 1.75 106 and 67).  At D = 64 one tile takes 1,300 cycles, two 2,700, an own
// tile and an item 1,300 to 1,400 each (five groups 39 us; with 3, 2 and 1.5 43).
// Swept with 1 to 4 rows a sequence; tiles of more rows, which take longer, weigh the
// same (of 16: the own keys' CTAs end a quarter later than the others).
constexpr int kOneWeight = 2;
constexpr int prefix_pair_weight(int D) { return D == 64 ? 4 : 3; }
constexpr float prefix_own_weight(int D) { return D == 64 ? 2.f : 1.5f; }
// Own items of at most so many tiles in the mean go whole to a softmax group each,
// in turn (100 to 2,000 keys: 55.7 us, with their tiles in turn 59.8; 24 tiles: no
// difference).
constexpr uint32_t kShortItem = 12;

// An entry of the list: group e, or the own keys of sequence e - groups.
struct PrefixEntry {
  int n;       // keys
  int cnt;     // units of an item
  int t0, t1;  // the group's tokens among the batch's B * Lq
  int items;   // per K/V head
  int weight;  // of a unit
};

__device__ __forceinline__ PrefixEntry prefix_entry(const PrefixParams& p, int e) {
  PrefixEntry s;
  if (e < p.groups) {
    int b0 = 0, b1 = p.B;
    if (p.starts != nullptr) {
      b0 = min(max(__ldcg(p.starts + e), 0), p.B);
      b1 = min(max(__ldcg(p.starts + e + 1), b0), p.B);
    }
    s.n = min(max(__ldcg(p.plens + e), 0), p.pcap);
    s.t0 = b0 * p.Lq;
    s.t1 = b1 * p.Lq;
    s.cnt = (s.n + 127) >> 7;
    s.items = s.cnt > 0 ? (s.t1 - s.t0 + 2 * p.tok - 1) / (2 * p.tok) : 0;
    s.weight = s.t1 - s.t0 > p.tok ? p.pair_weight : kOneWeight;
  } else {
    s.n = min(max(__ldcg(p.lens + e - p.groups), 0), p.cap);
    s.t0 = s.t1 = 0;
    s.cnt = (s.n + 127) >> 7;
    s.items = s.cnt > 0 ? 1 : 0;
    s.weight = kOneWeight;
  }
  return s;
}

// A group's first item's number: groups' numbers lie apart whatever their sizes
// (a group of n tokens has at most n / (2 tok) + 1 items a K/V head).
__device__ __forceinline__ int prefix_first_item(const PrefixParams& p, const PrefixEntry& s, int grp) {
  return (s.t0 / (2 * p.tok) + grp) * p.Hkv;
}

// Where the rows of a group's item's chunk in a part begin, among all partials: as
// many as the items before it have, whatever the groups' sizes, and the parts' 256.
// (B * Lq * H is below 2^31.)
__device__ __forceinline__ uint32_t prefix_first_row(const PrefixParams& p, const PrefixEntry& s, int hkv, int it, int part) {
  return static_cast<uint32_t>((s.t0 * p.Hkv + (s.t1 - s.t0) * hkv + 2 * p.tok * it) * p.g) + 256u * part;
}

// Walk over the chunks of one part.  OWN: own keys are in the list too.
template <bool OWN>
struct PrefixWalk {
  int e, hkv, it, k;  // entry, K/V head, item of it, first unit of the chunk
  int left;           // units of the chunk; 0: the part is done
  int rem;            // weight left in the part, the chunk's included
  PrefixEntry s;

  __device__ __forceinline__ int share() const {
    return s.weight == kOneWeight ? rem / kOneWeight : rem / s.weight;
  }
  __device__ __forceinline__ void next(const PrefixParams& p) {
    const bool ended = k + left < s.cnt;  // inside an item: the part's border
    rem -= left * s.weight;
    left = 0;
    k = 0;
    if (ended) return;
    if (++it == s.items) {
      it = 0;
      if (++hkv == p.Hkv) {
        hkv = 0;
#pragma unroll 1
        do {
          if (++e >= p.entries || rem < kOneWeight) return;
          s = prefix_entry(p, e);
        } while (s.items == 0);
      }
    }
    left = min(s.cnt, share());
  }
  __device__ __forceinline__ bool own(const PrefixParams& p) const { return OWN && e >= p.groups; }
  // First token of tile t of the item.
  __device__ __forceinline__ int token(const PrefixParams& p, int t) const { return s.t0 + (2 * it + t) * p.tok; }
  __device__ __forceinline__ bool pair(const PrefixParams& p) const { return !own(p) && token(p, 1) < s.t1; }
  // Rows of tile t.
  __device__ __forceinline__ int rows(const PrefixParams& p, int t) const {
    return own(p) ? p.rows : min(p.tok, s.t1 - token(p, t)) * p.g;
  }
};

template <int D>
struct PrefixLayout {
  static constexpr int KCH = D / 64;
  static constexpr uint32_t CHUNK = 128u * 128u;  // 128 rows x 64 columns
  static constexpr uint32_t TILE = KCH * CHUNK;
  static constexpr int STAGES = D == 128 ? 5 : 10;
  static constexpr uint32_t Q_OFF = 0;            // two tiles
  static constexpr uint32_t RING_OFF = 2 * TILE;
  static constexpr uint32_t MATE_OFF = RING_OFF + STAGES * TILE;  // m, l [128]
  static constexpr uint32_t BAR_OFF = MATE_OFF + 1024;
  static constexpr int B_QFULL = 0, B_QEMPTY = 2, B_KVFULL = 4, B_KVEMPTY = B_KVFULL + STAGES,
                       B_SFULL = B_KVEMPTY + STAGES, B_PFULL = B_SFULL + 2, B_OFULL = B_PFULL + 4,
                       B_OEMPTY = B_OFULL + 2, B_MFULL = B_OEMPTY + 2, B_MEMPTY = B_MFULL + 1, B_DONE = B_MEMPTY + 1,
                       NBAR = B_DONE + 1;
  static constexpr uint32_t USED = BAR_OFF + NBAR * 8;
  static constexpr uint32_t TM_S = 0, TM_O = 256;
  static constexpr int NTHREADS = 384;
  // Registers a thread at launch (65,536 / 384, in eights), and of the softmax
  // warpgroups and the other in a CTA of the list.
  static constexpr int REGS = 168, REGS_SOFTMAX = 200, REGS_OTHER = 104;
  static_assert(2 * REGS_SOFTMAX + REGS_OTHER == 3 * REGS, "register budgets sum to the launch's");
  // arrivals a barrier takes a phase
  __device__ static constexpr int arrivals(int i) {
    return (i >= B_PFULL && i < B_OFULL) || (i >= B_OEMPTY && i < B_DONE) ? 4 : 1;
  }
};

// What a CTA does: part c of the prefixes' list, or part c of G of the own keys'.
struct PrefixShare {
  bool own;
  int c, G;
};

// How the CTAs are shared out, and this one's part.  Called by the whole CTA (NT
// threads).  A CTA of the prefixes' list finds the start of its walk in plan
// {e, hkv, it, k, rem} and its entry behind.  OWN: own keys are not in the list and have CTAs of their
// own; plan[5] says whether their items are short.
template <int NT, bool OWN>
__device__ __forceinline__ PrefixShare prefix_plan(const PrefixParams& p, uint32_t* sums, int* plan) {
  const int lane = lane_id(), all = p.groups + p.B, per = (all + NT - 1) / NT;
  const int e0 = min(all, static_cast<int>(threadIdx.x) * per), e1 = min(all, e0 + per);
  uint32_t mine = 0;                // weight of the list
  uint32_t units = 0, items = 0;    // of own keys (OWN)
  int pairs = 0;
  PrefixEntry s = {};
#pragma unroll 1
  for (int e = e0; e < e1; ++e) {
    s = prefix_entry(p, e);
    const uint32_t n = static_cast<uint32_t>(s.items) * p.Hkv;
    if (OWN && e >= p.groups) {
      units += n * s.cnt;
      items += n;
    } else {
      pairs |= s.items > 0 && s.weight != kOneWeight;
      mine += n * s.cnt * s.weight;
    }
  }
  uint32_t incl = mine;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, h);
    if (lane >= h) incl += o;
    if (OWN) {
      units += __shfl_xor_sync(0xffffffffu, units, h);
      items += __shfl_xor_sync(0xffffffffu, items, h);
    }
  }
  constexpr int W = NT / 32;
  if (lane == 31) {
    sums[warp_id()] = incl;
    sums[W + warp_id()] = units;
    sums[2 * W + warp_id()] = items;
  }
  if (threadIdx.x == 0) plan[4] = 0;
  pairs = __syncthreads_or(pairs);
  uint32_t at = incl - mine, total = 0;
  units = items = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < static_cast<int>(warp_id())) at += sums[w];
    total += sums[w];
    units += sums[W + w];
    items += sums[2 * W + w];
  }
  // (starts that fall make groups overlap: more than there is room or time for)
  if (total > p.most) total = 0;
  const int CTAs = gridDim.x;
  int G = CTAs;
  if (OWN) {
    const float w = (static_cast<float>(units) + static_cast<float>(items)) * p.own_weight;
    if (items > 0)
      G = total > 0 ? min(max(static_cast<int>(CTAs * (total / (total + w))), 1), CTAs - 1) : 0;
    // (both CTAs of a cluster alike)
    if (items > 0 && total > 0 && CTAs > 2) G = min((G + 1) & ~1, CTAs - 2);
    if (threadIdx.x == 0) plan[5] = units <= kShortItem * items;
  }
  const PrefixShare r = {static_cast<int>(blockIdx.x) >= G, static_cast<int>(blockIdx.x) - (static_cast<int>(blockIdx.x) >= G ? G : 0),
                         CTAs - G};
  // Part c is [x0, x1); a unit that a border lies in is the next part's.  No part
  // may be shorter than the longest unit, so that none between two parts of an item
  // is without one; CTAs beyond that many parts have none.
  const uint32_t room = total / (pairs ? p.pair_weight : kOneWeight);
  const uint32_t n = room < static_cast<uint32_t>(G) ? max(room, 1u) : max(G, 1);
  const uint32_t q = total / n, rest = total - q * n, c = r.own ? n : r.c;
  const uint32_t x0 = c * q + min(c, rest), x1 = x0 + q + (c < rest ? 1 : 0);
  if (c < n && x1 > x0 && x0 - at < mine) {
#pragma unroll 1
    for (int e = e0; e < e1; ++e) {
      if (per > 1) s = prefix_entry(p, e);
      const uint32_t here = static_cast<uint32_t>(s.items) * s.cnt * p.Hkv * s.weight;
      if (x0 - at < here) {
        const int u = (x0 - at) / s.weight, item = u / s.cnt;
        plan[0] = e;
        plan[1] = item / s.items;
        plan[2] = item - plan[1] * s.items;
        plan[3] = u - item * s.cnt;
        plan[4] = min(x1 - at - u * s.weight, 1u << 30);
        *reinterpret_cast<PrefixEntry*>(plan + 8) = s;
        break;
      }
      at += here;
    }
  }
  __syncthreads();
  return r;
}

// Part c of G of the own keys' tiles, for a CTA of their own: its walk in plan {b, hkv,
// k, tiles}.  An item weighs a tile more than it has (its Q, and its end), before its
// first: tile k begins at k + 1, the first at 0.  No part is narrower than 2, so that
// none inside an item is without a tile.  Called by the whole CTA (NT threads).
template <int NT>
__device__ __forceinline__ void prefix_own_plan(const PagedOwnParams& p, int c, int G, uint32_t* sums, int* plan) {
  const int lane = lane_id(), per = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  uint32_t tiles = 0, items = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int cnt = paged_seq_of(p.lens[b], p).cnt;
    tiles += cnt * p.Hkv;
    items += cnt > 0 ? p.Hkv : 0;
  }
  uint32_t t_at = tiles, i_at = items;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, t_at, h), b = __shfl_up_sync(0xffffffffu, i_at, h);
    if (lane >= h) {
      t_at += a;
      i_at += b;
    }
  }
  constexpr int W = NT / 32;
  if (lane == 31) {
    sums[warp_id()] = t_at;
    sums[W + warp_id()] = i_at;
  }
  __syncthreads();
  t_at -= tiles;
  i_at -= items;
  uint32_t all_tiles = 0, total = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w < static_cast<int>(warp_id())) {
      t_at += sums[w];
      i_at += sums[W + w];
    }
    all_tiles += sums[w];
    total += sums[w] + sums[W + w];
  }
  const uint32_t n = min(static_cast<uint32_t>(G), max(total / 2, 1u));
  const uint32_t q = total / n, rest = total - q * n;
  // The part's first tile, and the next part's: the first at or behind a border.
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t part = c + i, x = part < n ? part * q + min(part, rest) : total;
    if (x >= total) {
      if (threadIdx.x == 0) plan[4 + i] = all_tiles;
      continue;
    }
    uint32_t ta = t_at, at = t_at + i_at;
    if (x - at >= tiles + items) continue;  // (in another thread's sequences)
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const uint32_t cnt = paged_seq_of(p.lens[b], p).cnt;
      const uint32_t all = cnt > 0 ? (cnt + 1) * p.Hkv : 0;
      if (x - at < all) {
        const uint32_t item = (x - at) / (cnt + 1), r = x - at - item * (cnt + 1);
        const uint32_t k = r == 0 ? 0 : max(r - 1, 1u);  // (cnt: the next item's first)
        plan[4 + i] = ta + item * cnt + k;
        break;
      }
      at += all;
      ta += cnt * p.Hkv;
    }
  }
  __syncthreads();
  const uint32_t first = plan[4], last = plan[5];
  if (threadIdx.x == 0) plan[3] = last - first;
  if (first < last && first - t_at < tiles) {
    uint32_t ta = t_at;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const uint32_t cnt = paged_seq_of(p.lens[b], p).cnt;
      if (first - ta < cnt * p.Hkv) {
        plan[0] = b;
        plan[1] = (first - ta) / cnt;
        plan[2] = (first - ta) % cnt;
        break;
      }
      ta += cnt * p.Hkv;
    }
  }
  __syncthreads();
}

template <bool OWN>
__device__ __forceinline__ PrefixWalk<OWN> prefix_walk(const PrefixParams& p, const int* plan) {
  PrefixWalk<OWN> w;
  w.rem = plan[4];
  w.left = 0;
  if (w.rem > 0) {
    w.e = plan[0];
    w.hkv = plan[1];
    w.it = plan[2];
    w.k = plan[3];
    w.s = *reinterpret_cast<const PrefixEntry*>(plan + 8);
    w.left = min(w.s.cnt - w.k, w.share());
  }
  return w;
}

// The roles of a CTA of the list; every warp of the CTA comes here and leaves
// together.
template <int D, bool BF16, bool OWN>
__device__ __forceinline__ void prefix_body(const CUtensorMap& tmQ, const CUtensorMap& tmOwnQ, const CUtensorMap& tmK,
                                            const CUtensorMap& tmV, const PrefixParams& p, uint8_t* gbase,
                                            uint32_t base, uint32_t tmem, AbortState* ab, const int* plan,
                                            int part) {
  using Ly = PrefixLayout<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr uint32_t IDESC_S = idesc_f16(BF16, 128, 128, false, false);
  constexpr uint32_t IDESC_PV = idesc_f16(BF16, 128, D, false, true);
  auto bar = [&](int i) -> uint32_t { return base + Ly::BAR_OFF + 8u * i; };
  unsigned int* err = device_error_word();
  const uint32_t warp = warp_id(), lane = lane_id();

  if (warp == 10) {
    // ------------------------------------------------------------ producer
    setmaxnreg_dec<Ly::REGS_OTHER>();
    const int page_log = 31 - __clz(p.page);  // (a page is a power of two)
    const int box_log = min(page_log, kOwnBoxLog), box = 1 << box_log, nbox = 128 >> box_log;
    const int per_batch = 32 >> (7 - box_log);
    uint32_t stage = 0, phase = 0, used = 0, slot = 0;
    uint32_t q_used = 0, q_odd = 0;  // bit t: slot t was filled; an odd number of times
    bool ok = true;
    const uint64_t first = policy_evict_first(), normal = policy_evict_normal();
#pragma unroll 1
    for (auto w = prefix_walk<OWN>(p, plan); ok && w.left > 0; w.next(p)) {
      const bool own = w.own(p), pair = w.pair(p);
      // What one item alone reads leaves the L2 first (64 sequences behind 32,768 keys 59
      // us, kept like other data 64; four items of 256 sequences 103, kept 96).
      const uint64_t policy = own || w.s.items == 1 ? first : normal;
      // Page ids of the next tiles, one box per lane, a batch ahead.
      const int max_pages = own ? p.max_pages : p.prefix_pages;
      const int* table = own ? p.table + static_cast<size_t>(w.e - p.groups) * p.max_pages
                             : p.ptable + static_cast<size_t>(w.e) * p.prefix_pages;
      auto pages = [&](int j) -> int {
        const int at = ((w.k + j) * 128 + static_cast<int>(lane) * box) >> page_log;
        return at < max_pages ? table[at] : -1;
      };
      int ids = 0, ahead = pages(0);
      // Q: both slots, or the two in turn.
      const int t0 = pair ? 0 : slot, t1 = pair ? 2 : slot + 1;
#pragma unroll 1
      for (int t = t0; t < t1; ++t) {
        if ((q_used >> t & 1u) && !prefix_wait(bar(Ly::B_QEMPTY + t), (q_odd >> t & 1u) ^ 1u, ab, err, 1101)) {
          ok = false;
          break;
        }
        q_used |= 1u << t;
        q_odd ^= 1u << t;
        if (lane == 0) {
          const CUtensorMap* map = own ? &tmOwnQ : &tmQ;
          mbar_arrive_expect_tx(bar(Ly::B_QFULL + t), Ly::KCH * static_cast<uint32_t>(own ? p.rows : p.tok * p.g) * 128u);
#pragma unroll
          for (int c = 0; c < Ly::KCH; ++c)
            tma_load_4d(base + Ly::Q_OFF + t * Ly::TILE + c * Ly::CHUNK, map, bar(Ly::B_QFULL + t), c * 64,
                        w.hkv * p.g, own ? 0 : w.token(p, pair ? t : 0), own ? w.e - p.groups : 0);
        }
        __syncwarp();
      }
      if (!pair) slot ^= 1;
      // K_j, V_j: one ring step each.
      int pid = 0, k0 = 0;
      uint32_t boxes = 0;
      bool go = false;
#pragma unroll 1
      for (int jv = 0; ok && jv < 2 * w.left; ++jv) {
        if ((jv & 1) == 0) {
          const int j = jv >> 1, x = j & (per_batch - 1);  // (a power of two)
          if (x == 0) {
            ids = ahead;
            if (j + per_batch < w.left) ahead = pages(j + per_batch);
          }
          pid = __shfl_sync(0xffffffffu, ids, (x * nbox + static_cast<int>(lane)) & 31);
          k0 = (w.k + j) * 128 + static_cast<int>(lane) * box;
          go = static_cast<int>(lane) < nbox && k0 < w.s.n;
          boxes = __popc(__ballot_sync(0xffffffffu, go));
        }
        if (!prefix_wait(bar(Ly::B_KVEMPTY + stage), phase ^ 1u, ab, err, 1102)) {
          ok = false;
          break;
        }
        if (lane == 0)
          mbar_arrive_expect_tx(bar(Ly::B_KVFULL + stage), boxes * box * static_cast<uint32_t>(D) * 2u);
        __syncwarp();
        if (go) {
          const uint32_t dst = base + Ly::RING_OFF + stage * Ly::TILE + lane * box * 128u;
          const CUtensorMap* map = jv & 1 ? &tmV : &tmK;
#pragma unroll
          for (int c = 0; c < Ly::KCH; ++c)
            tma_load_4d_hint(dst + c * Ly::CHUNK, map, bar(Ly::B_KVFULL + stage), c * 64, w.hkv, k0 & (p.page - 1), pid,
                             policy);
        }
        used |= 1u << stage;
        if (++stage == Ly::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      // Unwinding: let copies in flight land.  The newest use of a stage before
      // the write position has this round's parity, the others the last round's.
#pragma unroll 1
      for (int s = 0; s < Ly::STAGES + 2; ++s) {
        const int t = s - Ly::STAGES;
        if (t >= 0 ? q_used >> t & 1u : used >> s & 1u)
          mbar_wait_drain(bar(t >= 0 ? Ly::B_QFULL + t : Ly::B_KVFULL + s),
                          t >= 0 ? (q_odd >> t & 1u) ^ 1u : s < static_cast<int>(stage) ? phase : phase ^ 1u);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    setmaxnreg_dec<Ly::REGS_OTHER>();
    // Bits t: phases of slot t's Q, of tile t's P and O.
    uint32_t stage = 0, phase = 0, slot = 0, q_odd = 0, p_odd = 0, o_used = 0, o_odd = 0;
    bool ok = true;
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
      __syncwarp();
    };
    auto take = [&](uint32_t& at, unsigned int site) -> bool {
      at = stage;
      if (!prefix_wait(bar(Ly::B_KVFULL + stage), phase, ab, err, site)) return false;
      if (++stage == Ly::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      return true;
    };
    // Before the first PV of tile t: the last chunk's O has been read.
    auto o_free = [&](int t) -> bool {
      if ((o_used >> t & 1u) && !prefix_wait(bar(Ly::B_OEMPTY + t), (o_odd >> t & 1u) ^ 1u, ab, err, 1106)) return false;
      o_used |= 1u << t;
      o_odd ^= 1u << t;
      return true;
    };
    // V's rows behind the last key are zero, whatever their slots hold (P is zero
    // there, but 0 x NaN is not).
    auto clear = [&](uint32_t vs, int valid) {
#pragma unroll 1
      for (int i = valid * 8 + static_cast<int>(lane); i < 128 * 8; i += 32)
#pragma unroll
        for (int c = 0; c < Ly::KCH; ++c)
          reinterpret_cast<uint4*>(gbase + Ly::RING_OFF + vs * Ly::TILE + c * Ly::CHUNK)[i] = make_uint4(0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
    };
    auto s_products = [&](int t, uint64_t qd, uint64_t kd) {  // one thread
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        const uint64_t off = ((k >> 2) * Ly::CHUNK + (k & 3) * 32u) >> 4;
        mma_ss(tmem + Ly::TM_S + 128u * t, qd + off, kd + off, IDESC_S, k > 0 ? 1u : 0u);
      }
      tc_commit(bar(Ly::B_SFULL + t));
    };
    auto pv_products = [&](int t, uint64_t vd, int h, bool start) {  // one thread; half h of the keys
#pragma unroll
      for (int k = 0; k < 4; ++k)
        mma_ts(tmem + Ly::TM_O + static_cast<uint32_t>(D) * t, tmem + Ly::TM_S + 128u * t + 32u * h + 8u * k,
               vd + ((8192u * h + 2048u * k) >> 4), IDESC_PV, (!start || h > 0 || k > 0) ? 1u : 0u);
    };
    const uint64_t q0 = sdesc_sw128(base + Ly::Q_OFF, 16, 1024), k0 = sdesc_sw128(base + Ly::RING_OFF, 16, 1024),
                   v0 = sdesc_sw128(base + Ly::RING_OFF, Ly::CHUNK, 1024);
    constexpr uint64_t TILE16 = Ly::TILE >> 4;
#pragma unroll 1
    for (auto w = prefix_walk<OWN>(p, plan); ok && w.left > 0; w.next(p)) {
      const int n = w.left, last_valid = w.s.n - (w.k + n - 1) * 128;  // keys of the chunk's last tile
      uint32_t ks = 0, vs = 0;
      if (w.pair(p)) {
        // Two tiles.  Between a tile's PV and the other's nothing but its next S: what
        // this warp does in between, the tensor cores wait for.
        if (!prefix_wait(bar(Ly::B_QFULL), q_odd & 1u, ab, err, 1103) ||
            !prefix_wait(bar(Ly::B_QFULL + 1), q_odd >> 1 & 1u, ab, err, 1103) || !take(ks, 1104)) {
          ok = false;
          break;
        }
        q_odd ^= 3u;
        tc_fence_after();
        if (elect_one()) {
          s_products(0, q0, k0 + ks * TILE16);
          s_products(1, q0 + TILE16, k0 + ks * TILE16);
          tc_commit(bar(Ly::B_KVEMPTY + ks));
        }
        __syncwarp();
        if (!o_free(0) || !o_free(1)) { ok = false; break; }
#pragma unroll 1
        for (int j = 0; ok && j < n; ++j) {
          const bool more = j + 1 < n;
          if (!take(vs, 1104) || (more && !take(ks, 1105))) { ok = false; break; }
          if (!more && last_valid < 128) clear(vs, last_valid);
          const uint64_t vd = v0 + vs * TILE16, kd = k0 + ks * TILE16;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!prefix_wait(bar(Ly::B_PFULL + 2 * t), p_odd >> t & 1u, ab, err, 1107)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) pv_products(t, vd, 0, j == 0);
            __syncwarp();
            if (!prefix_wait(bar(Ly::B_PFULL + 2 * t + 1), p_odd >> t & 1u, ab, err, 1108)) { ok = false; break; }
            tc_fence_after();
            if (elect_one()) {
              pv_products(t, vd, 1, false);
              if (!more) tc_commit(bar(Ly::B_OFULL + t));
              if (t == 1) tc_commit(bar(Ly::B_KVEMPTY + vs));
              if (more) {
                s_products(t, q0 + t * TILE16, kd);
                if (t == 1) tc_commit(bar(Ly::B_KVEMPTY + ks));
              }
            }
            __syncwarp();
          }
          p_odd ^= 3u;
        }
        if (!ok) break;
        commit(Ly::B_QEMPTY);
        commit(Ly::B_QEMPTY + 1);
        continue;
      }
      // One tile: step j is S of unit j, which is one group's, then PV of unit j - 1,
      // the other's.
      if (!prefix_wait(bar(Ly::B_QFULL + slot), q_odd >> slot & 1u, ab, err, 1103)) { ok = false; break; }
      q_odd ^= 1u << slot;
      const uint64_t qd = q0 + slot * TILE16;
#pragma unroll 1
      for (int j = 0; ok && j <= n; ++j) {
        if ((j > 0 && !take(vs, 1104)) || (j < n && !take(ks, 1105))) { ok = false; break; }
        tc_fence_after();
        if (j < n) {
          if (elect_one()) {
            s_products(j & 1, qd, k0 + ks * TILE16);
            tc_commit(bar(Ly::B_KVEMPTY + ks));
          }
          __syncwarp();
        }
        if (j == 0) continue;
        if (j == n && last_valid < 128) clear(vs, last_valid);
        const int t = (j - 1) & 1;
        if (j < 3 && !o_free(t)) { ok = false; break; }
        const uint64_t vd = v0 + vs * TILE16;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!prefix_wait(bar(Ly::B_PFULL + 2 * t + h), p_odd >> t & 1u, ab, err, 1109)) { ok = false; break; }
          tc_fence_after();
          if (elect_one()) {
            pv_products(t, vd, h, j < 3);
            if (h == 1) {
              if (j + 1 >= n) tc_commit(bar(Ly::B_OFULL + t));  // the group's last step
              tc_commit(bar(Ly::B_KVEMPTY + vs));
            }
          }
          __syncwarp();
        }
        p_odd ^= 1u << t;
      }
      if (!ok) break;
      commit(Ly::B_QEMPTY + slot);
      slot ^= 1;
    }
    commit(Ly::B_DONE);
    mbar_wait_drain(bar(Ly::B_DONE), 0);
  } else if (warp >= 8) {
    setmaxnreg_dec<Ly::REGS_OTHER>();
  } else {
    // ------------------------------------------------------------ softmax
    setmaxnreg_inc<Ly::REGS_SOFTMAX>();
    const int t = warp >> 2;          // two tiles: the tile; one: steps j % 2 = t
    const int r = threadIdx.x & 127;  // row of the tile == TMEM lane
    const uint32_t lane_off = ((warp & 3u) * 32u) << 16;
    const uint32_t tS = tmem + lane_off + Ly::TM_S + 128u * t;
    const uint32_t tO = tmem + lane_off + Ly::TM_O;
    const float sl2 = p.sl2;
    float* mate = reinterpret_cast<float*>(gbase + Ly::MATE_OFF);
    uint32_t s_cnt = 0, o_cnt[2] = {0, 0}, mates = 0;
    bool ok = true;
#pragma unroll 1
    for (auto w = prefix_walk<OWN>(p, plan); ok && w.left > 0; w.next(p)) {
      const bool pair = w.pair(p), own = w.own(p);
      const int rows = w.rows(p, pair ? t : 0), step = pair ? 1 : 2;
      const bool live = r < rows, some = static_cast<int>((warp & 3u) * 32u) < rows;  // (some: this warp has a row)
      // Own keys come last and all have as many rows: warps without one are done, and
      // the first warp arrives for them.
      if (own && !some) break;
      const uint32_t arrive = own && (warp & 3u) == 0 ? 4 - (p.rows - 1) / 32 : 1;
      const int seen = own ? w.s.n - p.Lq + 1 + (r * p.ginv >> 16) : w.s.n;  // keys this row sees
      float m = -INFINITY, l = 0.f;
#pragma unroll 1
      for (int j = pair ? 0 : t; j < w.left; j += step) {
        if (!prefix_wait(bar(Ly::B_SFULL + t), s_cnt & 1, ab, err, 1110)) { ok = false; break; }
        ++s_cnt;
        if (!some) {
          if (lane == 0) {
            mbar_arrive(bar(Ly::B_PFULL + 2 * t));
            mbar_arrive(bar(Ly::B_PFULL + 2 * t + 1));
          }
          continue;
        }
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
        const int lim = seen - (w.k + j) * 128;
        if (__any_sync(0xffffffffu, lim < 128)) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= lim) sr[c] = __float_as_uint(-INFINITY);
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
        if (j < step) {
          m = m_new;
        } else if (__any_sync(0xffffffffu, live && (m_new - m) * sl2 > 8.0f)) {
          // Some row's maximum grew by more than 2^8: this warp's rows move theirs.
          // (What the lanes without a row see is left of other chunks.)
          // (A row that has seen nothing so far has O = l = 0.)
          if (m_new != -INFINITY) alpha = ex2((m - m_new) * sl2);
          m = m_new;
          rescale = true;
        }
        // Half h of P is in TMEM.  Before the first, O is scaled if the maximum
        // moved (the commit behind this S covers the tile's, or group's, last PV).
        auto p_ready = [&](int h) {
          if (h == 0 && rescale) {
            // (16 at a time, in a loop: beside 128 scores more registers would be spilled)
#pragma unroll 1
            for (int cc = 0; cc < D / 16; ++cc) {
              uint32_t o[16];
              tmem_ld16(tO + D * t + 16 * cc, o);
              tmem_ld_wait16(o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
              tmem_st16(tO + D * t + 16 * cc, o);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) prefix_arrive(bar(Ly::B_PFULL + 2 * t + h), arrive);
        };
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
      const bool two = !pair && w.left > 1;  // one tile's O in two parts
      const uint32_t oc0 = o_cnt[0], oc1 = o_cnt[1];
      ++o_cnt[0];  // (every chunk fills O_0, who waits for it or not)
      if (pair || two) ++o_cnt[1];
      float f0 = 1.f, f1 = 0.f;              // factors of O_t, or O_0 and O_1
      if (!pair) {
        if (t == 0) {
          // Warps 4-7 finish the tile.
          if (mates > 0 && !prefix_wait(bar(Ly::B_MEMPTY), (mates - 1) & 1, ab, err, 1111)) { ok = false; break; }
          ++mates;
          mate[r] = m;
          mate[128 + r] = l;
          __syncwarp();
          if (lane == 0) prefix_arrive(bar(Ly::B_MFULL), arrive);
          continue;
        }
        if (!prefix_wait(bar(Ly::B_MFULL), mates & 1, ab, err, 1112)) { ok = false; break; }
        ++mates;
        const float m0 = mate[r], l0 = mate[128 + r], top = fmaxf(m0, m);
        __syncwarp();
        if (lane == 0) prefix_arrive(bar(Ly::B_MEMPTY), arrive);
        f0 = m0 == -INFINITY ? 0.f : ex2((m0 - top) * sl2);
        f1 = m == -INFINITY ? 0.f : ex2((m - top) * sl2);
        l = l0 * f0 + l * f1;
        m = top;
      }
      const int o0 = pair ? t : 0;
      if (!prefix_wait(bar(Ly::B_OFULL + o0), (o0 ? oc1 : oc0) & 1, ab, err, 1113) ||
          (two && !prefix_wait(bar(Ly::B_OFULL + 1), oc1 & 1, ab, err, 1114))) {
        ok = false;
        break;
      }
      const int item = own ? (w.e - p.groups) * p.Hkv + w.hkv
                           : prefix_first_item(p, w.s, w.e) + w.hkv * w.s.items + w.it;
      if (some) {
        tc_fence_after();
        const float inv = l > 0.f ? 1.f / l : 0.f;
        f0 *= inv;
        f1 *= inv;
        const uint32_t row0 = own ? static_cast<uint32_t>(item + part) * p.rows
                                : prefix_first_row(p, w.s, w.hkv, w.it, part) + (pair && t ? p.tok * p.g : 0);
        const float lse = l == 0.f ? -INFINITY : m * sl2 + __log2f(l);  // (NaN stays NaN)
        if (live) (own ? p.own_lse : p.part_lse)[row0 + r] = lse;
        float4* dst = reinterpret_cast<float4*>(own ? p.own_o : p.part_o) + static_cast<size_t>(own ? row0 + r : row0) * (D / 4) +
                      (own ? 0 : r);
        const int pitch = own ? 1 : w.rows(p, pair ? t : 0);
#pragma unroll 1
        for (int cc = 0; cc < D / 32; ++cc) {
          uint32_t o[32];
          tmem_ld32(tO + D * o0 + 32 * cc, o);
          tmem_ld_wait32(o);
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(o[i]) * f0;
          if (two) {
            tmem_ld32(tO + D + 32 * cc, o);
            tmem_ld_wait32(o);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = fmaf(__uint_as_float(o[i]), f1, v[i]);
          }
          if (live) {
#pragma unroll
            for (int i = 0; i < 8; ++i, dst += pitch)
              *dst = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        tc_fence_before();
      }
      // The item's first and last part, for the join.
      if (r == 0 && (!pair || t == 0)) {
        int* ends = p.ends + 2 * (own ? static_cast<size_t>(p.items) + item : static_cast<size_t>(item));
        if (w.k == 0) ends[0] = part;
        if (w.k + w.left == w.s.cnt) ends[1] = part;
      }
      __syncwarp();
      if (lane == 0) {
        prefix_arrive(bar(Ly::B_OEMPTY + o0), arrive);
        if (two) prefix_arrive(bar(Ly::B_OEMPTY + 1), arrive);
      }
    }
  }
}

// Shared memory of a CTA: the layout of its role, behind both the common words.
template <int D, int R>
struct PrefixShared {
  static constexpr uint32_t OWN_USED = PagedLayout<D, R == 0 ? 8 : R>::SMEM_USED;
  static constexpr uint32_t PREFIX_USED = PrefixLayout<D>::USED;
  static constexpr uint32_t OFF = R > 0 && OWN_USED > PREFIX_USED ? (OWN_USED + 15) / 16 * 16 : (PREFIX_USED + 15) / 16 * 16;
  // plan [16], lens [32], sums [3][12], tmem slot, abort flag
  static constexpr uint32_t PLAN = OFF, LENS = OFF + 64, SUMS = OFF + 192, SLOT = OFF + 336, FLAG = OFF + 340;
  static constexpr uint32_t ALLOC = OFF + 352 + 1024;
  static constexpr int NTHREADS = PrefixLayout<D>::NTHREADS;
  static_assert(ALLOC <= 232448, "shared memory");
};

// R: query rows a thread of the paged decode's roles takes (g * Lq rounded up to
// 8, 16 or 32), or 0: own keys are in the list of prefixes.
template <int D, bool BF16, int R>
__global__ void __launch_bounds__(384, 1)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmOwnQ,
                     const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const PrefixParams p, const PagedOwnParams o) {
  using Sh = PrefixShared<D, R>;
  constexpr int NT = Sh::NTHREADS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Sh::SLOT);
  AbortState* ab = reinterpret_cast<AbortState*>(gbase + Sh::FLAG);
  int* plan = reinterpret_cast<int*>(gbase + Sh::PLAN);
  uint32_t* sums = reinterpret_cast<uint32_t*>(gbase + Sh::SUMS);
  const uint32_t warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) ab->flag = 0;
  if (warp == 10 && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmOwnQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 9) {
    tmem_alloc(base + Sh::SLOT, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  pdl_wait();
  pdl_launch_dependents();  // (now: what runs behind it may read what was there before this kernel)
  const PrefixShare mine = prefix_plan<NT, R != 0>(p, sums, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (R == 0 || !mine.own) {
    using Ly = PrefixLayout<D>;
    if (threadIdx.x < Ly::NBAR) mbar_init(base + Ly::BAR_OFF + 8u * threadIdx.x, Ly::arrivals(threadIdx.x));
    fence_barrier_init();
    __syncthreads();
    prefix_body<D, BF16, R == 0>(tmQ, tmOwnQ, tmK, tmV, p, gbase, base, tmem, ab, plan, mine.c);
  } else if constexpr (R != 0) {
    using Ly = PagedLayout<D, R>;
    // Query rows past g * Lq, and P rows no thread writes, are zero.
#pragma unroll 1
    for (uint32_t i = threadIdx.x; i < (Ly::QS * Ly::QT + Ly::PB * Ly::PT) / 16u; i += NT)
      reinterpret_cast<uint4*>(gbase + Ly::Q_OFF)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
#pragma unroll 1
    for (int i = threadIdx.x; i < Ly::NBAR; i += NT) mbar_init(base + Ly::BAR_OFF + 8u * i, Ly::arrivals(i));
    fence_barrier_init();
    const bool brief = plan[5] != 0;
    int* lens_s = reinterpret_cast<int*>(gbase + Sh::LENS);
    const int len = (o.B <= 32 && static_cast<int>(lane) < o.B) ? o.lens[lane] : 0;
    if (warp == 0) lens_s[lane] = len;
    __syncthreads();  // (plan is read, and written again)
    prefix_own_plan<NT>(o, mine.c, mine.G, sums, plan);
    paged_body<D, BF16, R>(tmOwnQ, tmK, tmV, o, gbase, base, tmem, ab, plan, o.B <= 32 ? lens_s : o.lens, mine.c, mine.G,
                                 brief);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

struct PrefixJoinParams {
  PrefixParams p;
  void* O;     // [B, Lq, H, D]
  float* LSE;  // [B, H, Lq], natural log
  int G;       // CTAs of fa_prefix_kernel
};

// Join each row's partials: those of its prefix's chunks and of its own keys'.
// SP threads join 4 dims of one row, each every SP-th of the prefix's partials; the
// lanes run over the g heads of a K/V head, whose rows lie together in a prefix's
// partial, then over the dims.  Block (x, y): token and K/V head x, the 128 / SP
// cells from y * 128 / SP on.  Bound by latency: two loads that depend on one
// another (an item's parts, the partials) behind fa_prefix_kernel's end, so what does
// not depend goes out together, and SP is 1 where a row has few partials.
template <int D, bool BF16, int SP>
__global__ void __launch_bounds__(128) fa_prefix_join_kernel(const PrefixJoinParams a) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int C = SP == 1 ? 6 : 5, CELLS = 32 / SP;  // partials at a time; cells of a warp
  const PrefixParams& p = a.p;
  const int pair = blockIdx.x;
  const int tk = pair / p.Hkv, hkv = pair - tk * p.Hkv;
  const int b = tk / p.Lq, ql = tk - b * p.Lq;
  const int lane = lane_id(), sp = lane / CELLS;
  const int cell = (blockIdx.y * 4 + static_cast<int>(warp_id())) * CELLS + lane % CELLS;
  const int d4 = cell / p.g, hg = cell - d4 * p.g;
  const bool in = d4 < D / 4;
  pdl_launch_dependents();
  // Lengths and starts are from before fa_prefix_kernel, whose CTAs let this one begin
  // once all before it is done: they are read while it runs.
  const int own_n = min(max(__ldcg(p.lens + b), 0), p.cap);
  const int own_item = b * p.Hkv + hkv;
  // The sequence's group.
  int grp = 0;
  if (p.groups > 1) {
    int lo = 0, hi = p.groups;  // the last group that starts at or before b
#pragma unroll 1
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldcg(p.starts + mid) <= b) lo = mid;
      else hi = mid;
    }
    grp = lo;
  }
  const PrefixEntry s = prefix_entry(p, grp);
  const bool pad = own_n - p.Lq + ql < 0;
  pdl_wait();
  const int2 oe = __ldcg(reinterpret_cast<const int2*>(p.ends) + p.items + own_item);
  float mx = -INFINITY, den = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](float lse, const float4& o) {
    const float m = fmaxf(mx, lse);
    // (each for itself: a NaN LSE has no part in m, but its weight is NaN)
    const float old = mx == -INFINITY ? 0.f : ex2(mx - m), w = lse == -INFINITY ? 0.f : ex2(lse - m);
    den = fmaf(den, old, w);
    acc.x = fmaf(acc.x, old, w * o.x);
    acc.y = fmaf(acc.y, old, w * o.y);
    acc.z = fmaf(acc.z, old, w * o.z);
    acc.w = fmaf(acc.w, old, w * o.w);
    mx = m;
  };
  if (!pad && in) {
    // The chunks of the row's tile.
    int n = 0, row = 0, pitch = 0;
    uint32_t row0 = 0;
    if (s.items > 0 && tk >= s.t0 && tk < s.t1) {
      const int tile = (tk - s.t0) / p.tok;
      row = (tk - s.t0 - tile * p.tok) * p.g + hg;
      pitch = min(p.tok, s.t1 - s.t0 - tile * p.tok) * p.g;
      const int item = prefix_first_item(p, s, grp) + hkv * s.items + (tile >> 1);
      const int2 e = __ldcg(reinterpret_cast<const int2*>(p.ends) + item);
      const int c0 = min(max(e.x, 0), a.G - 1);  // (in bounds even where starts fall)
      n = min(max(e.y, c0), a.G - 1) - c0 + 1;
      row0 = prefix_first_row(p, s, hkv, tile >> 1, c0) + (tile & 1 ? p.tok * p.g : 0);
    }
    // The own keys' first partial, nearly always the only one, beside them.
    const int o0 = min(max(oe.x, 0), a.G - 1), o1 = min(max(oe.y, o0), a.G - 1);
    const size_t own_at = static_cast<size_t>(own_item + o0) * p.rows + ql * p.g + hg;
    const float4* own_o = reinterpret_cast<const float4*>(p.own_o) + d4;
    const float ol = __ldcg(p.own_lse + own_at);
    const float4 oo = __ldcg(own_o + own_at * (D / 4));
    const float* lses = p.part_lse + row0 + row;
    const float4* os = reinterpret_cast<const float4*>(p.part_o) + static_cast<size_t>(row0) * (D / 4) + d4 * pitch + row;
#pragma unroll 1
    for (int q0 = sp; q0 < n; q0 += SP * C) {
      float ls[C];
      float4 o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int q = q0 + SP * c;
        ls[c] = -INFINITY;
        o[c] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (q < n) {
          ls[c] = __ldcg(lses + static_cast<size_t>(q) * 256);
          o[c] = __ldcg(os + static_cast<size_t>(q) * (256 * (D / 4)));
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c) add(ls[c], o[c]);
    }
    if (sp == 0) {
      add(ol, oo);
#pragma unroll 1
      for (int c = 1; c <= o1 - o0; ++c)
        add(__ldcg(p.own_lse + own_at + static_cast<size_t>(c) * p.rows),
            __ldcg(own_o + (own_at + static_cast<size_t>(c) * p.rows) * (D / 4)));
    }
  }
#pragma unroll
  for (int h = CELLS; h < 32; h <<= 1) {
    const float om = __shfl_xor_sync(0xffffffffu, mx, h), od = __shfl_xor_sync(0xffffffffu, den, h);
    const float4 oa = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, h), __shfl_xor_sync(0xffffffffu, acc.y, h),
                                  __shfl_xor_sync(0xffffffffu, acc.z, h), __shfl_xor_sync(0xffffffffu, acc.w, h));
    const float m = fmaxf(mx, om);
    const float u = mx == -INFINITY ? 0.f : ex2(mx - m), v = om == -INFINITY ? 0.f : ex2(om - m);
    // (a side that has seen NaN alone has no maximum: its den carries it)
    den = (mx == -INFINITY ? den : den * u) + (om == -INFINITY ? od : od * v);
    acc.x = acc.x * u + oa.x * v;
    acc.y = acc.y * u + oa.y * v;
    acc.z = acc.z * u + oa.z * v;
    acc.w = acc.w * u + oa.w * v;
    mx = m;
  }
  if (!in || sp != 0) return;
  const int h = hkv * p.g + hg;
  const float inv = den > 0.f ? 1.f / den : (den == 0.f ? 0.f : den);  // (NaN stays NaN)
  *reinterpret_cast<uint2*>(reinterpret_cast<T*>(a.O) + (static_cast<size_t>(tk) * p.H + h) * D + 4 * d4) =
      make_uint2(pack2<T>(acc.x * inv, acc.y * inv), pack2<T>(acc.z * inv, acc.w * inv));
  if (d4 == 0)
    a.LSE[(static_cast<size_t>(b) * p.H + h) * p.Lq + ql] =
        den == 0.f ? -INFINITY : (mx + __log2f(den)) * 0.6931471805599453f;
}

}  // namespace fa
