// Decoding against a paged key/value cache: a few new tokens per sequence,
// one length per sequence, keys and values in pages anywhere in a pool.
//
// Mathematics: the softmax of the dense forward over the visible keys of each
// sequence.  A (sequence, K/V head) is one item; the keys of an item come in
// 128-key tiles; tiles of one item that different CTAs process give partial
// (O_s, LSE_s) in fp32, joined by LSE = ln sum exp(LSE_s) and
// O = sum exp(LSE_s - LSE) O_s.
//
// Bound by the read of K and V, so the kernel is built to keep that read
// going without a pause:
//   - one persistent CTA per SM.  The tiles of all items form one list (item by
//     item); CTA c takes the c-th of G equal contiguous parts of it, whatever
//     the lengths are.  Lengths are read on the device: every CTA scans them
//     once.  An item inside one CTA is written directly; only items cut by a
//     part's border leave partials, at most two per CTA, so the workspace does
//     not grow with the lengths.
//   - one TMA ring of K and V tiles runs through the whole part, across items.
//   - the products are transposed, S^T = K Q^T and O^T = V^T P^T: the 128 keys
//     (or the head dims) fill the 128 rows of the MMA and the g * Lq packed
//     query rows are its N, 16 at least.  A thread then owns one key and only
//     as many scores as there are query rows, where Q K^T with the queries in
//     128 padded rows makes every warp exponentiate 128 keys for a handful of
//     live lanes.
// Warps 0-3: softmax (thread = key of the tile), epilogue (thread = head dim);
// warp 4: TMA producer; warp 5: TMEM allocation and MMA issue.
// Row maxima are reduced over the 32 keys of a warp by a halving exchange
// (lane r ends with row r), then over the four warps through shared memory;
// a row's max moves only when it grew by more than 2^8 in exp2 units, as in
// the dense forward.
// Keys that no query sees (behind the length, before the window) may lie in
// pages that were never written: their scores are replaced, not multiplied,
// and their V rows are set to zero in shared memory before the PV product.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "fwd.cuh"  // pack2
#include "ptx.cuh"

namespace fa {

// Meta record each CTA of the decode kernel leaves for the kernels after it.
struct PagedMeta {
  long long t0;     // first tile of its part in the list of all tiles
  int n;            // tiles in its part (0: nothing)
  int b, hkv, k;    // first item and the first tile visited of it
  int first_open;   // 1: the first item goes on in a later CTA
  int last_bh;      // last item (b * Hkv + hkv) if it starts here and goes on later, else -1
  int last_slot;    // its partial slot
  int pad[7];
};
static_assert(sizeof(PagedMeta) == 64, "one 64-byte record per CTA");

struct PagedParams {
  const int* table;  // [B, max_pages]
  const int* lens;   // [B]
  void* O;           // [B, Lq, H, D]
  float* LSE;        // [B, H, Lq] natural log
  PagedMeta* meta;   // [G]
  float* part_o;     // [2 G, rows, D]
  float* part_lse;   // [2 G, rows], log2 units
  float* scores;     // [tiles, rows, 128] raw scores for the weights, or NULL
  int B, Lq, H, Hkv, g, rows;
  int page, max_pages, cap;  // cap = max_pages * page
  int window, sinks;         // window 0: none (then sinks 0)
  float sl2;                 // log2(e) / sqrt(D)
};

// The tiles one sequence's items visit: ns sink tiles, then lo, lo + 1, ....
struct PagedSeq {
  int n;    // length
  int wlo;  // first key the earliest query's window reaches
  int ns, lo, cnt;
};

__device__ __forceinline__ PagedSeq paged_seq(int b, const PagedParams& p) {
  PagedSeq s;
  s.n = min(max(p.lens[b], 0), p.cap);
  s.wlo = p.window ? max(max(s.n - p.Lq, 0) - p.window + 1, 0) : 0;
  s.lo = s.wlo >> 7;
  s.ns = min((min(p.sinks, s.n) + 127) >> 7, s.lo);
  s.cnt = s.n > 0 ? s.ns + ((s.n + 127) >> 7) - s.lo : 0;
  return s;
}

// Walk over the tiles of one CTA's part.
struct PagedWalk {
  int b, hkv, k;  // item and tile index within its list
  int rem;        // tiles left in the part, this one included
  int item;       // items begun before this one in the part
  bool first;     // first tile of its item in this part
  PagedSeq s;

  __device__ __forceinline__ int tile() const { return k < s.ns ? k : s.lo + k - s.ns; }
  __device__ __forceinline__ bool last() const { return rem == 1 || k + 1 == s.cnt; }
  __device__ __forceinline__ void next(const PagedParams& p) {
    --rem;
    ++k;
    first = false;
    if (rem > 0 && k == s.cnt) {
      k = 0;
      first = true;
      ++item;
      if (++hkv == p.Hkv) {
        hkv = 0;
        do {
          ++b;
          if (b >= p.B) {
            rem = 0;
            return;
          }
          s = paged_seq(b, p);
        } while (s.cnt == 0);
      }
    }
  }
};

// R: query rows a thread processes (g * Lq rounded up); N: MMA columns.
template <int D, int R>
struct PagedLayout {
  static constexpr int N = R < 16 ? 16 : R;
  static constexpr int KCH = D / 64;
  static constexpr uint32_t CHUNK = 128u * 128u;  // 128 keys x 64 columns
  static constexpr uint32_t TILE = KCH * CHUNK;
  static constexpr uint32_t QCH = N * 128u;       // N rows x 64 columns
  static constexpr uint32_t QT = KCH * QCH;
  static constexpr uint32_t PT = 2 * QCH;         // N rows x 128 keys
  static constexpr int QS = (D == 128 && N == 128) ? 1 : 2;
  static constexpr int STAGES =
      D == 128 ? (N == 16 ? 6 : N == 32 ? 5 : N == 64 ? 4 : 3) : (N <= 32 ? 12 : N == 64 ? 10 : 7);
  static constexpr uint32_t RING_OFF = 0;
  static constexpr uint32_t Q_OFF = STAGES * TILE;
  static constexpr uint32_t P_OFF = Q_OFF + QS * QT;
  static constexpr uint32_t ST_OFF = P_OFF + 2 * PT;  // wmax[2][4][N], mb[4][N], aux[4][N]
  static constexpr uint32_t BAR_OFF = ST_OFF + 16u * N * 4u;
  static constexpr int B_QFULL = 0, B_QEMPTY = QS, B_KVFULL = 2 * QS, B_KVEMPTY = B_KVFULL + STAGES,
                       B_SFULL = B_KVEMPTY + STAGES, B_PFULL = B_SFULL + 2, B_PVDONE = B_PFULL + 2,
                       B_OFULL = B_PVDONE + 2, B_OEMPTY = B_OFULL + 2, B_XMAX = B_OEMPTY + 2,
                       B_XSUM = B_XMAX + 1, B_DONE = B_XSUM + 1, NBAR = B_DONE + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;  // tmem slot, abort flag, plan
  static constexpr uint32_t USED = MISC_OFF + 128;
  // At D = 64 the PV product still takes 128 rows of V^T; rows 64-127 come
  // from the 16 KB behind the tile and their results are never read.  Behind
  // the last ring stage that much must still be shared memory of this CTA.
  static constexpr uint32_t SMEM_USED = (D == 64 && USED < Q_OFF + CHUNK) ? Q_OFF + CHUNK : USED;
  static constexpr uint32_t SMEM_ALLOC = SMEM_USED + 1024;
  static constexpr uint32_t TM_S = 0, TM_O = 2 * N;
  static constexpr uint32_t TMEM_COLS = 4 * N;
  static constexpr int NTHREADS = 192;
  static_assert(SMEM_ALLOC <= 232448, "shared memory");
  static_assert(NBAR * 8 % 8 == 0 && BAR_OFF % 8 == 0 && ST_OFF % 16 == 0, "alignment");
};

// Reduce x[i] (row i of CW) over the warp's lanes: lane r gets row r % CW.
template <int CW, bool MAX>
__device__ __forceinline__ float paged_rows_reduce(float (&x)[CW], uint32_t lane) {
  auto op = [](float a, float b) { return MAX ? fmaxf(a, b) : a + b; };
#pragma unroll
  for (int h = CW / 2; h >= 1; h >>= 1) {
    const bool up = (lane & h) != 0;
#pragma unroll
    for (int i = 0; i < h; ++i) {
      const float keep = up ? x[i + h] : x[i], send = up ? x[i] : x[i + h];
      x[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, h));
    }
  }
  float v = x[0];
#pragma unroll
  for (int h = CW; h < 32; h <<= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, h));
  return v;
}

// Part of CTA blockIdx.x of the list of all tiles, computed by the whole CTA
// (NT threads; sums: NT / 32 + 1 long longs, out: 4 ints of shared memory).
// Returns the walk's start in `out` {b, hkv, k, n} and t0.
template <int NT>
__device__ __forceinline__ long long paged_plan(const PagedParams& p, int c, int G,
                                                long long* sums, int* out) {
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += static_cast<long long>(paged_seq(b, p).cnt) * p.Hkv;
  long long incl = mine;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, h);
    if (lane_id() >= static_cast<uint32_t>(h)) incl += o;
  }
  if (lane_id() == 31) sums[warp_id()] = incl;
  if (threadIdx.x == 0) out[3] = 0;
  __syncthreads();
  long long before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < static_cast<int>(warp_id())) before += sums[w];
    total += sums[w];
  }
  const long long t0 = total * c / G, t1 = total * (c + 1) / G;
  if (t1 > t0 && t0 >= before && t0 < before + mine) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const int cnt = paged_seq(b, p).cnt;
      const long long all = static_cast<long long>(cnt) * p.Hkv;
      if (t0 < at + all) {
        const int off = static_cast<int>(t0 - at);
        out[0] = b;
        out[1] = off / cnt;
        out[2] = off % cnt;
        out[3] = static_cast<int>(t1 - t0);
        break;
      }
      at += all;
    }
  }
  __syncthreads();
  return t0;
}

__device__ __forceinline__ PagedWalk paged_walk(const PagedParams& p, const int* plan) {
  PagedWalk w;
  w.rem = plan[3];
  w.b = plan[0];
  w.hkv = plan[1];
  w.k = plan[2];
  w.item = 0;
  w.first = true;
  if (w.rem > 0) w.s = paged_seq(w.b, p);
  return w;
}

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(192, 1)
    fa_paged_decode_kernel(const __grid_constant__ CUtensorMap tmQ,
                           const __grid_constant__ CUtensorMap tmK,
                           const __grid_constant__ CUtensorMap tmV, const PagedParams p) {
  using Ly = PagedLayout<D, R>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr int N = Ly::N;
  constexpr int CW = R < 32 ? R : 32, NCH = R / CW;
  constexpr uint32_t IDESC_S = idesc_f16(BF16, 128, N, false, false);
  constexpr uint32_t IDESC_PV = idesc_f16(BF16, 128, N, true, false);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + Ly::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Ly::MISC_OFF);
  AbortState* ab = reinterpret_cast<AbortState*>(gbase + Ly::MISC_OFF + 8);
  int* plan = reinterpret_cast<int*>(gbase + Ly::MISC_OFF + 16);
  long long* sums = reinterpret_cast<long long*>(gbase + Ly::MISC_OFF + 32);
  unsigned int* err = device_error_word();
  const uint32_t warp = warp_id(), lane = lane_id();

  pdl_launch_dependents();
  // Query rows past g * Lq, and P rows no thread writes, are zero.
  for (uint32_t i = threadIdx.x; i < (Ly::QS * Ly::QT + 2 * Ly::PT) / 16u; i += Ly::NTHREADS)
    reinterpret_cast<uint4*>(gbase + Ly::Q_OFF)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  if (threadIdx.x == 0) {
    for (int s = 0; s < Ly::QS; ++s) {
      mbar_init(bar(Ly::B_QFULL + s), 1);
      mbar_init(bar(Ly::B_QEMPTY + s), 1);
    }
    for (int s = 0; s < Ly::STAGES; ++s) {
      mbar_init(bar(Ly::B_KVFULL + s), 1);
      mbar_init(bar(Ly::B_KVEMPTY + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(Ly::B_SFULL + i), 1);
      mbar_init(bar(Ly::B_PFULL + i), 4);
      mbar_init(bar(Ly::B_PVDONE + i), 1);
      mbar_init(bar(Ly::B_OFULL + i), 1);
      mbar_init(bar(Ly::B_OEMPTY + i), 4);
    }
    mbar_init(bar(Ly::B_XMAX), 4);
    mbar_init(bar(Ly::B_XSUM), 4);
    mbar_init(bar(Ly::B_DONE), 1);
    ab->flag = 0;
    fence_barrier_init();
  }
  if (warp == 5) {
    tmem_alloc(base + Ly::MISC_OFF, Ly::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  const long long t0 = paged_plan<Ly::NTHREADS>(p, blockIdx.x, gridDim.x, sums, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 4) {
    // ------------------------------------------------------------ producer
    // Ring order: K_0, then K_{i+1}, V_i per tile.  Lane j loads the j-th box
    // (a page, or 128 rows of one) of the tile.
    const int box = min(p.page, 128), nbox = 128 / box;
    uint32_t stage = 0, phase = 0, used = 0, qcnt = 0;
    bool ok = true;
    const uint64_t stream = policy_evict_first();
    // Boxes that hold a key some query sees; the others are not loaded.
    auto mine = [&](const PagedWalk& w) -> bool {
      const int k0 = w.tile() * 128 + static_cast<int>(lane) * box;
      return static_cast<int>(lane) < nbox && k0 < w.s.n && (k0 + box > w.s.wlo || k0 < p.sinks);
    };
    auto page_of = [&](const PagedWalk& w) -> int {
      const int k0 = w.tile() * 128 + static_cast<int>(lane) * box;
      return mine(w) ? p.table[static_cast<size_t>(w.b) * p.max_pages + k0 / p.page] : -1;
    };
    auto load = [&](const CUtensorMap* map, const PagedWalk& w, int pid) -> bool {
      if (!mbar_wait_warp(bar(Ly::B_KVEMPTY + stage), phase ^ 1u, ab, err, 1001)) return false;
      const bool go = mine(w);
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, go));
      if (lane == 0)
        mbar_arrive_expect_tx(bar(Ly::B_KVFULL + stage), boxes * box * static_cast<uint32_t>(D) * 2u);
      __syncwarp();
      if (go) {
        const int row0 = (w.tile() * 128 + static_cast<int>(lane) * box) % p.page;
        for (int c = 0; c < Ly::KCH; ++c)
          tma_load_4d_hint(base + Ly::RING_OFF + stage * Ly::TILE + c * Ly::CHUNK + lane * box * 128u,
                           map, bar(Ly::B_KVFULL + stage), c * 64, w.hkv, row0, pid, stream);
      }
      used |= 1u << stage;
      if (++stage == Ly::STAGES) {
        stage = 0;
        phase ^= 1u;
      }
      return true;
    };
    auto load_q = [&](const PagedWalk& w) -> bool {
      const uint32_t slot = qcnt % Ly::QS, round = qcnt / Ly::QS;
      if (round > 0 && !mbar_wait_warp(bar(Ly::B_QEMPTY + slot), (round - 1) & 1, ab, err, 1002))
        return false;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(Ly::B_QFULL + slot), Ly::KCH * p.rows * 128u);
        for (int c = 0; c < Ly::KCH; ++c)
          tma_load_4d(base + Ly::Q_OFF + slot * Ly::QT + c * Ly::QCH, &tmQ, bar(Ly::B_QFULL + slot),
                      c * 64, w.hkv * p.g, 0, w.b);
      }
      ++qcnt;
      return true;
    };
    PagedWalk kw = paged_walk(p, plan), vw = kw;
    if (kw.rem > 0) {
      int pid_k = page_of(kw);
      ok = load_q(kw) && load(&tmK, kw, pid_k);
      while (ok && vw.rem > 0) {
        const int pid_v = pid_k;
        if (kw.rem > 1) {
          kw.next(p);
          pid_k = page_of(kw);
          if (kw.first) ok = load_q(kw);
          ok = ok && load(&tmK, kw, pid_k);
        }
        ok = ok && load(&tmV, vw, pid_v);
        vw.next(p);
      }
      if (!ok && lane == 0) {
        // Unwinding: let copies in flight land.  The newest use of a stage
        // before the write position has this round's parity, the others the
        // last round's.
        for (int s = 0; s < Ly::STAGES; ++s)
          if (used >> s & 1u)
            mbar_wait_drain(bar(Ly::B_KVFULL + s), s < static_cast<int>(stage) ? phase : phase ^ 1u);
        for (uint32_t c = qcnt > Ly::QS ? qcnt - Ly::QS : 0; c < qcnt; ++c)
          mbar_wait_drain(bar(Ly::B_QFULL + c % Ly::QS), (c / Ly::QS) & 1);
      }
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ MMA issuer
    uint32_t stage = 0, phase = 0;
    bool ok = true;
    auto commit = [&](int b) {
      if (elect_one()) tc_commit(bar(b));
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
    PagedWalk sw = paged_walk(p, plan), vw = sw;
    // S^T of tile i (the walk sw's).
    auto issue_s = [&](int i) -> bool {
      const uint32_t qslot = sw.item % Ly::QS;
      if (sw.first) {
        if (!mbar_wait_warp(bar(Ly::B_QFULL + qslot), (sw.item / Ly::QS) & 1, ab, err, 1003)) return false;
      }
      uint32_t ks;
      if (!take(ks, 1004)) return false;
      const uint64_t kd = sdesc_sw128(base + Ly::RING_OFF + ks * Ly::TILE, 16, 1024);
      const uint64_t qd = sdesc_sw128(base + Ly::Q_OFF + qslot * Ly::QT, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ss(tmem + Ly::TM_S + (i & 1) * N, kd + (((k >> 2) * Ly::CHUNK + (k & 3) * 32u) >> 4),
                 qd + (((k >> 2) * Ly::QCH + (k & 3) * 32u) >> 4), IDESC_S, k > 0 ? 1u : 0u);
        tc_commit(bar(Ly::B_SFULL + (i & 1)));
        tc_commit(bar(Ly::B_KVEMPTY + ks));
        if (sw.last()) tc_commit(bar(Ly::B_QEMPTY + qslot));
      }
      __syncwarp();
      sw.next(p);
      return true;
    };
    if (vw.rem > 0) ok = issue_s(0);
    for (int i = 0; ok && vw.rem > 0; ++i) {
      const int buf = i & 1, ob = vw.item & 1;
      // S(i+1) goes into the buffer tile i-1 left: its P is in shared memory
      // and its scores were read before that P was handed over.
      if (sw.rem > 0 && !issue_s(i + 1)) { ok = false; break; }
      uint32_t vs;
      if (!take(vs, 1005)) { ok = false; break; }
      if (vw.first && vw.item >= 2 &&
          !mbar_wait_warp(bar(Ly::B_OEMPTY + ob), ((vw.item >> 1) - 1) & 1, ab, err, 1006)) {
        ok = false;
        break;
      }
      if (!mbar_wait_warp(bar(Ly::B_PFULL + buf), (i >> 1) & 1, ab, err, 1007)) { ok = false; break; }
      tc_fence_after();
      const uint64_t vd = sdesc_sw128(base + Ly::RING_OFF + vs * Ly::TILE, Ly::CHUNK, 1024);
      const uint64_t pd = sdesc_sw128(base + Ly::P_OFF + buf * Ly::PT, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_ss(tmem + Ly::TM_O + ob * N, vd + ((2048u * k) >> 4),
                 pd + (((k >> 2) * Ly::QCH + (k & 3) * 32u) >> 4), IDESC_PV,
                 (!vw.first || k > 0) ? 1u : 0u);
        tc_commit(bar(Ly::B_PVDONE + buf));
        tc_commit(bar(Ly::B_KVEMPTY + vs));
        if (vw.last()) tc_commit(bar(Ly::B_OFULL + ob));
      }
      __syncwarp();
      vw.next(p);
    }
    commit(Ly::B_DONE);
    mbar_wait_drain(bar(Ly::B_DONE), 0);
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int t = threadIdx.x;  // key of the tile; head dim of the epilogue
    const uint32_t lane_off = (warp * 32u) << 16;
    const float sl2 = p.sl2;
    float* wmax = reinterpret_cast<float*>(gbase + Ly::ST_OFF);  // [2][4][N]
    float* mbuf = wmax + 8 * N + warp * N;                       // this warp's copy
    float* aux = wmax + 12 * N;                                  // [4][N]
    const int row_l = lane & (CW - 1);                           // row of a chunk this lane keeps
    float m[NCH], l[NCH];
    uint32_t vpos = 0;  // position of the tile's V in the ring's sequence
    uint32_t xsum = 0;
    bool ok = true;
    PagedWalk w = paged_walk(p, plan);
    const int total = w.rem;
    const int b0 = w.b, hkv0 = w.hkv, k0_first = w.k;
    int first_open = 0, last_bh = -1, last_slot = 0;
    int k_start = w.k;  // first tile of the current item in this part
    for (int i = 0; ok && w.rem > 0; ++i) {
      const int buf = i & 1;
      vpos = w.rem > 1 ? 2u * i + 2u : 2u * i + 1u;
      if (w.first) {
        k_start = w.k;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          m[c] = -INFINITY;
          l[c] = 0.f;
        }
      }
      if (!mbar_wait_warp(bar(Ly::B_SFULL + buf), (i >> 1) & 1, ab, err, 1008)) { ok = false; break; }
      tc_fence_after();
      uint32_t sr[N];
      const uint32_t tS = tmem + lane_off + Ly::TM_S + buf * N;
      if constexpr (N == 16) {
        tmem_ld16(tS, sr);
        tmem_ld_wait16(sr);
      } else {
#pragma unroll
        for (int c = 0; c < N / 32; ++c) tmem_ld32(tS + 32 * c, sr + 32 * c);
#pragma unroll
        for (int c = 0; c < N / 32; ++c) tmem_ld_wait32(sr + 32 * c);
      }
      const int key0 = w.tile() * 128, key = key0 + t;
      const int a0 = w.s.n - p.Lq;  // position of the first query
      const bool whole = key0 + 127 <= a0 && (p.window == 0 || key0 > w.s.n - 1 - p.window || key0 + 128 <= p.sinks);
      if (!whole) {
        int a = a0, hh = 0;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const bool hide = key > min(a, w.s.n - 1) || (p.window != 0 && key <= a - p.window && key >= p.sinks);
          if (hide) sr[r] = __float_as_uint(-INFINITY);
          if (++hh == p.g) {
            hh = 0;
            ++a;
          }
        }
      }
      if (p.scores != nullptr) {
        float* dst = p.scores + (t0 + i) * static_cast<long long>(p.rows) * 128 + t;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < p.rows) dst[r * 128] = __uint_as_float(sr[r]);
      }
      // Row maxima: over the warp's keys, then over the four warps.
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float x[CW];
#pragma unroll
        for (int r = 0; r < CW; ++r) x[r] = __uint_as_float(sr[c * CW + r]);
        const float v = paged_rows_reduce<CW, true>(x, lane);
        if (lane < CW) wmax[(buf * 4 + warp) * N + c * CW + row_l] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_XMAX));
      if (!mbar_wait_warp(bar(Ly::B_XMAX), i & 1, ab, err, 1009)) { ok = false; break; }
      bool grow = false;
      float alpha[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const float* wm = wmax + buf * 4 * N + c * CW + row_l;
        const float m_new = fmaxf(fmaxf(fmaxf(wm[0], wm[N]), fmaxf(wm[2 * N], wm[3 * N])), m[c]);
        alpha[c] = 1.f;
        if (m[c] == -INFINITY) {
          m[c] = m_new;  // nothing accumulated yet
        } else if ((m_new - m[c]) * sl2 > 8.0f) {
          alpha[c] = ex2((m[c] - m_new) * sl2);
          m[c] = m_new;
          grow = true;
        }
        if (lane < CW) {
          mbuf[c * CW + row_l] = m[c] == -INFINITY ? 0.f : m[c] * sl2;
          aux[warp * N + c * CW + row_l] = alpha[c];
        }
      }
      __syncwarp();
      // The four warps see the same maxima, so they agree here.
      if (__any_sync(0xffffffffu, grow)) {
        // O^T holds the item's earlier tiles once PV(i-1) is done (the phase
        // two tiles later needs this warp's P first).
        if (!mbar_wait_warp(bar(Ly::B_PVDONE + (buf ^ 1)), ((i - 1) >> 1) & 1, ab, err, 1010)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tO = tmem + lane_off + Ly::TM_O + (w.item & 1) * N;
        const float* al = aux + warp * N;
        constexpr int OC = N == 16 ? 16 : 32;
#pragma unroll
        for (int c = 0; c < N / OC; ++c) {
          uint32_t o[OC];
          if constexpr (OC == 16) {
            tmem_ld16(tO, o);
            tmem_ld_wait16(o);
          } else {
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait32(o);
          }
#pragma unroll
          for (int r = 0; r < OC; ++r)
            if (c * OC + r < R) o[r] = __float_as_uint(__uint_as_float(o[r]) * al[c * OC + r]);
          if constexpr (OC == 16)
            tmem_st16(tO, o);
          else
            tmem_st32(tO + 32 * c, o);
        }
        tmem_st_wait();
      }
      // P = exp2(s c - m c), to shared memory in the 16-bit type (the MMA's
      // operand); the row sums take the unrounded values.
      uint8_t* prow = gbase + Ly::P_OFF + buf * Ly::PT + (t >> 6) * Ly::QCH;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float x[CW];
#pragma unroll
        for (int r = 0; r < CW; ++r) {
          const int rr = c * CW + r;
          x[r] = ex2(fmaf(__uint_as_float(sr[rr]), sl2, -mbuf[rr]));
          *reinterpret_cast<T*>(prow + rr * 128 + (((t & 63) * 2) ^ ((rr & 7) << 4))) = static_cast<T>(x[r]);
        }
        l[c] = l[c] * alpha[c] + paged_rows_reduce<CW, false>(x, lane);
      }
      if (!whole) {
        // V rows of keys nobody sees: zero, whatever the page holds there.
        if (!mbar_wait_warp(bar(Ly::B_KVFULL + vpos % Ly::STAGES), (vpos / Ly::STAGES) & 1, ab, err, 1011)) {
          ok = false;
          break;
        }
        if (key >= w.s.n || (key < w.s.wlo && key >= p.sinks)) {
          uint4* v = reinterpret_cast<uint4*>(gbase + Ly::RING_OFF + (vpos % Ly::STAGES) * Ly::TILE + t * 128);
#pragma unroll
          for (int c = 0; c < Ly::KCH; ++c)
#pragma unroll
            for (int u = 0; u < 8; ++u) v[c * (Ly::CHUNK / 16) + u] = make_uint4(0, 0, 0, 0);
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_PFULL + buf));

      if (w.last()) {
        // ---- the item's end in this part: O^T / l and LSE, or a partial
        const int ob = w.item & 1;
        // Row sums of the four warps.
#pragma unroll
        for (int c = 0; c < NCH; ++c)
          if (lane < CW) aux[warp * N + c * CW + row_l] = l[c];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_XSUM));
        if (!mbar_wait_warp(bar(Ly::B_XSUM), xsum & 1, ab, err, 1012)) { ok = false; break; }
        ++xsum;
        const bool starts = k_start == 0, ends = w.k + 1 == w.s.cnt;
        const bool direct = starts && ends;
        const int slot = 2 * blockIdx.x + (w.item > 0 ? 1 : 0);
        if (w.item == 0 && !ends) first_open = 1;
        if (starts && !ends) {
          last_bh = w.b * p.Hkv + w.hkv;
          last_slot = slot;
        }
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int rr = c * CW + row_l;
          const float* ls = aux + rr;
          const float sum = (ls[0] + ls[N]) + (ls[2 * N] + ls[3 * N]);
          if (lane < CW) mbuf[rr] = sum > 0.f ? 1.f / sum : 0.f;
          if (warp == 0 && lane < CW && rr < p.rows) {
            const float lse2 = sum > 0.f ? m[c] * sl2 + __log2f(sum) : -INFINITY;
            if (direct)
              p.LSE[(static_cast<size_t>(w.b) * p.H + w.hkv * p.g + rr % p.g) * p.Lq + rr / p.g] =
                  lse2 * 0.6931471805599453f;
            else
              p.part_lse[static_cast<size_t>(slot) * p.rows + rr] = lse2;
          }
        }
        __syncwarp();
        if (!mbar_wait_warp(bar(Ly::B_OFULL + ob), (w.item >> 1) & 1, ab, err, 1013)) { ok = false; break; }
        tc_fence_after();
        if (t < D) {
          const uint32_t tO = tmem + lane_off + Ly::TM_O + ob * N;
          T* dst = reinterpret_cast<T*>(p.O) + (static_cast<size_t>(w.b) * p.Lq * p.H + w.hkv * p.g) * D + t;
          float* part = p.part_o + static_cast<size_t>(slot) * p.rows * D + t;
          constexpr int OC = N == 16 ? 16 : 32;
          int hh = 0;
#pragma unroll
          for (int c = 0; c < N / OC; ++c) {
            uint32_t o[OC];
            if constexpr (OC == 16) {
              tmem_ld16(tO, o);
              tmem_ld_wait16(o);
            } else {
              tmem_ld32(tO + 32 * c, o);
              tmem_ld_wait32(o);
            }
#pragma unroll
            for (int r = 0; r < OC; ++r) {
              const int rr = c * OC + r;
              if (rr < R && rr < p.rows) {
                const float v = __uint_as_float(o[r]) * mbuf[rr];
                if (direct)
                  dst[static_cast<size_t>(hh) * D] = static_cast<T>(v);
                else
                  part[rr * D] = v;
                if (++hh == p.g) {  // next query
                  hh = 0;
                  dst += static_cast<size_t>(p.H) * D;
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_OEMPTY + ob));
      }
      w.next(p);
    }
    if (t == 0) {
      PagedMeta mt;
      mt.t0 = t0;
      mt.n = ok ? total : 0;
      mt.b = b0;
      mt.hkv = hkv0;
      mt.k = k0_first;
      mt.first_open = first_open;
      mt.last_bh = ok ? last_bh : -1;
      mt.last_slot = last_slot;
      p.meta[blockIdx.x] = mt;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 5) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Ly::TMEM_COLS);
  }
}

// Join the partials of the items that the parts' borders cut: block c joins
// the item that starts in part c and goes on in the next ones.  It also writes
// O = 0, LSE = -inf of the empty sequences c, c + G, ....
template <int D, bool BF16>
__global__ void __launch_bounds__(256) fa_paged_join_kernel(const PagedParams p, int G) {
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  pdl_launch_dependents();
  pdl_wait();
  const int c = blockIdx.x, lane = lane_id();
  for (int b = c; b < p.B; b += G) {
    if (p.lens[b] > 0 && p.cap > 0) continue;
    T* dst = reinterpret_cast<T*>(p.O) + static_cast<size_t>(b) * p.Lq * p.H * D;
    for (int i = threadIdx.x; i < p.Lq * p.H * D; i += blockDim.x) dst[i] = static_cast<T>(0.f);
    for (int i = threadIdx.x; i < p.Lq * p.H; i += blockDim.x)
      p.LSE[static_cast<size_t>(b) * p.Lq * p.H + i] = -INFINITY;
  }
  const PagedMeta mt = p.meta[c];
  if (mt.n == 0 || mt.last_bh < 0) return;
  __shared__ int last_part;
  if (threadIdx.x == 0) {
    // The parts the item goes through: c, then the first items of the next
    // non-empty parts up to the one it ends in.
    int e = c + 1;
    while (e < G && (p.meta[e].n == 0 || p.meta[e].first_open)) ++e;
    last_part = e < G ? e : G - 1;
  }
  __syncthreads();
  const int e = last_part;
  const int b = mt.last_bh / p.Hkv, hkv = mt.last_bh - b * p.Hkv;
  constexpr int PER = D / 32;
  for (int row = warp_id(); row < p.rows; row += 8) {
    float mx = p.part_lse[static_cast<size_t>(mt.last_slot) * p.rows + row];
    for (int q = c + 1; q <= e; ++q)
      if (p.meta[q].n) mx = fmaxf(mx, p.part_lse[static_cast<size_t>(2 * q) * p.rows + row]);
    float den = 0.f, acc[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) acc[u] = 0.f;
    if (mx != -INFINITY) {
      for (int q = c; q <= e; ++q) {
        if (q > c && p.meta[q].n == 0) continue;
        const size_t at = static_cast<size_t>(q == c ? mt.last_slot : 2 * q) * p.rows + row;
        const float wgt = ex2(p.part_lse[at] - mx);
        den += wgt;
#pragma unroll
        for (int u = 0; u < PER; ++u) acc[u] = fmaf(wgt, p.part_o[at * D + lane + 32 * u], acc[u]);
      }
    }
    const float inv = den > 0.f ? 1.f / den : 0.f;
    const int ql = row / p.g, h = hkv * p.g + row - ql * p.g;
    T* dst = reinterpret_cast<T*>(p.O) + ((static_cast<size_t>(b) * p.Lq + ql) * p.H + h) * D;
#pragma unroll
    for (int u = 0; u < PER; ++u) dst[lane + 32 * u] = static_cast<T>(acc[u] * inv);
    if (lane == 0)
      p.LSE[(static_cast<size_t>(b) * p.H + h) * p.Lq + ql] =
          den > 0.f ? (mx + __log2f(den)) * 0.6931471805599453f : -INFINITY;
  }
}

// Add every visible key's attention weight, sum over the item's rows of
// exp(s - LSE), from the raw scores the decode kernel left.  Block (c, y)
// takes every gridDim.y-th tile of part c; each key belongs to one thread.
__global__ void __launch_bounds__(128)
    fa_paged_weights_kernel(const PagedParams p, float* __restrict__ weights, long long wstride) {
  pdl_wait();
  const PagedMeta mt = p.meta[blockIdx.x];
  __shared__ float lse2[128];
  const int plan[4] = {mt.b, mt.hkv, mt.k, mt.n};
  PagedWalk w = paged_walk(p, plan);
  const int Y = gridDim.y, y = blockIdx.y, t = threadIdx.x;
  for (int i = 0; w.rem > 0; ++i, w.next(p)) {
    if (w.first) {
      __syncthreads();
      if (t < p.rows) {
        const float v = p.LSE[(static_cast<size_t>(w.b) * p.H + w.hkv * p.g + t % p.g) * p.Lq + t / p.g];
        lse2[t] = v == -INFINITY ? 0.f : v * 1.4426950408889634f;  // (then every score is -inf)
      }
      __syncthreads();
    }
    if (i % Y != y) continue;
    const int key = w.tile() * 128 + t;
    if (key >= w.s.n) continue;
    const float* src = p.scores + (mt.t0 + i) * static_cast<long long>(p.rows) * 128 + t;
    float sum = 0.f;
    for (int r = 0; r < p.rows; ++r) sum += ex2(fmaf(src[r * 128], p.sl2, -lse2[r]));
    float* dst = weights + (static_cast<long long>(w.b) * p.Hkv + w.hkv) * wstride + key;
    *dst += sum;
  }
}

// Copy new keys and values into the pages, and set their slots' weights.
// One thread per 16 bytes of K (and of V).
__global__ void __launch_bounds__(256)
    fa_paged_write_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                          uint4* __restrict__ kc, uint4* __restrict__ vc, long long k_page,
                          long long v_page, const int* __restrict__ table,
                          const int* __restrict__ start, const int* __restrict__ counts,
                          float* __restrict__ weights, long long wstride,
                          const float* __restrict__ new_w, int B, int L, int Hkv, int units,
                          int page, int max_pages, int num_pages) {
  const int per = Hkv * units;  // 16-byte units of a token (units = D / 8 per head)
  const long long all = static_cast<long long>(B) * L * per;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < all; i += gridDim.x * 256ll) {
    const long long tok = i / per;
    const int u = static_cast<int>(i - tok * per);
    const int b = static_cast<int>(tok / L), j = static_cast<int>(tok - static_cast<long long>(b) * L);
    if (counts != nullptr && j >= counts[b]) continue;
    const long long pos = static_cast<long long>(start[b]) + j;
    if (pos < 0 || pos >= static_cast<long long>(max_pages) * page) continue;
    const int pid = table[static_cast<size_t>(b) * max_pages + pos / page];
    if (pid < 0 || pid >= num_pages) continue;
    const long long row = (pos % page) * per + u;
    kc[pid * k_page + row] = k[i];
    vc[pid * v_page + row] = v[i];
    if (weights != nullptr && u % units == 0) {
      const long long bh = static_cast<long long>(b) * Hkv + u / units;
      weights[bh * wstride + pos] = new_w != nullptr ? new_w[bh * L + j] : 0.f;
    }
  }
}

}  // namespace fa
