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
//   - one persistent CTA per SM (fewer when few items would be cut into so many
//     parts that joining them took longer).  The tiles of all items form one list (item by
//     item); CTA c takes the c-th of G equal contiguous parts of it, whatever
//     the lengths are.  Lengths are read on the device: every CTA scans them
//     once.  An item inside one CTA is written directly; only items cut by a
//     part's border leave partials, at most two per CTA, so the workspace does
//     not grow with the lengths.  The CTA that finishes last of an item's parts
//     joins them (a counter per part tells it), so there is no second kernel.
//   - one TMA ring of K and V tiles runs through the whole part, across items;
//     page ids are read 32 at a time and a batch ahead, as one read per tile
//     in the loader's way cost 700 cycles (of the 1440 that the K and V of a
//     tile take to arrive at D = 64).
//   - the products are transposed, S^T = K Q^T and O^T = V^T P^T: the 128 keys
//     (or the head dims) fill the 128 rows of the MMA and the g * Lq packed
//     query rows are its N, 16 at least.  A thread then owns one key and only
//     as many scores as there are query rows, where Q K^T with the queries in
//     128 padded rows makes every warp exponentiate 128 keys for a handful of
//     live lanes.
//   - two groups of four softmax warps take the tiles in turn (up to 64 packed
//     rows), each with a maximum, a sum and an O accumulator of its own that
//     are joined at the item's end: a tile's chain from scores to P takes 1500
//     cycles, as long as its K and V take to arrive at D = 64.
// Warps 0-7 (0-3 for 128 rows): softmax (thread = key of the tile), epilogue
// (thread = head dim); then a warp each for the TMA loads, the S^T products
// (and TMEM) and the O^T products: issuing a product holds its warp while it
// runs, and one warp for both took 1900 cycles a tile with its waits.
// Row maxima are reduced over the 32 keys of a warp by a halving exchange
// (lane r ends with row r), then over the four warps through shared memory;
// a row's max moves only when it grew by more than 2^8 in exp2 units, as in
// the dense forward.
// Keys that no query sees (behind the length, before the window) may lie in
// pages that were never written: their scores are replaced, not multiplied,
// and their V rows are set to zero in shared memory before the PV product.
// Measured (bf16, H32/8 D128): B16 16,384 keys 163 us, 6.58 TB/s (99% of the copy
// rate; pages of 16 keys 174 us); B64 1,024 keys 49 us; B1 131,072 keys 92 us;
// B1 500 keys 10.5 us, where launch, page ids, one tile and the join follow one
// another; four tokens each of B8, window 4,096: 34 us (21 for the bytes alone).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "fwd.cuh"  // pack2
#include "ptx.cuh"

namespace fa {

struct PagedParams {
  const int* table;  // [B, max_pages]
  const int* lens;   // [B]
  void* O;           // [B, Lq, H, D]
  float* LSE;        // [B, H, Lq] natural log
  unsigned long long* count;  // [G] arrivals at the item that starts in part c and goes on:
  unsigned long long nonce;   // nonce << 16 | arrivals, 0 again when all have come
  float* part_o;     // [2 G, rows, D]
  float* part_lse;   // [2 G, rows], log2 units
  float* scores;     // [B * Hkv, max_tiles, rows, 128] raw scores for the weights, or NULL
  int B, Lq, H, Hkv, g, rows;
  int ginv;                  // 65536 / g + 1: row / g = row * ginv >> 16 for the rows there are (128 at most)
  int page, max_pages, cap;  // cap = max_pages * page
  int max_tiles;             // ceil(cap / 128)
  int window, sinks;         // window 0: none (then sinks 0)
  float sl2;                 // log2(e) / sqrt(D)
};

// The tiles one sequence's items visit: ns sink tiles, then lo, lo + 1, ....
struct PagedSeq {
  int n;    // length
  int wlo;  // first key the earliest query's window reaches
  int ns, lo, cnt;
};

__device__ __forceinline__ PagedSeq paged_seq_of(int len, const PagedParams& p) {
  PagedSeq s;
  s.n = min(max(len, 0), p.cap);
  s.wlo = p.window ? max(max(s.n - p.Lq, 0) - p.window + 1, 0) : 0;
  s.lo = s.wlo >> 7;
  s.ns = min((min(p.sinks, s.n) + 127) >> 7, s.lo);
  s.cnt = s.n > 0 ? s.ns + ((s.n + 127) >> 7) - s.lo : 0;
  return s;
}

// Walk over the tiles of one CTA's part; a step costs a few instructions, an
// item's start reads the length.
struct PagedWalk {
  int b, hkv, k;  // item, and tile's place in its list
  int tile;       // the tile: keys [128 tile, 128 tile + 128)
  int left;       // tiles of the item left in the part, this one included
  int rem;        // tiles left in the part, this one included
  int item;       // items begun before this one in the part
  bool first;     // first tile of its item in this part
  const int* lens;  // [B]; a copy in shared memory when B <= 32
  PagedSeq s;

  __device__ __forceinline__ bool last() const { return left == 1; }
  __device__ __forceinline__ void enter() {
    tile = k < s.ns ? k : s.lo + k - s.ns;
    left = min(s.cnt - k, rem);
    first = true;
  }
  __device__ __forceinline__ void skip(const PagedParams& p, int n) {  // n <= left
    rem -= n;
    left -= n;
    first = false;
    if (left > 0) {
      k += n;
      tile = k < s.ns ? k : s.lo + k - s.ns;
    } else if (rem > 0) {
      k = 0;
      ++item;
      if (++hkv == p.Hkv) {
        hkv = 0;
        do {
          if (++b >= p.B) {
            rem = 0;
            return;
          }
          s = paged_seq_of(lens[b], p);
        } while (s.cnt == 0);
      }
      enter();
    }
  }
  __device__ __forceinline__ void next(const PagedParams& p) { skip(p, 1); }
};

// Part c of G of `total` tiles begins at tile:
__device__ __forceinline__ int paged_part(int total, int G, int c) {
  const int q = total / G, r = total - q * G;
  return c * q + min(c, r);
}
// The part that holds tile t.
__device__ __forceinline__ int paged_part_of(int total, int G, int t) {
  const int q = total / G, r = total - q * G, big = r * (q + 1);
  return t < big ? t / (q + 1) : r + (t - big) / q;
}

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
  static constexpr int NG = N <= 64 ? 2 : 1;      // softmax groups; K tiles loaded ahead of V
  static constexpr int NB = 2 * NG;               // S buffers
  static constexpr int PB = N <= 32 ? 4 : 2;      // P buffers
  static constexpr int QS = (D == 128 && N == 128) ? 1 : 2;
  static constexpr int STAGES = D == 128 ? (N == 16 ? 6 : N == 32 ? 5 : N == 64 ? 4 : 3)
                                         : (N == 16 ? 12 : N <= 64 ? 10 : 7);
  static constexpr uint32_t RING_OFF = 0;
  static constexpr uint32_t Q_OFF = STAGES * TILE;
  static constexpr uint32_t P_OFF = Q_OFF + QS * QT;
  // fp32 exchange areas: per group wmax[2][4][N], mb[4][N], alpha[4][N]; then
  // by item parity the groups' warps' row sums [2][4 NG][N] and maxima [2][NG][N]
  static constexpr uint32_t ST_OFF = P_OFF + PB * PT;
  static constexpr uint32_t SUM_OFF = ST_OFF + NG * 16u * N * 4u;
  static constexpr uint32_t MAX_OFF = SUM_OFF + 8u * NG * N * 4u;
  static constexpr uint32_t BAR_OFF = MAX_OFF + 2u * NG * N * 4u;
  static constexpr int B_QFULL = 0, B_QEMPTY = QS, B_KVFULL = 2 * QS, B_KVEMPTY = B_KVFULL + STAGES,
                       B_SFULL = B_KVEMPTY + STAGES, B_PFULL = B_SFULL + NB, B_PVDONE = B_PFULL + NB,
                       B_OFULL = B_PVDONE + NB, B_OEMPTY = B_OFULL + 2, B_XMAX = B_OEMPTY + 2,
                       B_XSUM = B_XMAX + NG, B_JOIN = B_XSUM + 2, B_DONE = B_JOIN + 2 * NG,
                       NBAR = B_DONE + 2;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;  // tmem slot, abort flag, plan
  static constexpr uint32_t USED = MISC_OFF + 256;
  // At D = 64 the PV product still takes 128 rows of V^T; rows 64-127 come
  // from the 16 KB behind the tile and their results are never read.  Behind
  // the last ring stage that much must still be shared memory of this CTA.
  static constexpr uint32_t SMEM_USED = (D == 64 && USED < Q_OFF + CHUNK) ? Q_OFF + CHUNK : USED;
  static constexpr uint32_t SMEM_ALLOC = SMEM_USED + 1024;
  static constexpr uint32_t TM_S = 0, TM_O = NB * N;  // O[item parity][group]
  static constexpr uint32_t TMEM_COLS = (NB + 2 * NG) * N;
  static constexpr int SW = 4 * NG;  // softmax warps; then the producer, S and O^T warps
  static constexpr int NTHREADS = 32 * SW + 96;
  // arrivals a barrier takes a phase
  __device__ static constexpr int arrivals(int i) {
    return (i >= B_PFULL && i < B_PVDONE) || (i >= B_OEMPTY && i < B_XSUM) ? 4
           : i >= B_XSUM && i < B_JOIN                                      ? SW
           : i >= B_JOIN && i < B_DONE && ((i - B_JOIN) & 1) == 0           ? 4
                                                                            : 1;
  }
  static_assert(SMEM_ALLOC <= 232448, "shared memory");
  static_assert(TMEM_COLS <= 512 && (TMEM_COLS & (TMEM_COLS - 1)) == 0, "TMEM");
  static_assert(BAR_OFF % 8 == 0 && ST_OFF % 16 == 0, "alignment");
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

// Part c of G of the list of all tiles: the start and length of the walk in
// `plan` {b, hkv, k, n}, t0 and the total in plan[4], plan[5].  Called by the
// whole CTA (NT threads); `len` is lens[lane] for the small case, read early.
template <int NT>
__device__ __forceinline__ void paged_plan(const PagedParams& p, int c, int G, int len, int* sums,
                                           int* plan) {
  const uint32_t lane = lane_id();
  if (p.B <= 32) {
    // Every warp for itself is faster than once for all; warp 0 writes.
    const int mine = static_cast<int>(lane) < p.B ? paged_seq_of(len, p).cnt * p.Hkv : 0;
    int incl = mine;
#pragma unroll
    for (int h = 1; h < 32; h <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, incl, h);
      if (lane >= static_cast<uint32_t>(h)) incl += o;
    }
    const int total = __shfl_sync(0xffffffffu, incl, 31);
    const int t0 = paged_part(total, G, c), n = paged_part(total, G, c + 1) - t0;
    const int off = t0 - (incl - mine);
    if (warp_id() == 0) {
      if (n > 0 && off >= 0 && off < mine) {
        const int cnt = mine / p.Hkv;
        plan[0] = lane;
        plan[1] = off / cnt;
        plan[2] = off - off / cnt * cnt;
      }
      if (lane == 0) {
        plan[3] = n;
        plan[4] = t0;
        plan[5] = total;
      }
    }
    __syncthreads();
    return;
  }
  const int per = (p.B + NT - 1) / NT;
  const int b0 = min(p.B, static_cast<int>(threadIdx.x) * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; ++b) mine += paged_seq_of(p.lens[b], p).cnt * p.Hkv;
  int incl = mine;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, h);
    if (lane >= static_cast<uint32_t>(h)) incl += o;
  }
  if (lane == 31) sums[warp_id()] = incl;
  __syncthreads();
  int before = incl - mine, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < static_cast<int>(warp_id())) before += sums[w];
    total += sums[w];
  }
  const int t0 = paged_part(total, G, c), n = paged_part(total, G, c + 1) - t0;
  if (threadIdx.x == 0) {
    plan[3] = n;
    plan[4] = t0;
    plan[5] = total;
  }
  if (n > 0 && t0 >= before && t0 < before + mine) {
    int at = before;
    for (int b = b0; b < b1; ++b) {
      const int cnt = paged_seq_of(p.lens[b], p).cnt, all = cnt * p.Hkv;
      if (t0 < at + all) {
        plan[0] = b;
        plan[1] = (t0 - at) / cnt;
        plan[2] = (t0 - at) % cnt;
        break;
      }
      at += all;
    }
  }
  __syncthreads();
}

__device__ __forceinline__ PagedWalk paged_walk(const PagedParams& p, const int* plan, const int* lens) {
  PagedWalk w;
  w.lens = lens;
  w.rem = plan[3];
  w.b = plan[0];
  w.hkv = plan[1];
  w.k = plan[2];
  w.item = 0;
  w.left = 0;
  if (w.rem > 0) {
    w.s = paged_seq_of(lens[w.b], p);
    w.enter();
  }
  return w;
}

// Count an arrival at an item of n parts; true for the last one.  The word needs
// no initialisation: whatever lies there without this call's nonce counts as
// none, and the last arrival leaves 0, so a captured call can be replayed.
// `cur`: the word as it was read a while ago.  One arrival puts the nonce there,
// all others add: at most three trips to the L2, however many come at once (with
// a swap for each, 50 parts of one item took 50 trips).
__device__ __forceinline__ int paged_count_in(unsigned long long* word, unsigned long long nonce, int n,
                                              unsigned long long cur) {
  int seen = 0;
  for (;;) {  // ends: a failed swap means that another part put the nonce there (nothing else writes)
    if ((cur >> 16) == nonce) {  // (it stays until the last part is here)
      seen = static_cast<int>(atomicAdd(word, 1ull) & 0xFFFFu);
      break;
    }
    const unsigned long long was = atomicCAS(word, cur, nonce << 16 | 1u);
    if (was == cur) break;
    cur = was;
  }
  const bool last = seen + 1 == n;
  if (last) atomicExch(word, 0ull);
  return last;
}

// The joined O and LSE of an item from `n` partials, in slots slot0, then
// slot1, slot1 + 2, ...; 128 threads, four head dims of U rows each.  One pass
// with the running maximum over C partials at a time.  What it costs is the
// latency of the L2 beside a full memory bus (about 2000 cycles), so a round's
// U * C reads go out together: past the last row or partial they repeat the last
// one with no weight instead of standing under a condition, and the warp meets
// before the first is used, or the compiler spreads them between their uses (16
// rows of 3 partials: 17,500 cycles with conditions and a float per read, 7400
// without the meeting, 3500 so).
// Reads past L1: other SMs wrote them.
template <int D, typename T, int R>
__device__ __forceinline__ void paged_join(const PagedParams& p, int b, int hkv, int slot0, int slot1,
                                           int n) {
  constexpr int U = R * (D / 4) >= 512 ? 4 : R * (D / 4) >= 256 ? 2 : 1, C = 16 / U;
  constexpr int PER_ROW = D / 4, ROWS = 128 / PER_ROW;  // threads of a row, rows of a step
  const int d = (threadIdx.x % PER_ROW) * 4, rt = (threadIdx.x & 127) / PER_ROW;
#pragma unroll 1
  for (int r0 = rt; r0 - rt < p.rows; r0 += U * ROWS) {  // as often for every lane
    float mx[U], den[U];
    float4 acc[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      mx[u] = -INFINITY;
      den[u] = 0.f;
      acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll 1
    for (int q0 = 0; q0 < n; q0 += C) {
      float ls[C][U];
      float4 o[C][U];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int q = min(q0 + c, n - 1);
        const size_t slot = q == 0 ? slot0 : slot1 + 2 * (q - 1);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const size_t at = slot * p.rows + min(r0 + u * ROWS, p.rows - 1);
          ls[c][u] = __ldcg(p.part_lse + at);
          o[c][u] = __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + d));
        }
      }
      __syncwarp();  // all reads out before the first is used
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool in = q0 + c < n;
          const float l = in ? ls[c][u] : -INFINITY;
          const float m = fmaxf(mx[u], l);
          // (each for itself: a NaN LSE has no part in m, but its weight is NaN)
          const float old = mx[u] == -INFINITY ? 0.f : ex2(mx[u] - m), w = l == -INFINITY ? 0.f : ex2(l - m);
          den[u] = fmaf(den[u], old, w);
          acc[u].x = fmaf(acc[u].x, old, in ? w * o[c][u].x : 0.f);
          acc[u].y = fmaf(acc[u].y, old, in ? w * o[c][u].y : 0.f);
          acc[u].z = fmaf(acc[u].z, old, in ? w * o[c][u].z : 0.f);
          acc[u].w = fmaf(acc[u].w, old, in ? w * o[c][u].w : 0.f);
          mx[u] = m;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int row = r0 + u * ROWS;
      if (row < p.rows) {
        const int ql = row * p.ginv >> 16, h = hkv * p.g + row - ql * p.g;
        const float inv = den[u] > 0.f ? __fdividef(1.f, den[u]) : 0.f;
        *reinterpret_cast<uint2*>(reinterpret_cast<T*>(p.O) +
                                  ((static_cast<size_t>(b) * p.Lq + ql) * p.H + h) * D + d) =
            make_uint2(pack2<T>(acc[u].x * inv, acc[u].y * inv), pack2<T>(acc[u].z * inv, acc[u].w * inv));
        if (d == 0)
          p.LSE[(static_cast<size_t>(b) * p.H + h) * p.Lq + ql] =
              den[u] == 0.f ? -INFINITY : (mx[u] + __log2f(den[u])) * 0.6931471805599453f;
      }
    }
  }
}

template <int D, bool BF16, int R>
__global__ void __launch_bounds__(PagedLayout<D, R>::NTHREADS, 1)
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
  int* sums = reinterpret_cast<int*>(gbase + Ly::MISC_OFF + 48);      // NTHREADS / 32
  int* lens_s = reinterpret_cast<int*>(gbase + Ly::MISC_OFF + 128);   // 32
  const int* lens = p.B <= 32 ? lens_s : p.lens;
  unsigned int* err = device_error_word();
  const uint32_t warp = warp_id(), lane = lane_id();

  // Query rows past g * Lq, and P rows no thread writes, are zero.
  for (uint32_t i = threadIdx.x; i < (Ly::QS * Ly::QT + Ly::PB * Ly::PT) / 16u; i += Ly::NTHREADS)
    reinterpret_cast<uint4*>(gbase + Ly::Q_OFF)[i] = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  for (int i = threadIdx.x; i < Ly::NBAR; i += Ly::NTHREADS) mbar_init(bar(i), Ly::arrivals(i));
  if (threadIdx.x == 0) ab->flag = 0;
  fence_barrier_init();
  if (warp == Ly::SW + 1) {
    tmem_alloc(base + Ly::MISC_OFF, Ly::TMEM_COLS);
    tmem_relinquish();
  }
  if (warp == Ly::SW && lane == 0) {
    tma_prefetch_desc(&tmQ);
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  tc_fence_before();
  // Everything above overlaps the end of the kernel before; nothing of global
  // memory was touched.
  pdl_launch_dependents();
  pdl_wait();
  const int len = (p.B <= 32 && static_cast<int>(lane) < p.B) ? p.lens[lane] : 0;
  if (warp == 0) lens_s[lane] = len;
  paged_plan<Ly::NTHREADS>(p, blockIdx.x, gridDim.x, len, sums, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == Ly::SW) {
    // ------------------------------------------------------------ producer
    // Ring order: the first NG K tiles, then K_{i+NG}, V_i.  Lane j loads the j-th box
    // (a page, or 128 rows of one) of the tile.
    const int page_log = 31 - __clz(p.page);  // (a page is a power of two)
    const int box = min(p.page, 128), nbox = 128 >> min(page_log, 7), per_batch = 32 >> (7 - min(page_log, 7));
    uint32_t stage = 0, phase = 0, used = 0, qcnt = 0;
    bool ok = true;
    const uint64_t stream = policy_evict_first();
    // Page ids of the next tiles, one box per lane: `cur` for the tiles from
    // cur_tile on, `nxt` for the batch behind it (of the same item or the next).
    PagedWalk ahead = paged_walk(p, plan, lens);
    int nxt = -1, nxt_n = 0, cur = -1, cur_at = 0, cur_n = 0;
    auto fetch = [&]() {
      nxt_n = 0;
      if (ahead.rem <= 0) return;
      nxt_n = min(per_batch, ahead.left);
      if (ahead.k < ahead.s.ns) nxt_n = min(nxt_n, ahead.s.ns - ahead.k);  // up to the gap
      const int at = (ahead.tile * 128 + static_cast<int>(lane) * box) >> page_log;
      nxt = (static_cast<int>(lane) < nxt_n * nbox && at < p.max_pages)
                ? p.table[static_cast<size_t>(ahead.b) * p.max_pages + at]
                : -1;
      ahead.skip(p, nxt_n);
    };
    // The page id of this lane's box of the next tile in order.
    auto next_page = [&]() -> int {
      if (cur_at == cur_n) {
        cur = nxt;
        cur_n = nxt_n;
        cur_at = 0;
        fetch();
      }
      return __shfl_sync(0xffffffffu, cur, (cur_at++ * nbox + static_cast<int>(lane)) & 31);
    };
    auto load = [&](const CUtensorMap* map, const PagedWalk& w, int pid) -> bool {
      if (!mbar_wait_warp(bar(Ly::B_KVEMPTY + stage), phase ^ 1u, ab, err, 1001)) return false;
      // Boxes that hold a key some query sees; the others are not loaded.
      const int k0 = w.tile * 128 + static_cast<int>(lane) * box;
      const bool go = static_cast<int>(lane) < nbox && k0 < w.s.n && (k0 + box > w.s.wlo || k0 < p.sinks);
      const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, go));
      if (lane == 0)
        mbar_arrive_expect_tx(bar(Ly::B_KVFULL + stage), boxes * box * static_cast<uint32_t>(D) * 2u);
      __syncwarp();
      if (go) {
        const int row0 = k0 & (p.page - 1);
#pragma unroll
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
    PagedWalk kw = ahead, vw = ahead;
    if (kw.rem > 0) {
      fetch();
      int pid[Ly::NG + 1];  // this lane's page of tiles i .. i + NG
      auto load_k = [&](int x) -> bool {
        if (kw.rem <= 0) return true;
        pid[x] = next_page();
        if (kw.first && !load_q(kw)) return false;
        if (!load(&tmK, kw, pid[x])) return false;
        kw.next(p);
        return true;
      };
#pragma unroll
      for (int x = 0; x < Ly::NG; ++x) ok = ok && load_k(x);
      while (ok && vw.rem > 0) {
        ok = load_k(Ly::NG) && load(&tmV, vw, pid[0]);
        vw.next(p);
#pragma unroll
        for (int x = 0; x < Ly::NG; ++x) pid[x] = pid[x + 1];
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
  } else if (warp == Ly::SW + 1) {
    // ------------------------------------------------------------ S^T = K Q^T
    // Ring place of K_j: j, or NG + 2 (j - NG) behind the first NG; of V_i:
    // the K tiles loaded before it, min(n, i + 1 + NG), plus i.
    PagedWalk w = paged_walk(p, plan, lens);
    bool ok = true;
    for (int i = 0; ok && w.rem > 0; w.skip(p, w.left)) {
      const uint32_t qslot = w.item % Ly::QS;
      if (!mbar_wait_warp(bar(Ly::B_QFULL + qslot), (w.item / Ly::QS) & 1, ab, err, 1003)) { ok = false; break; }
      const uint64_t qd = sdesc_sw128(base + Ly::Q_OFF + qslot * Ly::QT, 16, 1024);
      for (int x = 0; x < w.left; ++x, ++i) {
        const uint32_t pos = i < Ly::NG ? i : 2 * i - Ly::NG, ks = pos % Ly::STAGES;
        const int buf = i % Ly::NB;
        // The buffer's last tile is through: its scores are read, and its P is
        // too, so that the softmax may write P again once this S is there.
        if (i >= Ly::NB &&
            !mbar_wait_warp(bar(Ly::B_PVDONE + buf), (i / Ly::NB - 1) & 1, ab, err, 1017)) {
          ok = false;
          break;
        }
        if (!mbar_wait_warp(bar(Ly::B_KVFULL + ks), (pos / Ly::STAGES) & 1, ab, err, 1004)) { ok = false; break; }
        tc_fence_after();
        const uint64_t kd = sdesc_sw128(base + Ly::RING_OFF + ks * Ly::TILE, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + Ly::TM_S + buf * N, kd + (((k >> 2) * Ly::CHUNK + (k & 3) * 32u) >> 4),
                   qd + (((k >> 2) * Ly::QCH + (k & 3) * 32u) >> 4), IDESC_S, k > 0 ? 1u : 0u);
          tc_commit(bar(Ly::B_SFULL + buf));
          tc_commit(bar(Ly::B_KVEMPTY + ks));
          if (x + 1 == w.left) tc_commit(bar(Ly::B_QEMPTY + qslot));
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(bar(Ly::B_DONE));
    __syncwarp();
    mbar_wait_drain(bar(Ly::B_DONE), 0);
  } else if (warp == Ly::SW + 2) {
    // ------------------------------------------------------------ O^T += V^T P^T
    PagedWalk w = paged_walk(p, plan, lens);
    const int n_part = w.rem;
    bool ok = true;
    for (int i = 0; ok && w.rem > 0; w.skip(p, w.left)) {
      const int ob = w.item & 1;
      if (w.item >= 2 &&
          !mbar_wait_warp(bar(Ly::B_OEMPTY + ob), ((w.item >> 1) - 1) & 1, ab, err, 1006)) {
        ok = false;
        break;
      }
      for (int x = 0; x < w.left; ++x, ++i) {
        const uint32_t pos = min(n_part, i + 1 + Ly::NG) + i, vs = pos % Ly::STAGES;
        const int buf = i % Ly::NB;
        // P first: then K_i and all before it have landed, one of which may
        // have had V_i's stage before it.  (A wait for a phase's parity passes
        // as well while the phase before it is still open, so whoever waits for
        // a stage must know that its last fill has landed.)
        if (!mbar_wait_warp(bar(Ly::B_PFULL + buf), (i / Ly::NB) & 1, ab, err, 1007) ||
            !mbar_wait_warp(bar(Ly::B_KVFULL + vs), (pos / Ly::STAGES) & 1, ab, err, 1005)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t vd = sdesc_sw128(base + Ly::RING_OFF + vs * Ly::TILE, Ly::CHUNK, 1024);
        const uint64_t pd = sdesc_sw128(base + Ly::P_OFF + (i % Ly::PB) * Ly::PT, 16, 1024);
        if (elect_one()) {
          // (a group's first tile of the item has no O to add to)
#pragma unroll
          for (int k = 0; k < 8; ++k)
            mma_ss(tmem + Ly::TM_O + (ob * Ly::NG + i % Ly::NG) * N, vd + ((2048u * k) >> 4),
                   pd + (((k >> 2) * Ly::QCH + (k & 3) * 32u) >> 4), IDESC_PV,
                   (x >= Ly::NG || k > 0) ? 1u : 0u);
          tc_commit(bar(Ly::B_PVDONE + buf));
          tc_commit(bar(Ly::B_KVEMPTY + vs));
          if (x + 1 == w.left) tc_commit(bar(Ly::B_OFULL + ob));
        }
        __syncwarp();
      }
    }
    if (elect_one()) tc_commit(bar(Ly::B_DONE + 1));
    __syncwarp();
    mbar_wait_drain(bar(Ly::B_DONE + 1), 0);
  } else {
    // ------------------------------------------------------------ softmax + epilogue
    const int gr = warp >> 2, wq = warp & 3;  // group, warp of the group (its TMEM lanes)
    const int t = threadIdx.x & 127;          // key of the tile; head dim of the epilogue
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const float sl2 = p.sl2;
    float* wmax = reinterpret_cast<float*>(gbase + Ly::ST_OFF) + gr * 16 * N;  // [2][4][N]
    float* mbuf = wmax + 8 * N + wq * N;                                       // this warp's copy
    float* al = wmax + 12 * N + wq * N;                                        // the same
    float* sum_x = reinterpret_cast<float*>(gbase + Ly::SUM_OFF);  // [2][4 NG][N]
    float* max_x = reinterpret_cast<float*>(gbase + Ly::MAX_OFF);  // [2][NG][N]
    const int row_l = lane & (CW - 1);                           // row of a chunk this lane keeps
    // Row sums: each thread its own keys' part per row, added up at the item's
    // end; with more than 32 rows the registers do not reach and the lanes'
    // parts are added up every tile (l[c]: row row_l of chunk c).
    constexpr bool OWN_SUMS = R <= 32;
    constexpr int NL = OWN_SUMS ? R : NCH;
    float m[NCH], l[NL];
    uint32_t joins = 0;
    bool ok = true;
    PagedWalk w = paged_walk(p, plan, lens);
    const int t0 = plan[4], total = plan[5], n_part = plan[3], G = gridDim.x;
    int k_start = 0, in_item = 0;  // the item's first tile in this part; its tiles so far
    for (int i = 0; ok && w.rem > 0; ++i, w.next(p)) {
      if (w.first) {
        k_start = w.k;
        in_item = 0;
#pragma unroll
        for (int c = 0; c < NCH; ++c) m[c] = -INFINITY;
#pragma unroll
        for (int r = 0; r < NL; ++r) l[r] = 0.f;
      }
      ++in_item;
      if (i % Ly::NG == gr) {
      const int buf = i % Ly::NB, pbuf = i % Ly::PB, gi = i / Ly::NG;  // gi: tiles of this group
      if (!mbar_wait_warp(bar(Ly::B_SFULL + buf), (i / Ly::NB) & 1, ab, err, 1008)) { ok = false; break; }
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
      const int key0 = w.tile * 128, key = key0 + t;
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
        float* dst = p.scores + ((static_cast<size_t>(w.b) * p.Hkv + w.hkv) * p.max_tiles + w.k) *
                                    p.rows * 128 + t;
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
        if (lane < CW) wmax[((gi & 1) * 4 + wq) * N + c * CW + row_l] = v;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(Ly::B_XMAX + gr));
      if (!mbar_wait_warp(bar(Ly::B_XMAX + gr), gi & 1, ab, err, 1009)) { ok = false; break; }
      bool grow = false;
      float alpha[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const float* wm = wmax + (gi & 1) * 4 * N + c * CW + row_l;
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
          al[c * CW + row_l] = alpha[c];
        }
      }
      __syncwarp();
      // The group's four warps see the same maxima, so they agree here.
      if (__any_sync(0xffffffffu, grow)) {
        // The group's O^T holds its earlier tiles of the item once PV(i-NG) is
        // done (the next phase of that barrier needs this warp's P first).
        if (!mbar_wait_warp(bar(Ly::B_PVDONE + (i - Ly::NG) % Ly::NB), ((i - Ly::NG) / Ly::NB) & 1, ab, err, 1010)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t tO = tmem + lane_off + Ly::TM_O + ((w.item & 1) * Ly::NG + gr) * N;
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
        if constexpr (OWN_SUMS) {
#pragma unroll
          for (int r = 0; r < R; ++r) l[r] *= al[r];
        }
      }
      // P = exp2(s c - m c), to shared memory in the 16-bit type (the MMA's
      // operand); the row sums take the unrounded values.
      // (P's buffer: PV(i-NB) was done before S(i) was issued; with fewer P than
      // S buffers the later PV has to be waited for.)
      if (Ly::PB < Ly::NB && i >= Ly::PB &&
          !mbar_wait_warp(bar(Ly::B_PVDONE + (i - Ly::PB) % Ly::NB), ((i - Ly::PB) / Ly::NB) & 1, ab, err, 1016)) {
        ok = false;
        break;
      }
      uint8_t* prow = gbase + Ly::P_OFF + pbuf * Ly::PT + (t >> 6) * Ly::QCH;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        float x[CW];
#pragma unroll
        for (int r = 0; r < CW; ++r) {
          const int rr = c * CW + r;
          x[r] = ex2(fmaf(__uint_as_float(sr[rr]), sl2, -mbuf[rr]));
          *reinterpret_cast<T*>(prow + rr * 128 + (((t & 63) * 2) ^ ((rr & 7) << 4))) = static_cast<T>(x[r]);
        }
        if constexpr (OWN_SUMS) {
#pragma unroll
          for (int r = 0; r < CW; ++r) l[c * CW + r] += x[r];
        } else {
          l[c] = l[c] * alpha[c] + paged_rows_reduce<CW, false>(x, lane);
        }
      }
      if (!whole) {
        // V rows of keys nobody sees: zero, whatever the page holds there.  The
        // stage's last fill must have landed before its next one is waited for:
        // it was a K up to K_i (S_i is here), or at the latest V_{i - STAGES/2},
        // which PV_{i-NB}, done before S_i, does not cover when STAGES/2 < NB.
        // (PV_{i-LAST+NB} needs this tile's P, so that barrier is at most one
        // phase on.)
        constexpr int LAST = Ly::STAGES / 2;
        if (LAST < Ly::NB && i >= LAST &&
            !mbar_wait_warp(bar(Ly::B_PVDONE + (i - LAST) % Ly::NB), ((i - LAST) / Ly::NB) & 1, ab, err, 1018)) {
          ok = false;
          break;
        }
        const uint32_t vpos = min(n_part, i + 1 + Ly::NG) + i;  // V's place in the ring's order
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
      if (lane == 0) mbar_arrive(bar(Ly::B_PFULL + buf));  // (a group may be two tiles ahead of the MMA)
      }

      if (w.last()) {
        // ---- the item's end in this part: O^T / l and LSE, or a partial.  Both
        // groups leave their row sums and maxima; the groups take turns at the
        // rest, so the other goes on with the next item.  (It comes back to
        // these areas two items later, after that item's exchange with this one.)
        const int ob = w.item & 1;
        float* sx = sum_x + ob * 4 * Ly::NG * N;
        float* mx = max_x + ob * Ly::NG * N;
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          float v;
          if constexpr (OWN_SUMS) {
            float x[CW];
#pragma unroll
            for (int r = 0; r < CW; ++r) x[r] = l[c * CW + r];
            v = paged_rows_reduce<CW, false>(x, lane);
          } else {
            v = l[c];
          }
          if (lane < CW) {
            sx[warp * N + c * CW + row_l] = v;
            if (wq == 0) mx[gr * N + c * CW + row_l] = m[c];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_XSUM + ob));
        if (Ly::NG == 2 && gr != ob) continue;
        if (!mbar_wait_warp(bar(Ly::B_XSUM + ob), (w.item >> 1) & 1, ab, err, 1012)) { ok = false; break; }
        const bool direct = k_start == 0 && w.k + 1 == w.s.cnt;
        const int slot = 2 * blockIdx.x + (w.item > 0 ? 1 : 0);
        // Factors of the groups' O^T rows: mbuf for group 0, al for group 1.
#pragma unroll
        for (int c = 0; c < NCH; ++c) {
          const int rr = c * CW + row_l;
          float top = mx[rr], f[Ly::NG], sum = 0.f;
          if constexpr (Ly::NG == 2) top = fmaxf(top, mx[N + rr]);
#pragma unroll
          for (int x = 0; x < Ly::NG; ++x) {
            const float* ls = sx + 4 * x * N + rr;
            f[x] = mx[x * N + rr] == -INFINITY ? 0.f : ex2((mx[x * N + rr] - top) * sl2);
            sum += f[x] * ((ls[0] + ls[N]) + (ls[2 * N] + ls[3 * N]));
          }
          const float inv = sum > 0.f ? 1.f / sum : 0.f;
          if (lane < CW) {
            mbuf[rr] = f[0] * inv;
            if constexpr (Ly::NG == 2) al[rr] = f[1] * inv;
          }
          if (wq == 0 && lane < CW && rr < p.rows) {
            const float lse2 = sum == 0.f ? -INFINITY : top * sl2 + __log2f(sum);  // (NaN stays NaN)
            const int ql = rr * p.ginv >> 16;
            if (direct)
              p.LSE[(static_cast<size_t>(w.b) * p.H + w.hkv * p.g + rr - ql * p.g) * p.Lq + ql] =
                  lse2 * 0.6931471805599453f;
            else
              p.part_lse[static_cast<size_t>(slot) * p.rows + rr] = lse2;
          }
        }
        __syncwarp();
        if (!mbar_wait_warp(bar(Ly::B_OFULL + ob), (w.item >> 1) & 1, ab, err, 1013)) { ok = false; break; }
        tc_fence_after();
        // A group that had no tile of the item left nothing in its O.
        const bool has[2] = {in_item >= 2 || i % Ly::NG == 0, in_item >= 2 || i % Ly::NG == 1};
        if (t < D) {
          const uint32_t tO = tmem + lane_off + Ly::TM_O + ob * Ly::NG * N;
          T* dst = reinterpret_cast<T*>(p.O) + (static_cast<size_t>(w.b) * p.Lq * p.H + w.hkv * p.g) * D + t;
          float* part = p.part_o + static_cast<size_t>(slot) * p.rows * D + t;
          constexpr int OC = 16;
          int hh = 0;
#pragma unroll
          for (int c = 0; c < N / OC; ++c) {
            uint32_t o[Ly::NG][OC];
#pragma unroll
            for (int x = 0; x < Ly::NG; ++x) tmem_ld16(tO + x * N + OC * c, o[x]);
#pragma unroll
            for (int x = 0; x < Ly::NG; ++x) tmem_ld_wait16(o[x]);
            float v[OC];
#pragma unroll
            for (int r = 0; r < OC; ++r) {
              const int rr = c * OC + r;
              if (rr >= R) break;
              v[r] = has[0] ? __uint_as_float(o[0][r]) * mbuf[rr] : 0.f;
              if constexpr (Ly::NG == 2) v[r] = has[1] ? fmaf(__uint_as_float(o[1][r]), al[rr], v[r]) : v[r];
            }
            if (!direct) {
#pragma unroll
              for (int r = 0; r < OC; ++r)
                if (c * OC + r < R && c * OC + r < p.rows) part[(c * OC + r) * D] = v[r];
            } else {
#pragma unroll
              for (int r = 0; r < OC; ++r)
                if (c * OC + r < R && c * OC + r < p.rows) {
                  dst[static_cast<size_t>(hh) * D] = static_cast<T>(v[r]);
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
        if (!direct) {
          // ---- a partial: count it in; the CTA that comes last joins the item
          const int start = t0 + i - w.k;  // the item's first tile
          const int c0 = paged_part_of(total, G, start);
          const int c1 = paged_part_of(total, G, start + w.s.cnt - 1);
          unsigned long long* word = p.count + c0;
          const unsigned long long word_was = t == 0 ? __ldcg(word) : 0ull;
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(Ly::B_JOIN + 2 * gr));
          if (!mbar_wait_warp(bar(Ly::B_JOIN + 2 * gr), joins & 1, ab, err, 1014)) { ok = false; break; }
          int* flag = plan + 6 + gr;
          if (t == 0) {
            __threadfence();  // the group's partial, before the count
            const int last = paged_count_in(word, p.nonce, c1 - c0 + 1, word_was);
            if (last) __threadfence();  // the count, before the others' partials
            *flag = last;
            mbar_arrive(bar(Ly::B_JOIN + 2 * gr + 1));
          }
          if (!mbar_wait_warp(bar(Ly::B_JOIN + 2 * gr + 1), joins & 1, ab, err, 1015)) { ok = false; break; }
          ++joins;
          if (*flag) {
            const int slot0 = 2 * c0 + (start > paged_part(total, G, c0) ? 1 : 0);
            paged_join<D, T, R>(p, w.b, w.hkv, slot0, 2 * (c0 + 1), c1 - c0 + 1);
          }
        }
      }
    }
    // Empty sequences: O = 0, LSE = -inf.
    for (int b = blockIdx.x; gr == 0 && b < p.B; b += G) {
      if (p.lens[b] > 0) continue;
      T* dst = reinterpret_cast<T*>(p.O) + static_cast<size_t>(b) * p.Lq * p.H * D;
      for (int x = t; x < p.Lq * p.H * D; x += 128) dst[x] = static_cast<T>(0.f);
      for (int x = t; x < p.Lq * p.H; x += 128)
        p.LSE[static_cast<size_t>(b) * p.Lq * p.H + x] = -INFINITY;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == Ly::SW + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Ly::TMEM_COLS);
  }
}

// Add every visible key's attention weight, sum over the item's rows of
// exp(s - LSE), from the raw scores the decode kernel left.  Block (x, bh):
// tiles 8x .. 8x + 7 of the item's list; each key belongs to one thread.
__global__ void __launch_bounds__(256)
    fa_paged_weights_kernel(const PagedParams p, float* __restrict__ weights, long long wstride) {
  pdl_wait();
  __shared__ float lse2[128];
  const int bh = blockIdx.y, b = bh / p.Hkv, hkv = bh - b * p.Hkv;
  const PagedSeq s = paged_seq_of(p.lens[b], p);
  const int k0 = blockIdx.x * 8;
  if (k0 >= s.cnt) return;
  const int t = threadIdx.x & 127;
  if (threadIdx.x < p.rows) {
    const float v = p.LSE[(static_cast<size_t>(b) * p.H + hkv * p.g + t % p.g) * p.Lq + t / p.g];
    lse2[t] = v == -INFINITY ? 0.f : v * 1.4426950408889634f;  // (then every score is -inf)
  }
  __syncthreads();
  float* dst = weights + static_cast<long long>(bh) * wstride + t;
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int k = k0 + 2 * x + (threadIdx.x >> 7);
    if (k >= s.cnt) break;
    const int key0 = (k < s.ns ? k : s.lo + k - s.ns) * 128;
    if (key0 + t >= s.n) break;
    const float* src = p.scores + (static_cast<size_t>(bh) * p.max_tiles + k) * p.rows * 128 + t;
    float sum = 0.f;
#pragma unroll 4
    for (int r = 0; r < p.rows; ++r) {
      const float x = src[r * 128];  // -inf: hidden, also from a row whose LSE is NaN
      sum += x == -INFINITY ? 0.f : ex2(fmaf(x, p.sl2, -lse2[r]));
    }
    dst[key0] += sum;
  }
}

// Copy new keys and values into the pages, and set their slots' weights.
// One thread per 16 bytes of K (and of V).  One token of 8 sequences, 32 heads of
// D 64: 2.4 us, a launch.
__global__ void __launch_bounds__(256)
    fa_paged_write_kernel(const uint4* __restrict__ k, const uint4* __restrict__ v,
                          uint4* __restrict__ kc, uint4* __restrict__ vc, long long k_page,
                          long long v_page, const int* __restrict__ table,
                          const int* __restrict__ start, const int* __restrict__ counts,
                          float* __restrict__ weights, long long wstride,
                          const float* __restrict__ new_w, int B, int L, int Hkv, int units,
                          int page, int max_pages, int num_pages) {
  pdl_launch_dependents();
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
