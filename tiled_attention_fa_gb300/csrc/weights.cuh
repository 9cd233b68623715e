// Key weights of a prompt: how much attention every key has received,
//   W[b, hkv, j] = sum over the group's heads h and the queries i that see j of
//                  exp(q_i . k_j / sqrt(D) - LSE[b, h, i]),
// the column sums of the softmax, from the LSE the forward left.
//
// The scores are recomputed transposed, S^T = K_j Q_i^T, so a thread owns a key
// and adds up its row of exponentials; no maximum is needed, as LSE bounds
// every exponent by 0.  At D = 128 a 128 x 128 step costs the tensor core, the
// exponential unit (32 results per clock) 512 cycles each and the shared memory
// 768 (K_j and Q_i read by the MMAs, Q_i written); the kernel keeps all three
// going at once.
//   warps 0-15  exponentials: four groups of four warps, group w takes the
//               steps w, w + 4, ... from TMEM buffer w (thread = key).  It takes
//               four: a group spends as long on barriers and on its own next
//               MMA as on exponentials
//   warp  16    TMA producer: K_j per item (two slots), Q_i through a ring
//   warp  17    TMEM allocation, MMA issue
//   warp  18    -LSE * log2e of each step's 128 queries into shared memory; its
//               arrival and the MMA's complete the same barrier
// Each role walks item by item and counts its steps in a tight inner loop: with
// one general step iterator (some 60 instructions a step, in warps that issue
// one every few cycles) a step took 1180 cycles.
// Work: an item is one (batch, K/V head, 128-key tile), its steps the group's
// heads times the Q tiles that see it.  Under causal masking items differ by
// the whole length, so the steps of all items form one list and CTA c takes
// the c-th of G equal contiguous parts.  An item cut by a part's border leaves
// 128 partial sums per part, added up in order by a second kernel: the result
// does not depend on timing.
// Measured: B1 H32/8 L4096 D128, all keys: 70 us, 983 TFLOP/s of the products
// (52% of the bf16 burst rate; the exponentials alone need 29 us), 1050 cycles
// a step; B2 H16 L8192 D64 causal 198 us.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "ptx.cuh"

namespace fa {

struct KwMeta {
  int n;           // steps of the part (0: nothing)
  int first_open;  // 1: the first item goes on in a later part
  int last_item;   // item that starts here and goes on later (bh * n_kv + j), else -1
  int last_slot;   // its partial slot
};

struct KwParams {
  const float* LSE;  // [B, H, Lq]
  float* W;          // [B, Hkv, Lk]
  KwMeta* meta;      // [G]
  float* part;       // [2 G, 128]
  int B, Lq, Lk, H, Hkv, g, causal, past;
  int n_kv, n_q;
  int window, sinks;  // window 0: none
  float sl2;
};

// Q tiles [i0, i1) that see K/V tile j.
__host__ __device__ inline void kw_range(const KwParams& p, int j, int& i0, int& i1) {
  i0 = 0;
  i1 = p.n_q;
  if (!p.causal) return;
  const int d = j * 128 - p.past;
  i0 = d > 0 ? d / 128 : 0;
  if (p.window && j * 128 >= p.sinks) {
    const int last = d + 126 + p.window;  // last query that sees a key of the tile
    const int e = last < 0 ? 0 : last / 128 + 1;
    if (e < i1) i1 = e;
    if (i1 < i0) i1 = i0;
  }
}

// Walk over the items of one part.  Step s of the item (s < n) is head
// (off + s) / per of the group and Q tile i0 + (off + s) % per.
struct KwWalk {
  int n;        // steps of this item in the part (0: the part is done)
  int off;      // steps of the item before this part
  int i0, per;  // Q tiles [i0, i0 + per)
  int rem;      // steps of the part behind this item
  int item;     // items of the part before this one
  bool ends;    // the item's last step lies in this part
  int bh, j;

  __device__ __forceinline__ void enter(const KwParams& p, int from, int left) {
    int i1;
    kw_range(p, j, i0, i1);
    per = i1 - i0;
    off = from;
    const int all = per * p.g - off;
    n = min(all, left);
    ends = all <= left;
    rem = left - n;
  }
  __device__ __forceinline__ void next(const KwParams& p) {
    ++item;
    if (rem == 0) {
      n = 0;
      return;
    }
    do {
      if (++j == p.n_kv) {
        j = 0;
        if (++bh >= p.B * p.Hkv) {
          n = 0;
          return;
        }
      }
      enter(p, 0, rem);
    } while (per == 0);
  }
};

template <int D>
struct KwLayout {
  static constexpr int KCH = D / 64;
  static constexpr uint32_t CHUNK = 128u * 128u;
  static constexpr uint32_t TILE = KCH * CHUNK;
  static constexpr int STAGES = D == 64 ? 8 : 4, COMB = 16;
  static constexpr uint32_t K_OFF = 0;                       // two slots
  static constexpr uint32_t Q_OFF = 2 * TILE;                // STAGES tiles
  static constexpr int NG = 4;                               // groups, S buffers
  static constexpr uint32_t STAT_OFF = Q_OFF + STAGES * TILE;  // [NG][128] -LSE * log2e
  static constexpr uint32_t COMB_OFF = STAT_OFF + NG * 512u;   // [COMB][NG - 1][128] sums
  static constexpr uint32_t BAR_OFF = COMB_OFF + COMB * (NG - 1) * 512u;
  static constexpr int B_KFULL = 0, B_KEMPTY = 2, B_QFULL = 4, B_QEMPTY = B_QFULL + STAGES,
                       B_SFULL = B_QEMPTY + STAGES, B_SEMPTY = B_SFULL + NG, B_CFULL = B_SEMPTY + NG,
                       B_DONE = B_CFULL + COMB, NBAR = B_DONE + 1;
  static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;
  static constexpr uint32_t SMEM_USED = MISC_OFF + 192;
  static constexpr uint32_t SMEM_ALLOC = SMEM_USED + 1024;
  static constexpr int NTHREADS = 128 * NG + 96;
  static_assert(SMEM_ALLOC <= 232448, "shared memory");
};

// Start of part c of G: fills plan {bh, j, step within the item, steps}.
template <int NT>
__device__ __forceinline__ void kw_plan(const KwParams& p, int c, int G, long long* sums, int* plan) {
  const int per = (p.n_kv + NT - 1) / NT;
  const int j0 = min(p.n_kv, static_cast<int>(threadIdx.x) * per), j1 = min(p.n_kv, j0 + per);
  long long mine = 0;
  for (int j = j0; j < j1; ++j) {
    int a, e;
    kw_range(p, j, a, e);
    mine += static_cast<long long>(e - a) * p.g;
  }
  long long incl = mine;
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, h);
    if (lane_id() >= static_cast<uint32_t>(h)) incl += o;
  }
  if (lane_id() == 31) sums[warp_id()] = incl;
  if (threadIdx.x == 0) plan[3] = 0;
  __syncthreads();
  long long before = incl - mine, head = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w < static_cast<int>(warp_id())) before += sums[w];
    head += sums[w];
  }
  const long long total = head * p.B * p.Hkv;
  const long long t0 = total * c / G, t1 = total * (c + 1) / G;
  if (t1 > t0) {
    const long long bh = t0 / head, r = t0 - bh * head;
    if (r >= before && r < before + mine) {
      long long at = before;
      for (int j = j0; j < j1; ++j) {
        int a, e;
        kw_range(p, j, a, e);
        const long long steps = static_cast<long long>(e - a) * p.g;
        if (r < at + steps) {
          plan[0] = static_cast<int>(bh);
          plan[1] = j;
          plan[2] = static_cast<int>(r - at);
          plan[3] = static_cast<int>(t1 - t0);
          break;
        }
        at += steps;
      }
    }
  }
  __syncthreads();
}

__device__ __forceinline__ KwWalk kw_walk(const KwParams& p, const int* plan) {
  KwWalk w;
  w.bh = plan[0];
  w.j = plan[1];
  w.item = 0;
  w.n = w.rem = 0;
  if (plan[3] > 0) w.enter(p, plan[2], plan[3]);
  return w;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(608, 1)
    fa_key_weights_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK, const KwParams p) {
  using Ly = KwLayout<D>;
  constexpr uint32_t IDESC_S = idesc_f16(BF16, 128, 128, false, false);

  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) -> uint32_t { return base + Ly::BAR_OFF + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(gbase + Ly::MISC_OFF);
  AbortState* ab = reinterpret_cast<AbortState*>(gbase + Ly::MISC_OFF + 8);
  int* plan = reinterpret_cast<int*>(gbase + Ly::MISC_OFF + 16);
  long long* sums = reinterpret_cast<long long*>(gbase + Ly::MISC_OFF + 32);
  float* stats = reinterpret_cast<float*>(gbase + Ly::STAT_OFF);
  float* comb = reinterpret_cast<float*>(gbase + Ly::COMB_OFF);
  unsigned int* err = device_error_word();
  const uint32_t warp = warp_id(), lane = lane_id();

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(Ly::B_KFULL + s), 1);
      mbar_init(bar(Ly::B_KEMPTY + s), 1);
    }
    for (int s = 0; s < Ly::STAGES; ++s) {
      mbar_init(bar(Ly::B_QFULL + s), 1);
      mbar_init(bar(Ly::B_QEMPTY + s), 1);
    }
    for (int s = 0; s < Ly::NG; ++s) {
      mbar_init(bar(Ly::B_SFULL + s), 2);  // the MMA and the LSE warp
      mbar_init(bar(Ly::B_SEMPTY + s), 4);
    }
    for (int s = 0; s < Ly::COMB; ++s) mbar_init(bar(Ly::B_CFULL + s), 4 * (Ly::NG - 1));
    mbar_init(bar(Ly::B_DONE), 1);
    ab->flag = 0;
    fence_barrier_init();
  }
  if (warp == 17) {
    tmem_alloc(base + Ly::MISC_OFF, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  kw_plan<Ly::NTHREADS>(p, blockIdx.x, gridDim.x, sums, plan);
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  KwWalk w = kw_walk(p, plan);
  if (warp == 16) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    uint32_t stage = 0, phase = 0;
    int done = 0;
    for (; ok && w.n > 0; w.next(p)) {
      const int b = w.bh / p.Hkv, hkv = w.bh - b * p.Hkv;
      const uint32_t slot = w.item & 1;
      if (w.item >= 2 && !mbar_wait_warp(bar(Ly::B_KEMPTY + slot), ((w.item >> 1) - 1) & 1, ab, err, 1101)) {
        ok = false;
        break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(Ly::B_KFULL + slot), Ly::TILE);
        for (int c = 0; c < Ly::KCH; ++c)
          tma_load_4d(base + Ly::K_OFF + slot * Ly::TILE + c * Ly::CHUNK, &tmK,
                      bar(Ly::B_KFULL + slot), c * 64, hkv, w.j * 128, b);
      }
      int h = w.off / w.per, i = w.i0 + w.off - h * w.per;
      h += hkv * p.g;
      for (int s = 0; s < w.n; ++s) {
        if (!mbar_wait_warp(bar(Ly::B_QEMPTY + stage), phase ^ 1u, ab, err, 1102)) { ok = false; break; }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(Ly::B_QFULL + stage), Ly::TILE);
#pragma unroll
          for (int c = 0; c < Ly::KCH; ++c)
            tma_load_4d(base + Ly::Q_OFF + stage * Ly::TILE + c * Ly::CHUNK, &tmQ,
                        bar(Ly::B_QFULL + stage), c * 64, h, i * 128, b);
        }
        ++done;
        if (++stage == Ly::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++i == w.i0 + w.per) {
          i = w.i0;
          ++h;
        }
      }
    }
    if (!ok && lane == 0) {
      // Unwinding: let copies in flight land.
      for (int c = w.item > 1 ? w.item - 1 : 0; c <= w.item; ++c)
        mbar_wait_drain(bar(Ly::B_KFULL + (c & 1)), (c >> 1) & 1);
      for (int c = done > Ly::STAGES ? done - Ly::STAGES : 0; c < done; ++c)
        mbar_wait_drain(bar(Ly::B_QFULL + c % Ly::STAGES), (c / Ly::STAGES) & 1);
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------ MMA issuer
    bool ok = true;
    uint32_t stage = 0, phase = 0, buf = 0, use = 0;  // use: rounds of the S buffers
    for (; ok && w.n > 0; w.next(p)) {
      const uint32_t slot = w.item & 1;
      if (!mbar_wait_warp(bar(Ly::B_KFULL + slot), (w.item >> 1) & 1, ab, err, 1103)) { ok = false; break; }
      const uint64_t kd = sdesc_sw128(base + Ly::K_OFF + slot * Ly::TILE, 16, 1024);
      for (int s = 0; s < w.n; ++s) {
        if (!mbar_wait_warp(bar(Ly::B_QFULL + stage), phase, ab, err, 1104)) { ok = false; break; }
        const uint64_t qd = sdesc_sw128(base + Ly::Q_OFF + stage * Ly::TILE, 16, 1024);
        if (!mbar_wait_warp(bar(Ly::B_SEMPTY + buf), (use & 1) ^ 1u, ab, err, 1105)) { ok = false; break; }
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint64_t off = ((k >> 2) * Ly::CHUNK + (k & 3) * 32u) >> 4;
            mma_ss(tmem + 128 * buf, kd + off, qd + off, IDESC_S, k > 0 ? 1u : 0u);
          }
          tc_commit(bar(Ly::B_SFULL + buf));
          tc_commit(bar(Ly::B_QEMPTY + stage));
          if (s + 1 == w.n) tc_commit(bar(Ly::B_KEMPTY + slot));
        }
        __syncwarp();
        if (++buf == Ly::NG) {
          buf = 0;
          ++use;
        }
        if (++stage == Ly::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (elect_one()) tc_commit(bar(Ly::B_DONE));
    __syncwarp();
    mbar_wait_drain(bar(Ly::B_DONE), 0);
  } else if (warp == 18) {
    // ------------------------------------------------------------ LSE of the queries
    // Read one step ahead.  A query past the end, or one that sees nothing
    // (LSE = -inf), gets -inf and adds nothing.
    bool ok = true;
    uint32_t buf = 0, use = 0;
    for (; ok && w.n > 0; w.next(p)) {
      int h = w.off / w.per, i = w.i0 + w.off - h * w.per;
      const float* row = p.LSE + (static_cast<size_t>(w.bh) * p.g + h) * p.Lq;
      float next[4];
      auto fetch = [&]() {
        const int q0 = i * 128 + lane;
#pragma unroll
        for (int u = 0; u < 4; ++u) next[u] = q0 + 32 * u < p.Lq ? row[q0 + 32 * u] : -INFINITY;
        if (++i == w.i0 + w.per) {
          i = w.i0;
          row += p.Lq;
        }
      };
      fetch();
      for (int s = 0; s < w.n; ++s) {
        float cur[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          cur[u] = next[u] == -INFINITY ? -INFINITY : -next[u] * 1.4426950408889634f;
        if (s + 1 < w.n) fetch();
        if (!mbar_wait_warp(bar(Ly::B_SEMPTY + buf), (use & 1) ^ 1u, ab, err, 1108)) { ok = false; break; }
#pragma unroll
        for (int u = 0; u < 4; ++u) stats[buf * 128 + lane + 32 * u] = cur[u];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_SFULL + buf));
        if (++buf == Ly::NG) {
          buf = 0;
          ++use;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ exponentials and sums
    const int wg = warp >> 2, t = threadIdx.x & 127;
    const uint32_t lane_off = ((warp & 3u) * 32u) << 16;
    const float sl2 = p.sl2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    bool ok = true;
    int first_open = 0, last_item = -1, last_slot = 0;
    const uint32_t tS = tmem + lane_off + 128 * wg;
    const float* st = stats + wg * 128;
    uint32_t use = 0;
    const int total = w.n + w.rem;
    int skip = wg;  // steps until this group's next one
    for (; ok && w.n > 0; w.next(p)) {
      const int key = w.j * 128 + t;
      float sum = 0.f;
      const int d0 = key - p.past;
      const bool windowed = p.window && key >= p.sinks;
      int s = skip;
      int i = w.i0 + (w.off + skip) % w.per;  // Q tile of step s
      for (; s < w.n; s += Ly::NG) {
        if (!mbar_wait_warp(bar(Ly::B_SFULL + wg), use & 1, ab, err, 1106)) { ok = false; break; }
        ++use;
        tc_fence_after();
        // Query columns [lo, hi) see this key.
        const int d = d0 - i * 128;
        int lo = 0, hi = 128;
        if (p.causal) lo = max(0, d);
        if (windowed) hi = min(hi, d + p.window);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        uint32_t sv[32];
        auto chunk = [&](int c, const uint32_t* x, auto masked) {
          const uint4* nl4 = reinterpret_cast<const uint4*>(st + c);
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 l4 = nl4[u];
            float a[4], e[4];
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[4 * u]), __uint_as_float(x[4 * u + 1])), sl2x2,
                            f2_pack(__uint_as_float(l4.x), __uint_as_float(l4.y))), a[0], a[1]);
            f2_unpack(ffma2(f2_pack(__uint_as_float(x[4 * u + 2]), __uint_as_float(x[4 * u + 3])), sl2x2,
                            f2_pack(__uint_as_float(l4.z), __uint_as_float(l4.w))), a[2], a[3]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              e[y] = ex2(a[y]);
              if constexpr (decltype(masked)::value) {
                const int q = c + 4 * u + y;
                e[y] = (q >= lo && q < hi) ? e[y] : 0.f;
              }
            }
            acc[2 * (u & 1)] = fadd2(acc[2 * (u & 1)], f2_pack(e[0], e[1]));
            acc[2 * (u & 1) + 1] = fadd2(acc[2 * (u & 1) + 1], f2_pack(e[2], e[3]));
          }
        };
        // Not unrolled: four groups and two versions of the loop share the
        // instruction cache.
        if (__all_sync(0xffffffffu, lo <= 0 && hi >= 128)) {
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            tmem_ld32(tS + c, sv);
            tmem_ld_wait32(sv);
            chunk(c, sv, std::false_type{});
          }
        } else {
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            tmem_ld32(tS + c, sv);
            tmem_ld_wait32(sv);
            chunk(c, sv, std::true_type{});
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_SEMPTY + wg));
        float x[8];
#pragma unroll
        for (int y = 0; y < 4; ++y) f2_unpack(acc[y], x[2 * y], x[2 * y + 1]);
        sum += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
        i += Ly::NG;
        while (i >= w.i0 + w.per) i -= w.per;
      }
      if (!ok) break;
      skip = s - w.n;
      // The item's end in this part: groups 1-3 hand their sums to group 0.  A
      // slot is used again 16 items, so at least 16 steps, later, and no group
      // is that far ahead: group 0's next step is at most four past this item's
      // end, the S buffers let the others finish three more, and walk over
      // three that are not theirs.
      const int cs = w.item % Ly::COMB;
      float* cb = comb + cs * (Ly::NG - 1) * 128 + t;
      if (wg != 0) {
        cb[(wg - 1) * 128] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(Ly::B_CFULL + cs));
      } else {
        if (!mbar_wait_warp(bar(Ly::B_CFULL + cs), (w.item / Ly::COMB) & 1, ab, err, 1107)) { ok = false; break; }
        const float v = (sum + cb[0]) + (cb[128] + cb[256]);
        const bool starts = w.off == 0;
        if (starts && w.ends) {
          if (key < p.Lk) p.W[static_cast<size_t>(w.bh) * p.Lk + key] = v;
        } else {
          const int slot = 2 * blockIdx.x + (w.item > 0 ? 1 : 0);
          p.part[static_cast<size_t>(slot) * 128 + t] = v;
          if (w.item == 0 && !w.ends) first_open = 1;
          if (starts) {
            last_item = w.bh * p.n_kv + w.j;
            last_slot = slot;
          }
        }
      }
    }
    if (threadIdx.x == 0) p.meta[blockIdx.x] = KwMeta{ok ? total : 0, first_open, ok ? last_item : -1, last_slot};
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Block c adds up, in order, the partial sums of the item that starts in part
// c and goes on in the next ones; and it writes the zeros of the K/V tiles c,
// c + G, ... of a head that no query sees, for every head.
__global__ void __launch_bounds__(128) fa_key_weights_join_kernel(const KwParams p, int G) {
  pdl_wait();
  const int c = blockIdx.x, t = threadIdx.x;
  if (p.window) {
    for (int j = c; j < p.n_kv; j += G) {
      int i0, i1;
      kw_range(p, j, i0, i1);
      if (i0 < i1 || j * 128 + t >= p.Lk) continue;
      for (int bh = 0; bh < p.B * p.Hkv; ++bh) p.W[static_cast<size_t>(bh) * p.Lk + j * 128 + t] = 0.f;
    }
  }
  const KwMeta mt = p.meta[c];
  if (mt.n == 0 || mt.last_item < 0) return;
  float sum = p.part[static_cast<size_t>(mt.last_slot) * 128 + t];
  for (int q = c + 1; q < G; ++q) {
    const KwMeta m = p.meta[q];
    if (m.n == 0) continue;
    sum += p.part[static_cast<size_t>(2 * q) * 128 + t];
    if (!m.first_open) break;
  }
  const int bh = mt.last_item / p.n_kv, key = (mt.last_item - bh * p.n_kv) * 128 + t;
  if (key < p.Lk) p.W[static_cast<size_t>(bh) * p.Lk + key] = sum;
}

}  // namespace fa
