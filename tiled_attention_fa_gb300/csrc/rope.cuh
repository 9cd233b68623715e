// Rotary positions: queries and keys (or their gradients) turned by their
// positions, and the append of new tokens to a paged cache with the keys turned
// on their way into the pages.
//
// Mathematics: the first `rotary` dims of a head are rotary / 2 pairs (x, y);
// pair i of a token at position n (on the pair's axis) becomes
//   (x cos t - y sin t, x sin t + y cos t),   t = n f_i,
// the backward pass turns by -t.  The pairs are halves (i, i + rotary / 2) or
// neighbours (2 i, 2 i + 1).
//
// Angles: the table holds f_i / 2 pi, the turns a position adds, as a 64-bit
// fixed-point fraction whose low 8 bits are the pair's axis.  The turns of
// position n are the product of two integers modulo 2^64, exact for every 32-bit
// position (what the entry itself is off by grows with it); its top 32 bits are
// the angle, to which sincospif answers in 32 bits.  An fp32 product n f_i at n = 100,000 is
// already off by 2^-8 rad.
//
// Bound by the read and the write of the heads.  A thread owns one unit of a
// token's heads, two 16-byte vectors that hold 8 whole pairs (or 16 dims that
// are not turned), and so 8 angles, which it computes once and uses for every
// 2^hs_log-th head of the token: no table of cosines is read or kept.  It loads
// the units of two heads before it turns the first, which fits 64 registers and so
// four blocks an SM (four heads, 94 registers: append of B4 L2047 32.9 us, now 30.1).
// Measured (bf16, H32/8 D128, in a graph): B1 L8192 28.2 us, 6.0 TB/s with the
// launch; B4 L4096, 3 axes, forward and backward 108 us, 6.2 TB/s; append of B4
// L2047 30.2 us; B1 L200 3.5 us; append of B256 L1 4.6 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "common.cuh"
#include "fwd.cuh"  // pack2
#include "ptx.cuh"

namespace fa {

// One tensor [B, L, heads, D] and where its turned form goes; strides between
// batch entries and tokens in 16-byte vectors.
struct RopeTensor {
  const uint4* x;
  uint4* y;
  long long xb, xt, yb, yt;
};

struct RopeParams {
  RopeTensor q, k, v;      // (append: k.y, v.y are the pools; v unused otherwise)
  const longlong2* table;  // rotary / 2 entries
  const int* pos;          // [axes, B, L], or NULL: the token's number (append: its slot)
  int axes, B, L, H, Hkv;  // Hkv 0: no keys
  int nrot;                // turned units of a head: rotary / 16
  int hs_log;              // threads per unit of a token: 2^hs_log
  int back;                // turn by -t
  // append
  const int *block_table, *start, *counts;
  long long k_page, v_page;  // vectors between two pages
  float* weights;
  const float* new_w;
  long long wstride;
  int page_log, max_pages, num_pages;
};

template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t v) {
  return __half22float2(*reinterpret_cast<const __half2*>(&v));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t v) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

// Turn the 8 pairs of a unit; each result is rounded once, to the tensor's type.
template <typename T, bool NEIGHBOURS>
__device__ __forceinline__ void rope_turn(uint4& lo, uint4& hi, const float (&cs)[8], const float (&sn)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const float2 u = unpack2<T>(a[w]), v = unpack2<T>(b[w]);
    if constexpr (NEIGHBOURS) {  // u is pair w, v pair 4 + w
      a[w] = pack2<T>(u.x * cs[w] - u.y * sn[w], u.x * sn[w] + u.y * cs[w]);
      b[w] = pack2<T>(v.x * cs[4 + w] - v.y * sn[4 + w], v.x * sn[4 + w] + v.y * cs[4 + w]);
    } else {  // u the x of pairs 2w, 2w + 1, v their y
      a[w] = pack2<T>(u.x * cs[2 * w] - v.x * sn[2 * w], u.y * cs[2 * w + 1] - v.y * sn[2 * w + 1]);
      b[w] = pack2<T>(u.x * sn[2 * w] + v.x * cs[2 * w], u.y * sn[2 * w + 1] + v.y * cs[2 * w + 1]);
    }
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

// UN = D / 16 units a head.
template <typename T, int UN, bool NEIGHBOURS, bool APPEND>
__global__ void __launch_bounds__(256, 4) fa_rope_kernel(const RopeParams p) {
  constexpr int ROWS = 256 / UN, C = 2;
  const int u = threadIdx.x % UN, row = threadIdx.x / UN;
  const int HS = 1 << p.hs_log, hs = row & (HS - 1);
  const long long tokens = static_cast<long long>(p.B) * p.L;
  const long long tok = static_cast<long long>(blockIdx.x) * (ROWS >> p.hs_log) + (row >> p.hs_log);
  if (tok >= tokens) return;
  // (B * L is below 2^31 wherever H * B * L is)
  const int b = static_cast<int>(static_cast<unsigned>(tok) / static_cast<unsigned>(p.L));
  const int j = static_cast<int>(tok) - b * p.L;

  pdl_launch_dependents();
  pdl_wait();
  const uint4* qx = p.q.x + b * p.q.xb + j * p.q.xt;
  const uint4* kx = p.k.x + b * p.k.xb + j * p.k.xt;
  const uint4* vx = p.v.x + b * p.v.xb + j * p.v.xt;
  uint4* qy = p.q.y + b * p.q.yb + j * p.q.yt;
  uint4* ky = p.k.y;
  uint4* vy = p.v.y;
  bool put = true;  // keys (and values) have a place
  long long at = j, slot = 0;
  if constexpr (APPEND) {
    // (page_log < 9; a slot beyond the table is above every int's shift)
    slot = at = static_cast<long long>(p.start[b]) + j;
    put = (p.counts == nullptr || j < p.counts[b]) && slot >= 0 && (slot >> p.page_log) < p.max_pages;
    if (put) {
      const int pid = p.block_table[static_cast<long long>(b) * p.max_pages + (slot >> p.page_log)];
      put = pid >= 0 && pid < p.num_pages;
      const long long in_page = (slot & ((1 << p.page_log) - 1)) * static_cast<long long>(p.Hkv) * (2 * UN);
      ky += (put ? pid : 0) * p.k_page + in_page;
      vy += (put ? pid : 0) * p.v_page + in_page;
    }
  } else {
    ky += b * p.k.yb + j * p.k.yt;
  }

  float cs[8], sn[8];
  const bool turn = u < p.nrot;
  if (turn) {
    if (p.pos != nullptr && p.axes == 1) at = p.pos[tok];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const longlong2 e = p.table[4 * u + i];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const long long f = x ? e.y : e.x;
        if (p.axes > 1) at = p.pos[min(static_cast<int>(f & 255), p.axes - 1) * tokens + tok];
        const unsigned long long turns =
            (static_cast<unsigned long long>(f) & ~255ull) * static_cast<unsigned long long>(at);
        // half turns in [-1, 1)
        const float t = static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f;
        sincospif(t, &sn[2 * i + x], &cs[2 * i + x]);
        if (p.back) sn[2 * i + x] = -sn[2 * i + x];
      }
    }
  }
  // The unit's vectors in a head.
  const int o1 = turn ? (NEIGHBOURS ? 2 * u : u) : 2 * u;
  const int o2 = turn && !NEIGHBOURS ? u + p.nrot : o1 + 1;

  const int turned = p.H + p.Hkv, all = APPEND ? turned + p.Hkv : turned;
#pragma unroll 1
  for (int h0 = hs; h0 < all; h0 += C * HS) {
    uint4 lo[C], hi[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = h0 + c * HS;
      if (h < all && (h < p.H || put)) {
        const uint4* x = h < p.H ? qx + h * (2 * UN) : h < turned ? kx + (h - p.H) * (2 * UN) : vx + (h - turned) * (2 * UN);
        lo[c] = x[o1];
        hi[c] = x[o2];
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int h = h0 + c * HS;
      if (h < all && (h < p.H || put)) {
        if (turn && h < turned) rope_turn<T, NEIGHBOURS>(lo[c], hi[c], cs, sn);
        uint4* y = h < p.H ? qy + h * (2 * UN) : h < turned ? ky + (h - p.H) * (2 * UN) : vy + (h - turned) * (2 * UN);
        y[o1] = lo[c];
        y[o2] = hi[c];
        if constexpr (APPEND) {
          if (p.weights != nullptr && u == 0 && h >= p.H && h < turned) {
            const long long bh = static_cast<long long>(b) * p.Hkv + h - p.H;
            p.weights[bh * p.wstride + slot] = p.new_w != nullptr ? p.new_w[bh * p.L + j] : 0.f;
          }
        }
      }
    }
  }
}

}  // namespace fa
