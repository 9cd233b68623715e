// Internal (C++) entry points between the C ABI and the kernel units.
#pragma once

#include <cuda_runtime.h>

#include "../../include/fa.h"

namespace fa {

fa_status run_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Lq,
                  int Lk, int H, int Hkv, int D, int causal, int dtype, cudaStream_t s);
fa_status run_fwd_fp8(const void* Q8, const void* K8, const void* V8, float q_scale, float k_scale,
                      float v_scale, void* O, float* LSE, int B, int Lq, int Lk, int H, int Hkv,
                      int causal, int out_dtype, cudaStream_t s);
fa_status run_window_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                         int Lq, int Lk, int H, int Hkv, int D, int window, int sinks, int dtype,
                         cudaStream_t s);
unsigned int fwd_read_error(cudaStream_t s);
fa_status run_selftest_wait(unsigned long long limit_ns, cudaStream_t s);

fa_status run_bwd_prep(const void* O, const void* dO, float* Delta, float* dq_accum, int B, int L,
                       int H, int D, int dtype, cudaStream_t s);
fa_status run_bwd(const void* Q, const void* K, const void* V, const void* dO, const float* LSE,
                  const float* Delta, void* dQ, void* dK, void* dV, float* dq_accum,
                  int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                  int dtype, cudaStream_t s);
fa_status run_bwd_main(const void* Q, const void* K, const void* V, const void* dO,
                       const float* LSE, const float* Delta, void* dK, void* dV, float* dq_accum,
                       int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                       int dtype, cudaStream_t s);
fa_status run_bwd_post(const float* dq_accum, void* dQ, int B, int L, int H, int D, int dtype,
                       cudaStream_t s);
fa_status run_window_bwd(const void* Q, const void* K, const void* V, const void* dO,
                         const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                         float* ws, size_t ws_bytes, int zero_accum, int B, int Lq, int Lk, int H,
                         int Hkv, int D, int window, int sinks, int dtype, cudaStream_t s);
size_t window_bwd_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D, int window,
                                 int sinks);
unsigned int bwd_read_error(cudaStream_t s);
fa_status run_bwd_noalloc(const void* Q, const void* K, const void* V, const void* dO,
                          const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                          int B, int L, int H, int Hkv, int D, int causal, int dtype,
                          cudaStream_t s);

// Split-KV decoding (decode.cu).
struct DecodePlan {
  int nsplit;  // key slices per (batch, K/V head)
  int tps;     // 128-key tiles per slice
  int n_kv;    // 128-key tiles in all
};
DecodePlan decode_plan(int B, int Lq, int Lk, int H, int Hkv, int sms);
size_t decode_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D);
fa_status run_decode(const void* Q, const void* K, const void* V, void* O, float* LSE, void* ws,
                     size_t ws_bytes, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                     int dtype, cudaStream_t s);
fa_status run_decode_slices(const void* Q, const void* K, const void* V, void* ws, size_t ws_bytes,
                            int B, int Lq, int Lk, int H, int Hkv, int D, int causal, int dtype,
                            cudaStream_t s);
fa_status run_decode_merge(const void* ws, size_t ws_bytes, void* O, float* LSE, int B, int Lq,
                           int Lk, int H, int Hkv, int D, int dtype, cudaStream_t s);
unsigned int decode_read_error(cudaStream_t s);

// Paged cache (paged.cu).
struct PagedDecodeArgs {
  const void *Q, *K, *V;
  const int *table, *lens;
  void* O;
  float* LSE;
  float* weights;
  long long weights_stride, k_page_stride, v_page_stride;
  void* workspace;
  size_t workspace_bytes;
  int B, Lq, H, Hkv, D, page, max_pages, num_pages, window, sinks, dtype;
};
size_t paged_decode_workspace_size(int B, int Lq, long long cap, int H, int Hkv, int D, bool weights);
fa_status run_paged_decode(const PagedDecodeArgs& a, cudaStream_t s);
fa_status run_paged_write(const void* K, const void* V, void* Kc, void* Vc, long long k_page,
                          long long v_page, const int* table, const int* start, const int* counts,
                          float* weights, long long wstride, const float* new_w, int B, int L,
                          int Hkv, int D, int page, int max_pages, int num_pages, cudaStream_t s);
unsigned int paged_read_error(cudaStream_t s);

// Decoding behind shared prefixes (prefix.cu).
struct PrefixDecodeArgs {
  const void *Q, *K, *V;
  const int *prefix_table, *prefix_lens, *group_starts, *table, *lens;
  void* O;
  float* LSE;
  long long k_page_stride, v_page_stride;
  void* workspace;
  size_t workspace_bytes;
  int B, Lq, H, Hkv, D, page, groups, prefix_pages, max_pages, num_pages, dtype;
};
size_t paged_prefix_workspace_size(const PrefixDecodeArgs& a);
fa_status run_paged_prefix(const PrefixDecodeArgs& a, cudaStream_t s);
unsigned int prefix_read_error(cudaStream_t s);

// Rotary positions and the append to the paged cache (rope.cu).
struct RopeView {  // [B, L, heads, D], the last two dims contiguous
  const void* p;
  long long batch, token;  // elements between two batch entries, two tokens
};
struct RopeArgs {
  RopeView q, k, qy, ky;
  const void* table;
  const int* positions;
  int axes, B, L, H, Hkv, D, rotary, neighbours, back, dtype;
};
struct PagedAppendArgs {
  RopeView v;
  void *K_pool, *V_pool;
  const int *table, *start, *counts;
  float* weights;
  const float* new_weights;
  long long weights_stride, k_page_stride, v_page_stride;
  int page, max_pages, num_pages;
};
fa_status run_rope(const RopeArgs& a, cudaStream_t s);
fa_status run_paged_append(const RopeArgs& a, const PagedAppendArgs& c, cudaStream_t s);

// Eviction (evict.cu).
struct PagedEvictArgs {
  void *K, *V;
  const int *table, *lens, *dst_table;
  const float* weights;
  int *kept, *new_lens;
  float* new_weights;
  long long weights_stride, k_page_stride, v_page_stride;
  int B, Hkv, D, page, max_pages, dst_pages, num_pages, keep, sinks, recent;
};
fa_status run_paged_evict(const PagedEvictArgs& a, cudaStream_t s);

// Key weights of a prompt (weights.cu).
size_t key_weights_workspace_size();
fa_status run_key_weights(const void* Q, const void* K, const float* LSE, float* W, void* ws,
                          size_t ws_bytes, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                          int window, int sinks, int dtype, cudaStream_t s);
unsigned int weights_read_error(cudaStream_t s);

inline int padded_len(int L) { return (L + 127) / 128 * 128; }

}  // namespace fa
