// C ABI: argument validation and dispatch to the kernel units.
#include <cmath>
#include <cstdint>

#include "../../include/fa.h"
#include "internal.h"

namespace {

unsigned int g_last_site = 0;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Index arrays (tables, lengths) need their element's alignment only.
bool ints_ok(const int* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

bool ptr_ok(const void* p) { return p != nullptr && aligned16(p); }

// Do two buffers of na and nb bytes share any?
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Bytes of key weights [pairs, n] fp32 whose rows lie `stride` apart.
size_t weights_bytes(long long pairs, long long stride, long long n) {
  return static_cast<size_t>((pairs - 1) * stride + n) * sizeof(float);
}

// Lq query rows, Lk key rows (equal for the square entry points).
fa_status check_shape(int B, int Lq, int Lk, int H, int Hkv, int D, int dtype) {
  if (B < 1 || Lq < 1 || Lk < 1 || H < 1 || Hkv < 1) return FA_ERR_INVALID_ARG;
  if (Lq > (1 << 30) || Lk > (1 << 30) || H > (1 << 20) || B > (1 << 20)) return FA_ERR_INVALID_ARG;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  // Work-item and element counts must fit the kernels' integer arithmetic.
  const int Lmax = Lq > Lk ? Lq : Lk;
  const long long items = static_cast<long long>(B) * H * ((Lmax + 127) / 128);
  const long long elems = static_cast<long long>(B) * fa::padded_len(Lmax) * H * D;
  if (items >= (1ll << 31) || elems >= (1ll << 40)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * H * fa::padded_len(Lmax) >= (1ll << 31)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_shape(int B, int L, int H, int Hkv, int D, int dtype) {
  return check_shape(B, L, L, H, Hkv, D, dtype);
}

}  // namespace

extern "C" {

fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int L,
                 int H, int Hkv, int D, int causal, int dtype, void* stream) {
  fa_status st = check_shape(B, L, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(O) || !ptr_ok(LSE))
    return FA_ERR_INVALID_ARG;
  return fa::run_fwd(Q, K, V, O, LSE, B, L, L, H, Hkv, D, causal, dtype,
                     static_cast<cudaStream_t>(stream));
}

fa_status fa_fwd_kv(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Lq,
                    int Lk, int H, int Hkv, int D, int causal, int dtype, void* stream) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (causal && Lk < Lq) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(O) || !ptr_ok(LSE))
    return FA_ERR_INVALID_ARG;
  return fa::run_fwd(Q, K, V, O, LSE, B, Lq, Lk, H, Hkv, D, causal, dtype,
                     static_cast<cudaStream_t>(stream));
}

fa_status fa_fwd_fp8(const void* Q8, const void* K8, const void* V8, float q_scale,
                     float k_scale, float v_scale, void* O, float* LSE, int B, int Lq, int Lk,
                     int H, int Hkv, int D, int causal, int out_dtype, void* stream) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, out_dtype);
  if (st != FA_OK) return st;
  if (D != 128) return FA_ERR_UNSUPPORTED;
  if (causal && Lk < Lq) return FA_ERR_INVALID_ARG;
  for (float sc : {q_scale, k_scale, v_scale})
    if (!(sc > 0.f) || !std::isfinite(sc)) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q8) || !ptr_ok(K8) || !ptr_ok(V8) || !ptr_ok(O) || !ptr_ok(LSE))
    return FA_ERR_INVALID_ARG;
  return fa::run_fwd_fp8(Q8, K8, V8, q_scale, k_scale, v_scale, O, LSE, B, Lq, Lk, H, Hkv, causal,
                         out_dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_bwd_preprocess(const void* O, const void* dO, float* Delta, float* dq_accum, int B,
                            int L, int H, int D, int dtype, void* stream) {
  fa_status st = check_shape(B, L, H, H, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(O) || !ptr_ok(dO) || !ptr_ok(Delta)) return FA_ERR_INVALID_ARG;
  if (dq_accum != nullptr && !aligned16(dq_accum)) return FA_ERR_INVALID_ARG;
  return fa::run_bwd_prep(O, dO, Delta, dq_accum, B, L, H, D, dtype,
                          static_cast<cudaStream_t>(stream));
}

size_t fa_bwd_workspace_size(int B, int L, int H, int D) {
  if (B < 1 || L < 1 || H < 1 || D < 1) return 0;
  return static_cast<size_t>(B) * H * fa::padded_len(L) * D * sizeof(float);
}

fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                 float* dq_accum, int zero_accum, int B, int L, int H, int Hkv, int D, int causal,
                 int dtype, void* stream) {
  (void)O;
  fa_status st = check_shape(B, L, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(dO) || !ptr_ok(LSE) || !ptr_ok(Delta) ||
      !ptr_ok(dQ) || !ptr_ok(dK) || !ptr_ok(dV) || !ptr_ok(dq_accum))
    return FA_ERR_INVALID_ARG;
  return fa::run_bwd(Q, K, V, dO, LSE, Delta, dQ, dK, dV, dq_accum, zero_accum, B, L, L, H, Hkv, D,
                     causal, dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_bwd_kv(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                    const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                    float* dq_accum, int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D,
                    int causal, int dtype, void* stream) {
  (void)O;
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (causal && Lk < Lq) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(dO) || !ptr_ok(LSE) || !ptr_ok(Delta) ||
      !ptr_ok(dQ) || !ptr_ok(dK) || !ptr_ok(dV) || !ptr_ok(dq_accum))
    return FA_ERR_INVALID_ARG;
  return fa::run_bwd(Q, K, V, dO, LSE, Delta, dQ, dK, dV, dq_accum, zero_accum, B, Lq, Lk, H, Hkv,
                     D, causal, dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_window_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                        int Lq, int Lk, int H, int Hkv, int D, int window, int sinks, int dtype,
                        void* stream) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (Lk < Lq || window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(O) || !ptr_ok(LSE))
    return FA_ERR_INVALID_ARG;
  return fa::run_window_fwd(Q, K, V, O, LSE, B, Lq, Lk, H, Hkv, D, window, sinks, dtype,
                            static_cast<cudaStream_t>(stream));
}

size_t fa_window_bwd_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D, int window,
                                    int sinks) {
  if (check_shape(B, Lq, Lk, H, Hkv, D, FA_F16) != FA_OK || Lk < Lq || window < 1 || sinks < 0)
    return 0;
  return fa::window_bwd_workspace_size(B, Lq, Lk, H, Hkv, D, window, sinks);
}

fa_status fa_window_bwd(const void* Q, const void* K, const void* V, const void* dO,
                        const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                        float* workspace, size_t workspace_bytes, int zero_accum, int B, int Lq,
                        int Lk, int H, int Hkv, int D, int window, int sinks, int dtype,
                        void* stream) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (Lk < Lq || window < 1 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(dO) || !ptr_ok(LSE) || !ptr_ok(Delta) ||
      !ptr_ok(dQ) || !ptr_ok(dK) || !ptr_ok(dV) || !ptr_ok(workspace))
    return FA_ERR_INVALID_ARG;
  return fa::run_window_bwd(Q, K, V, dO, LSE, Delta, dQ, dK, dV, workspace, workspace_bytes,
                            zero_accum, B, Lq, Lk, H, Hkv, D, window, sinks, dtype,
                            static_cast<cudaStream_t>(stream));
}

fa_status fa_bwd_main(const void* Q, const void* K, const void* V, const void* dO,
                      const float* LSE, const float* Delta, void* dK, void* dV, float* dq_accum,
                      int zero_accum, int B, int L, int H, int Hkv, int D, int causal, int dtype,
                      void* stream) {
  fa_status st = check_shape(B, L, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(dO) || !ptr_ok(LSE) || !ptr_ok(Delta) ||
      !ptr_ok(dK) || !ptr_ok(dV) || !ptr_ok(dq_accum))
    return FA_ERR_INVALID_ARG;
  return fa::run_bwd_main(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B, L, L, H, Hkv, D,
                          causal, dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_bwd_postprocess(const float* dq_accum, void* dQ, int B, int L, int H, int D,
                             int dtype, void* stream) {
  fa_status st = check_shape(B, L, H, H, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(dq_accum) || !ptr_ok(dQ)) return FA_ERR_INVALID_ARG;
  return fa::run_bwd_post(dq_accum, dQ, B, L, H, D, dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* LSE, const float* Delta, void* dQ,
                         void* dK, void* dV, int B, int L, int H, int Hkv, int D, int causal,
                         int dtype, void* stream) {
  (void)O;
  fa_status st = check_shape(B, L, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(dO) || !ptr_ok(LSE) || !ptr_ok(Delta) ||
      !ptr_ok(dQ) || !ptr_ok(dK) || !ptr_ok(dV))
    return FA_ERR_INVALID_ARG;
  return fa::run_bwd_noalloc(Q, K, V, dO, LSE, Delta, dQ, dK, dV, B, L, H, Hkv, D, causal, dtype,
                             static_cast<cudaStream_t>(stream));
}

size_t fa_decode_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D) {
  if (B < 1 || Lq < 1 || Lk < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || (D != 64 && D != 128))
    return 0;
  return fa::decode_workspace_size(B, Lq, Lk, H, Hkv, D);
}

namespace {
fa_status check_decode(int B, int Lq, int Lk, int H, int Hkv, int D, int causal, int dtype) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (causal && Lk < Lq) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(H / Hkv) * Lq > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}
}  // namespace

fa_status fa_decode(const void* Q, const void* K, const void* V, void* O, float* LSE,
                    void* workspace, size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv,
                    int D, int causal, int dtype, void* stream) {
  const fa_status st = check_decode(B, Lq, Lk, H, Hkv, D, causal, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(O) || !ptr_ok(LSE) || !ptr_ok(workspace))
    return FA_ERR_INVALID_ARG;
  return fa::run_decode(Q, K, V, O, LSE, workspace, workspace_bytes, B, Lq, Lk, H, Hkv, D, causal,
                        dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_decode_slices(const void* Q, const void* K, const void* V, void* workspace,
                           size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv, int D,
                           int causal, int dtype, void* stream) {
  const fa_status st = check_decode(B, Lq, Lk, H, Hkv, D, causal, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ptr_ok(workspace)) return FA_ERR_INVALID_ARG;
  return fa::run_decode_slices(Q, K, V, workspace, workspace_bytes, B, Lq, Lk, H, Hkv, D, causal,
                               dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_decode_merge(const void* workspace, size_t workspace_bytes, void* O, float* LSE, int B,
                          int Lq, int Lk, int H, int Hkv, int D, int dtype, void* stream) {
  const fa_status st = check_decode(B, Lq, Lk, H, Hkv, D, 0, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(workspace) || !ptr_ok(O) || !ptr_ok(LSE)) return FA_ERR_INVALID_ARG;
  return fa::run_decode_merge(workspace, workspace_bytes, O, LSE, B, Lq, Lk, H, Hkv, D, dtype,
                              static_cast<cudaStream_t>(stream));
}

namespace {
// The pools and tables shared by every paged call.
fa_status check_pool(int B, int Hkv, int D, int page, int max_pages, int num_pages,
                     long long k_page_stride, long long v_page_stride, int dtype) {
  if (B < 1 || Hkv < 1 || page < 1 || max_pages < 1 || num_pages < 1) return FA_ERR_INVALID_ARG;
  if (B > (1 << 20) || Hkv > (1 << 20)) return FA_ERR_INVALID_ARG;
  if (dtype != FA_F16 && dtype != FA_BF16) return FA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (page != 16 && page != 32 && page != 64 && page != 128 && page != 256) return FA_ERR_UNSUPPORTED;
  if (static_cast<long long>(max_pages) * page > (1ll << 30)) return FA_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(page) * Hkv * D;
  for (long long st : {k_page_stride, v_page_stride})
    if (st < rows || st % 8 != 0 || st >= (1ll << 38)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// Weights of `cap` slots a row that a write of L tokens resets, or to new ones.
bool weights_ok(const float* weights, long long stride, const float* new_weights, int B, int L, int Hkv,
                long long cap) {
  if (weights == nullptr) return new_weights == nullptr;
  if (!aligned16(weights) || !aligned16(new_weights) || stride < cap || stride >= (1ll << 40)) return false;
  // A token's new weight may be another's slot: no order between the two.
  return new_weights == nullptr || !overlap(weights, weights_bytes(static_cast<long long>(B) * Hkv, stride, cap),
                                            new_weights, sizeof(float) * B * Hkv * static_cast<size_t>(L));
}
}  // namespace

size_t fa_paged_decode_workspace_size(int B, int Lq, int H, int Hkv, int D, int page, int max_pages,
                                      int weights) {
  if (B < 1 || Lq < 1 || H < 1 || Hkv < 1 || H % Hkv != 0 || (D != 64 && D != 128) || page < 1 ||
      max_pages < 1 || static_cast<long long>(H / Hkv) * Lq > 128)
    return 0;
  return fa::paged_decode_workspace_size(B, Lq, static_cast<long long>(max_pages) * page, H, Hkv, D,
                                         weights != 0);
}

fa_status fa_paged_decode(const void* Q, const void* K, const void* V, long long k_page_stride,
                          long long v_page_stride, const int* block_table, const int* lens, void* O,
                          float* LSE, float* weights, long long weights_stride, void* workspace,
                          size_t workspace_bytes, int B, int Lq, int H, int Hkv, int D, int page,
                          int max_pages, int num_pages, int window, int sinks, int dtype,
                          void* stream) {
  fa_status st = check_shape(B, Lq, Lq, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  st = check_pool(B, Hkv, D, page, max_pages, num_pages, k_page_stride, v_page_stride, dtype);
  if (st != FA_OK) return st;
  if (window < 0 || sinks < 0) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(H / Hkv) * Lq > 128) return FA_ERR_UNSUPPORTED;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ints_ok(block_table) || !ints_ok(lens) ||
      !ptr_ok(O) || !ptr_ok(LSE) || !ptr_ok(workspace))
    return FA_ERR_INVALID_ARG;
  if (weights != nullptr &&
      (!aligned16(weights) || weights_stride < static_cast<long long>(max_pages) * page))
    return FA_ERR_INVALID_ARG;
  fa::PagedDecodeArgs a;
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.table = block_table;
  a.lens = lens;
  a.O = O;
  a.LSE = LSE;
  a.weights = weights;
  a.weights_stride = weights_stride;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.B = B;
  a.Lq = Lq;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.max_pages = max_pages;
  a.num_pages = num_pages;
  a.window = window;
  a.sinks = sinks;
  a.dtype = dtype;
  return fa::run_paged_decode(a, static_cast<cudaStream_t>(stream));
}

fa_status fa_paged_write(const void* K, const void* V, void* K_pool, void* V_pool,
                         long long k_page_stride, long long v_page_stride, const int* block_table,
                         const int* start, const int* counts, float* weights,
                         long long weights_stride, const float* new_weights, int B, int L, int Hkv,
                         int D, int page, int max_pages, int num_pages, int dtype, void* stream) {
  fa_status st = check_shape(B, L, L, Hkv, Hkv, D, dtype);
  if (st != FA_OK) return st;
  st = check_pool(B, Hkv, D, page, max_pages, num_pages, k_page_stride, v_page_stride, dtype);
  if (st != FA_OK) return st;
  if (!ptr_ok(K) || !ptr_ok(V) || !ptr_ok(K_pool) || !ptr_ok(V_pool) || !ints_ok(block_table) ||
      !ints_ok(start))
    return FA_ERR_INVALID_ARG;
  if (counts != nullptr && !ints_ok(counts)) return FA_ERR_INVALID_ARG;
  if (!weights_ok(weights, weights_stride, new_weights, B, L, Hkv, static_cast<long long>(max_pages) * page))
    return FA_ERR_INVALID_ARG;
  return fa::run_paged_write(K, V, K_pool, V_pool, k_page_stride, v_page_stride, block_table, start,
                             counts, weights, weights_stride, new_weights, B, L, Hkv, D, page,
                             max_pages, num_pages, static_cast<cudaStream_t>(stream));
}

fa_status fa_paged_evict(void* K_pool, void* V_pool, long long k_page_stride,
                         long long v_page_stride, const int* block_table, const int* lens,
                         const float* weights, long long weights_stride, const int* dst_table,
                         int keep, int sinks, int recent, int* kept, int* new_lens,
                         float* new_weights, int B, int Hkv, int D, int page, int max_pages,
                         int dst_pages, int num_pages, int dtype, void* stream) {
  fa_status st = check_pool(B, Hkv, D, page, max_pages, num_pages, k_page_stride, v_page_stride, dtype);
  if (st != FA_OK) return st;
  if (keep < 1 || sinks < 0 || recent < 0 || static_cast<long long>(sinks) + recent > keep)
    return FA_ERR_INVALID_ARG;
  if (dst_pages < 1 || static_cast<long long>(dst_pages) * page > (1ll << 30) ||
      static_cast<long long>(dst_pages) * page < keep)
    return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (!ptr_ok(K_pool) || !ptr_ok(V_pool) || !ints_ok(block_table) || !ints_ok(lens) ||
      !ints_ok(dst_table) || !ints_ok(kept) || !ints_ok(new_lens) || !ptr_ok(weights) ||
      !ptr_ok(new_weights) || dst_table == block_table)
    return FA_ERR_INVALID_ARG;
  const long long cap = static_cast<long long>(max_pages) * page, pairs = static_cast<long long>(B) * Hkv;
  if (weights_stride < cap || weights_stride >= (1ll << 40)) return FA_ERR_INVALID_ARG;
  {
    // No output may share memory with an input or another output, but new_lens
    // may be lens.
    const struct {
      const void* p;
      size_t n;
    } in[4] = {{block_table, sizeof(int) * B * static_cast<size_t>(max_pages)},
               {dst_table, sizeof(int) * B * static_cast<size_t>(dst_pages)},
               {weights, weights_bytes(pairs, weights_stride, cap)},
               {lens, sizeof(int) * B}},
      out[3] = {{kept, sizeof(int) * pairs * keep},
                {new_weights, sizeof(float) * pairs * dst_pages * page},
                {new_lens, sizeof(int) * B}};
    for (int o = 0; o < 3; ++o) {
      for (int i = 0; i < 4; ++i)
        if (!(o == 2 && new_lens == lens && i == 3) && overlap(out[o].p, out[o].n, in[i].p, in[i].n))
          return FA_ERR_INVALID_ARG;
      for (int i = 0; i < o; ++i)
        if (overlap(out[o].p, out[o].n, out[i].p, out[i].n)) return FA_ERR_INVALID_ARG;
    }
  }
  fa::PagedEvictArgs a;
  a.K = K_pool;
  a.V = V_pool;
  a.table = block_table;
  a.lens = lens;
  a.dst_table = dst_table;
  a.weights = weights;
  a.kept = kept;
  a.new_lens = new_lens;
  a.new_weights = new_weights;
  a.weights_stride = weights_stride;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.B = B;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.max_pages = max_pages;
  a.dst_pages = dst_pages;
  a.num_pages = num_pages;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  return fa::run_paged_evict(a, static_cast<cudaStream_t>(stream));
}

namespace {

// One operand of the rotary calls: [B, L, heads, D] with free batch and token
// strides; an output's rows must lie apart.
bool view_ok(const fa::RopeView& v, bool output, int B, int L, int heads, int D) {
  const long long row = static_cast<long long>(heads) * D;
  if (!ptr_ok(v.p) || v.batch < 0 || v.token < 0 || v.batch % 8 != 0 || v.token % 8 != 0 ||
      v.batch >= (1ll << 38) || v.token >= (1ll << 38))
    return false;
  if (!output) return true;
  if (B == 1) return L == 1 || v.token >= row;
  if (L == 1) return v.batch >= row;
  return (v.token >= row && v.batch >= (L - 1) * v.token + row) || (v.batch >= row && v.token >= (B - 1) * v.batch + row);
}

// The output is the input itself or shares no memory with it.
bool in_place_or_apart(const fa::RopeView& x, const fa::RopeView& y, int B, int L, int heads, int D) {
  auto bytes = [&](const fa::RopeView& v) {
    return static_cast<size_t>((B - 1) * v.batch + (L - 1) * v.token + static_cast<long long>(heads) * D) * 2;
  };
  if (x.p == y.p && (B == 1 || x.batch == y.batch) && (L == 1 || x.token == y.token)) return true;
  return !overlap(x.p, bytes(x), y.p, bytes(y));
}

fa_status check_rope(const fa::RopeArgs& a, int heads) {
  if (a.Hkv < 0 || a.Hkv > (1 << 20) || a.H < 1 || a.H > (1 << 20)) return FA_ERR_INVALID_ARG;
  const fa_status st = check_shape(a.B, a.L, a.L, heads, heads, a.D, a.dtype);
  if (st != FA_OK) return st;
  if (a.rotary < 16 || a.rotary > a.D || a.rotary % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (a.axes < 1 || a.axes > 256 || !ptr_ok(a.table)) return FA_ERR_INVALID_ARG;
  if (a.positions == nullptr ? a.axes != 1 : !ints_ok(a.positions)) return FA_ERR_INVALID_ARG;
  if (!view_ok(a.q, false, a.B, a.L, a.H, a.D) || !view_ok(a.qy, true, a.B, a.L, a.H, a.D) ||
      !in_place_or_apart(a.q, a.qy, a.B, a.L, a.H, a.D))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

}  // namespace

fa_status fa_rope(const void* Q, long long q_batch, long long q_token, const void* K, long long k_batch,
                  long long k_token, void* Q_out, long long q_out_batch, long long q_out_token, void* K_out,
                  long long k_out_batch, long long k_out_token, const long long* table, const int* positions,
                  int axes, int B, int L, int H, int Hkv, int D, int rotary, int interleaved, int backward,
                  int dtype, void* stream) {
  const fa::RopeArgs a{{Q, q_batch, q_token}, {K, k_batch, k_token}, {Q_out, q_out_batch, q_out_token},
                       {K_out, k_out_batch, k_out_token}, table, positions, axes, B, L, H, Hkv, D, rotary,
                       interleaved, backward, dtype};
  const fa_status st = check_rope(a, Hkv > 0 && H > 0 && Hkv <= (1 << 20) && H <= (1 << 20) ? H + Hkv : H);
  if (st != FA_OK) return st;
  if (Hkv == 0) {
    if (K != nullptr || K_out != nullptr) return FA_ERR_INVALID_ARG;
  } else if (!view_ok(a.k, false, B, L, Hkv, D) || !view_ok(a.ky, true, B, L, Hkv, D) ||
             !in_place_or_apart(a.k, a.ky, B, L, Hkv, D)) {
    return FA_ERR_INVALID_ARG;
  }
  return fa::run_rope(a, static_cast<cudaStream_t>(stream));
}

fa_status fa_paged_append(const void* Q, long long q_batch, long long q_token, const void* K, long long k_batch,
                          long long k_token, const void* V, long long v_batch, long long v_token, void* Q_out,
                          long long q_out_batch, long long q_out_token, void* K_pool, void* V_pool,
                          long long k_page_stride, long long v_page_stride, const int* block_table,
                          const int* start, const int* counts, const long long* table, const int* positions,
                          int axes, float* weights, long long weights_stride, const float* new_weights, int B,
                          int L, int H, int Hkv, int D, int rotary, int interleaved, int page, int max_pages,
                          int num_pages, int dtype, void* stream) {
  const fa::RopeArgs a{{Q, q_batch, q_token}, {K, k_batch, k_token}, {Q_out, q_out_batch, q_out_token},
                       {}, table, positions, axes, B, L, H, Hkv, D, rotary, interleaved, 0, dtype};
  if (Hkv < 1 || Hkv > (1 << 20) || H < 1 || H > (1 << 20)) return FA_ERR_INVALID_ARG;
  fa_status st = check_rope(a, H + 2 * Hkv);
  if (st != FA_OK) return st;
  if (H % Hkv != 0) return FA_ERR_INVALID_ARG;
  st = check_pool(B, Hkv, D, page, max_pages, num_pages, k_page_stride, v_page_stride, dtype);
  if (st != FA_OK) return st;
  const fa::RopeView v{V, v_batch, v_token};
  if (!view_ok(a.k, false, B, L, Hkv, D) || !view_ok(v, false, B, L, Hkv, D) || !ptr_ok(K_pool) || !ptr_ok(V_pool) ||
      !ints_ok(block_table) || !ints_ok(start) || (counts != nullptr && !ints_ok(counts)))
    return FA_ERR_INVALID_ARG;
  if (!weights_ok(weights, weights_stride, new_weights, B, L, Hkv, static_cast<long long>(max_pages) * page))
    return FA_ERR_INVALID_ARG;
  const fa::PagedAppendArgs c{v, K_pool, V_pool, block_table, start, counts, weights, new_weights, weights_stride,
                              k_page_stride, v_page_stride, page, max_pages, num_pages};
  return fa::run_paged_append(a, c, static_cast<cudaStream_t>(stream));
}

namespace {
fa::PrefixDecodeArgs prefix_sizes(int B, int Lq, int H, int Hkv, int D, int page, int groups, int prefix_pages,
                                  int max_pages) {
  fa::PrefixDecodeArgs a = {};
  a.B = B;
  a.Lq = Lq;
  a.H = H;
  a.Hkv = Hkv;
  a.D = D;
  a.page = page;
  a.groups = groups;
  a.prefix_pages = prefix_pages;
  a.max_pages = max_pages;
  return a;
}

// What both prefix calls refuse.
fa_status check_prefix(int B, int Lq, int H, int Hkv, int D, int page, int groups, int prefix_pages, int max_pages,
                       int dtype) {
  fa_status st = check_shape(B, Lq, Lq, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  const long long least = static_cast<long long>(page < 1 ? 1 : page) * Hkv * D;
  for (int pages : {prefix_pages, max_pages}) {
    st = check_pool(B, Hkv, D, page, pages, 1, least, least, dtype);
    if (st != FA_OK) return st;
  }
  if (groups < 1 || groups > (1 << 20)) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(H / Hkv) * Lq > 128) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}
}  // namespace

size_t fa_paged_prefix_decode_workspace_size(int B, int Lq, int H, int Hkv, int D, int page, int groups,
                                             int prefix_pages, int max_pages) {
  if (check_prefix(B, Lq, H, Hkv, D, page, groups, prefix_pages, max_pages, FA_F16) != FA_OK) return 0;
  return fa::paged_prefix_workspace_size(prefix_sizes(B, Lq, H, Hkv, D, page, groups, prefix_pages, max_pages));
}

fa_status fa_paged_prefix_decode(const void* Q, const void* K, const void* V, long long k_page_stride,
                                 long long v_page_stride, const int* prefix_table, const int* prefix_lens,
                                 const int* group_starts, const int* block_table, const int* lens, void* O,
                                 float* LSE, void* workspace, size_t workspace_bytes, int B, int Lq, int H, int Hkv,
                                 int D, int page, int groups, int prefix_pages, int max_pages, int num_pages,
                                 int dtype, void* stream) {
  fa_status st = check_prefix(B, Lq, H, Hkv, D, page, groups, prefix_pages, max_pages, dtype);
  if (st != FA_OK) return st;
  st = check_pool(B, Hkv, D, page, max_pages, num_pages, k_page_stride, v_page_stride, dtype);
  if (st != FA_OK) return st;
  if (group_starts == nullptr ? groups != 1 : !ints_ok(group_starts)) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(V) || !ints_ok(prefix_table) || !ints_ok(prefix_lens) ||
      !ints_ok(block_table) || !ints_ok(lens) || !ptr_ok(O) || !ptr_ok(LSE) || !ptr_ok(workspace))
    return FA_ERR_INVALID_ARG;
  fa::PrefixDecodeArgs a = prefix_sizes(B, Lq, H, Hkv, D, page, groups, prefix_pages, max_pages);
  a.Q = Q;
  a.K = K;
  a.V = V;
  a.prefix_table = prefix_table;
  a.prefix_lens = prefix_lens;
  a.group_starts = group_starts;
  a.table = block_table;
  a.lens = lens;
  a.O = O;
  a.LSE = LSE;
  a.k_page_stride = k_page_stride;
  a.v_page_stride = v_page_stride;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  a.num_pages = num_pages;
  a.dtype = dtype;
  return fa::run_paged_prefix(a, static_cast<cudaStream_t>(stream));
}

size_t fa_key_weights_workspace_size(void) { return fa::key_weights_workspace_size(); }

fa_status fa_key_weights(const void* Q, const void* K, const float* LSE, float* W, void* workspace,
                         size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv, int D,
                         int causal, int window, int sinks, int dtype, void* stream) {
  fa_status st = check_shape(B, Lq, Lk, H, Hkv, D, dtype);
  if (st != FA_OK) return st;
  if (causal && Lk < Lq) return FA_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || (window > 0 && !causal)) return FA_ERR_INVALID_ARG;
  if (!ptr_ok(Q) || !ptr_ok(K) || !ptr_ok(LSE) || !ptr_ok(W) || !ptr_ok(workspace))
    return FA_ERR_INVALID_ARG;
  return fa::run_key_weights(Q, K, LSE, W, workspace, workspace_bytes, B, Lq, Lk, H, Hkv, D, causal,
                             window, sinks, dtype, static_cast<cudaStream_t>(stream));
}

fa_status fa_check_device_error(void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned int words[6] = {fa::fwd_read_error(s), fa::bwd_read_error(s),
                                 fa::decode_read_error(s), fa::paged_read_error(s),
                                 fa::weights_read_error(s), fa::prefix_read_error(s)};
  unsigned int site = 0;
  for (unsigned int w : words) {
    if (w == 0xFFFFFFFFu) return FA_ERR_CUDA;
    if (w && !site) site = w;
  }
  if (site) {
    g_last_site = site;
    return FA_ERR_DEVICE_TIMEOUT;
  }
  return FA_OK;
}

fa_status fa_selftest_bounded_wait(unsigned long long limit_ns, void* stream) {
  if (limit_ns < 1000000ull) limit_ns = 1000000ull;
  if (limit_ns > 1000000000ull) limit_ns = 1000000000ull;
  return fa::run_selftest_wait(limit_ns, static_cast<cudaStream_t>(stream));
}

unsigned int fa_last_error_site(void) { return g_last_site; }

const char* fa_status_string(fa_status s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported head dimension or dtype";
    case FA_ERR_CUDA: return "CUDA runtime or launch error";
    case FA_ERR_DEVICE_TIMEOUT: return "a kernel gave up a bounded wait";
    case FA_ERR_SCRATCH_TOO_SMALL:
      return "scratch too small: the problem needs more than fa_bwd_noalloc's fixed array or "
             "the workspace given";
  }
  return "unknown status";
}

const char* fa_version(void) { return "tiled_attention_fa_gb300 0.1 (sm_103a)"; }

}  // extern "C"
