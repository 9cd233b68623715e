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
  if (weights == nullptr && new_weights != nullptr) return FA_ERR_INVALID_ARG;
  if (weights != nullptr &&
      (!aligned16(weights) || !aligned16(new_weights) ||
       weights_stride < static_cast<long long>(max_pages) * page || weights_stride >= (1ll << 40)))
    return FA_ERR_INVALID_ARG;
  // A token's new weight may be another's slot: no order between the two.
  if (new_weights != nullptr &&
      overlap(weights,
              weights_bytes(static_cast<long long>(B) * Hkv, weights_stride,
                            static_cast<long long>(max_pages) * page),
              new_weights, sizeof(float) * B * Hkv * static_cast<size_t>(L)))
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
  const unsigned int words[5] = {fa::fwd_read_error(s), fa::bwd_read_error(s),
                                 fa::decode_read_error(s), fa::paged_read_error(s),
                                 fa::weights_read_error(s)};
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
