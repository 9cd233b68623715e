// Host side of the key weights: the workspace and the two launches.
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "weights.cuh"

namespace fa {

namespace {

size_t meta_bytes(int sms) { return (sizeof(KwMeta) * sms + 255) / 256 * 256; }

template <int D, bool BF16>
fa_status launch(const void* Q, const void* K, const KwParams& p, int G, cudaStream_t s) {
  using Ly = KwLayout<D>;
  CUtensorMap tq, tk;
  if (!make_bshd_map(&tq, Q, p.B, p.Lq, p.H, D, BF16) || !make_bshd_map(&tk, K, p.B, p.Lk, p.Hkv, D, BF16))
    return FA_ERR_CUDA;
  auto kern = fa_key_weights_kernel<D, BF16>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM_ALLOC) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  kern<<<G, Ly::NTHREADS, Ly::SMEM_ALLOC, s>>>(tq, tk, p);
  if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
  return launch_after(fa_key_weights_join_kernel, dim3(G), dim3(128), s, p, G) ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

size_t key_weights_workspace_size() {
  const int sms = sm_count() < 1 ? 1 : sm_count();
  return meta_bytes(sms) + 2 * static_cast<size_t>(sms) * 128 * sizeof(float);
}

fa_status run_key_weights(const void* Q, const void* K, const float* LSE, float* W, void* ws,
                          size_t ws_bytes, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                          int window, int sinks, int dtype, cudaStream_t s) {
  if (ws_bytes < key_weights_workspace_size()) return FA_ERR_SCRATCH_TOO_SMALL;
  const int sms = sm_count();
  const long long most = static_cast<long long>(B) * H * ((Lk + 127) / 128) * ((Lq + 127) / 128);
  // A CTA counts its part's steps in an int (2^31 steps of half a microsecond).
  if (most / (sms < 1 ? 1 : sms) >= (1ll << 31) - 1) return FA_ERR_UNSUPPORTED;
  KwParams p;
  p.LSE = LSE;
  p.W = W;
  p.meta = static_cast<KwMeta*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) + meta_bytes(sms));
  p.B = B;
  p.Lq = Lq;
  p.Lk = Lk;
  p.H = H;
  p.Hkv = Hkv;
  p.g = H / Hkv;
  p.causal = causal ? 1 : 0;
  p.past = Lk - Lq;
  p.n_kv = (Lk + 127) / 128;
  p.n_q = (Lq + 127) / 128;
  p.window = window < Lk ? window : 0;  // wider than the sequence: every key
  p.sinks = p.window ? (sinks < Lk ? sinks : Lk) : 0;
  p.sl2 = 1.4426950408889634f / sqrtf(static_cast<float>(D));
  const int G = most < sms ? static_cast<int>(most) : sms;
  const bool bf16 = dtype == FA_BF16;
  if (D == 64) return bf16 ? launch<64, true>(Q, K, p, G, s) : launch<64, false>(Q, K, p, G, s);
  return bf16 ? launch<128, true>(Q, K, p, G, s) : launch<128, false>(Q, K, p, G, s);
}

unsigned int weights_read_error(cudaStream_t s) { return read_and_clear_error(s); }

}  // namespace fa
