// Host launchers of the backward kernels (preprocess, main pass, dQ post-process).
#include <cmath>
#include <mutex>
#include <type_traits>

#include "bwd.cuh"
#include "common.cuh"
#include "internal.h"

namespace fa {

template <int D, bool BF16>
static fa_status launch_prep(const void* O, const void* dO, float* Delta, float* dq_accum, int B,
                             int L, int H, cudaStream_t s) {
  const int Lpad = padded_len(L);
  // Heads per CTA: all of them when (batch, chunk) pairs alone fill the GPU
  // twice over, else fewer (halving) until they do.
  const long long pairs = static_cast<long long>(B) * (Lpad / 32);
  int hg = H;
  while (hg > 1 && pairs * ((H + hg - 1) / hg) < 2LL * sm_count()) hg = (hg + 1) / 2;
  const long long grid = pairs * ((H + hg - 1) / hg);
  if (grid > 0x7FFFFFFFLL) return FA_ERR_UNSUPPORTED;
  const size_t smem = static_cast<size_t>(hg) * 32 * sizeof(float);
  auto kern = fa_bwd_prep_kernel<D, BF16>;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return FA_ERR_UNSUPPORTED;
  kern<<<static_cast<unsigned>(grid), 256, smem, s>>>(O, dO, Delta, dq_accum, B, L, H, Lpad, hg);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status run_bwd_prep(const void* O, const void* dO, float* Delta, float* dq_accum, int B, int L,
                       int H, int D, int dtype, cudaStream_t s) {
  const bool bf16 = dtype == FA_BF16;
  if (static_cast<size_t>(H) * 32 * sizeof(float) > 200 * 1024) return FA_ERR_UNSUPPORTED;
  if (D == 64)
    return bf16 ? launch_prep<64, true>(O, dO, Delta, dq_accum, B, L, H, s)
                : launch_prep<64, false>(O, dO, Delta, dq_accum, B, L, H, s);
  return bf16 ? launch_prep<128, true>(O, dO, Delta, dq_accum, B, L, H, s)
              : launch_prep<128, false>(O, dO, Delta, dq_accum, B, L, H, s);
}

// L2 size of the current device (cached per device).
static double l2_bytes() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  static int cache[64] = {0};
  if (dev >= 0 && dev < 64 && cache[dev]) return cache[dev];
  cudaDeviceGetAttribute(&n, cudaDevAttrL2CacheSize, dev);
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

namespace {

// The window's units (see BwdParams); p holds Lq, Lk, past, n_kv, n_q, Hkv.
void plan_window(BwdParams& p, int B, int window, int sinks) {
  p.window = window < p.Lk ? window : p.Lk;  // as good as every key when larger
  p.sinks = sinks < p.Lk ? sinks : p.Lk;
  if (static_cast<long long>(p.window) + p.sinks >= p.Lk) {  // hides no key: no sink tiles apart
    p.window = p.Lk;
    p.sinks = 0;
  }
  p.n_sink = (p.sinks + 127) / 128;
  p.srows = p.sinks < 128 ? p.sinks : 128;
  p.chunk = (p.window + 254) / 128;  // Q tiles a window tile is seen by: equal units
  int most = 0;
  for (int j = 0; j < p.n_sink; ++j) {
    int lo, reach;
    bwd_win_range(p, j, lo, reach);
    const int left = p.n_q - reach;
    most = left > most ? left : most;
  }
  // Far units beyond 8 per SM only cost parts (a slot of 2 * srows * D floats each
  // in the workspace, which would grow with sinks * Lq / window), so theirs are
  // then longer: at most 8 per SM, or one per sink tile where those are more.
  if (most > 0) {
    const long long tiles = static_cast<long long>(B) * p.Hkv * p.n_sink, per = 8ll * sm_count() / tiles;
    const int least = per > 1 ? static_cast<int>((most + per - 1) / per) : most;
    if (p.chunk < least) p.chunk = least;
  }
  p.n_rest = (most + p.chunk - 1) / p.chunk;
  p.n_items = B * p.Hkv * (p.n_kv + p.n_sink * p.n_rest);
  // Few units of many heads leave SMs idle: cut them by query heads.  Costs in
  // steps of a 128 x 128 tile: a unit's start and end take about 3, its fp32
  // parts 1 more and their sum a launch and a share of the traffic.  Whole and
  // cut, with the dQ post-process: B1 H32/4 L735 D128 window 723 126 and 48 us,
  // B2 H16/2 L1000 D64 window 300 81 and 32, B1 H8/1 L4000 D128 window 1000 179
  // and 63.
  p.hs = 1;
  const int g = p.H / p.Hkv, sms = sm_count();
  const double steps = static_cast<double>(g) * (p.chunk < p.n_q ? p.chunk : p.n_q);
  const double units = static_cast<double>(p.n_items);
  double best = std::ceil(units / (sms < 1 ? 1 : sms)) * (steps + 3);
  for (int hs = 2; hs <= g && sms > 0 && units * hs <= 8.0 * sms; ++hs) {
    if (g % hs != 0) continue;
    const double cost = std::ceil(units * hs / sms) * (steps / hs + 4) + 2 + units * hs / 100;
    if (cost < 0.85 * best) {
      best = cost;
      p.hs = hs;
    }
  }
  if (p.hs > 1) {
    p.n_items *= p.hs;
    p.srows = 128;
  }
}

// fp32 parts of dK and dV, of 2 * srows * D elements each.
size_t window_slots(const BwdParams& p) {
  const size_t bh = static_cast<size_t>(p.B) * p.Hkv;
  if (p.hs > 1) return bh * (p.n_kv + static_cast<size_t>(p.n_sink) * p.n_rest) * p.hs;
  return p.n_rest ? bh * p.n_sink * (1 + p.n_rest) : 0;
}

size_t dq_bytes(int B, int L, int H, int D) {
  return (static_cast<size_t>(B) * H * padded_len(L) * D * sizeof(float) + 255) / 256 * 256;
}

BwdParams window_plan(int B, int Lq, int Lk, int H, int Hkv, int window, int sinks) {
  BwdParams p = {};
  p.B = B;
  p.H = H;
  p.Lq = Lq;
  p.Lk = Lk;
  p.past = Lk - Lq;
  p.Hkv = Hkv;
  p.n_kv = (Lk + 127) / 128;
  p.n_q = (Lq + 127) / 128;
  plan_window(p, B, window, sinks);
  return p;
}

}  // namespace

size_t window_bwd_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D, int window, int sinks) {
  const BwdParams p = window_plan(B, Lq, Lk, H, Hkv, window, sinks);
  return dq_bytes(B, Lq, H, D) + window_slots(p) * 2 * p.srows * D * sizeof(float);
}

// window > 0 (WIN, causal calls only): the backward of run_window_fwd.
template <int D, bool BF16, bool WIN = false>
static fa_status launch_bwd(const void* Q, const void* K, const void* V, const void* dO,
                            const float* LSE, const float* Delta, void* dK, void* dV,
                            float* dq_accum, int zero_accum, int B, int Lq, int Lk, int H,
                            int Hkv, int causal, cudaStream_t s, int window = 0, int sinks = 0,
                            float* sink_part = nullptr) {
  using Ly = BwdLayout<D>;
  const int Lpad = padded_len(Lq);
  if (zero_accum &&
      cudaMemsetAsync(dq_accum, 0, static_cast<size_t>(B) * H * Lpad * D * sizeof(float), s) !=
          cudaSuccess)
    return FA_ERR_CUDA;
  CUtensorMap tq, tk, tv, tdo;
  if (!make_bshd_map(&tq, Q, B, Lq, H, D, BF16) || !make_bshd_map(&tk, K, B, Lk, Hkv, D, BF16) ||
      !make_bshd_map(&tv, V, B, Lk, Hkv, D, BF16) || !make_bshd_map(&tdo, dO, B, Lq, H, D, BF16))
    return FA_ERR_CUDA;
  BwdParams p;
  p.LSE = LSE;
  p.Delta = Delta;
  p.dq_accum = dq_accum;
  p.dK = dK;
  p.dV = dV;
  p.B = B;
  p.Lq = Lq;
  p.Lk = Lk;
  p.past = Lk - Lq;
  p.H = H;
  p.Hkv = Hkv;
  p.causal = causal ? 1 : 0;
  p.n_kv = (Lk + 127) / 128;
  p.n_q = Lpad / 128;
  p.Lpad = Lpad;
  p.n_items = B * Hkv * p.n_kv;
  p.ipu = p.causal ? 2 : 1;
  p.n_units = p.causal ? B * Hkv * ((p.n_kv + 1) / 2) : p.n_items;
  p.snake = 0;
  {
    // Causal problems of at most four rounds of pair units leave much of the
    // last round idle, so deal single tiles in snake order instead -- when
    // every head's Q and dO fit in 0.6 of L2 together (the snake order runs
    // all heads at once; the pair order a few heads at a time).  Measured,
    // fp16 causal: B1 H32 D128 L1024 0.0446 -> 0.0436 ms, L4096 (64 MiB of
    // Q, dO; 512 pair units) 0.371 -> 0.335 ms; L8192 (128 MiB) 1.184 ->
    // 1.257 ms and B8 H32 L1024 D64 (1,024 pair units) 0.162 -> 0.184 ms
    // with it, hence the limits.
    const int sm = sm_count();
    const double qdo_bytes = 4.0 * B * H * static_cast<double>(Lq) * D;  // Q and dO, 16-bit
    if (!WIN && p.causal && p.n_items >= sm && p.n_units <= 4 * sm && qdo_bytes <= 0.6 * l2_bytes()) {
      p.snake = 1;
      p.ipu = 1;
      p.n_units = (p.n_items + sm - 1) / sm * sm;
    }
  }
  if (WIN) {
    plan_window(p, B, window, sinks);
    p.ipu = 1;
    p.n_units = p.n_items;
    p.sink_part = sink_part;
  }
  p.scale = 1.f / sqrtf(static_cast<float>(D));
  p.sl2 = 1.4426950408889634f * p.scale;
  int dev = 0, optin = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&optin, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
  if (optin < static_cast<int>(Ly::SMEM_ALLOC)) return FA_ERR_UNSUPPORTED;
  auto kern = fa_bwd_kernel<D, BF16, WIN>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Ly::SMEM_ALLOC) !=
      cudaSuccess)
    return FA_ERR_CUDA;
  {
    // The kernel re-balances registers between its warpgroups (setmaxnreg:
    // Ly::REGS_COMPUTE twice, REGS_DRAIN, REGS_OTHER per thread); the budgets
    // add up only when every thread starts with NTHREADS_REGS.  Any other
    // allocation would leave an increase waiting for registers that never
    // come back, so refuse to launch instead.
    static int num_regs = -1;
    static std::once_flag once;
    std::call_once(once, [&] {
      cudaFuncAttributes a;
      if (cudaFuncGetAttributes(&a, kern) == cudaSuccess) num_regs = a.numRegs;
    });
    if (num_regs != Ly::NTHREADS_REGS) return FA_ERR_UNSUPPORTED;
  }
  const int grid = p.n_units < sm_count() ? p.n_units : sm_count();  // persistent CTAs
  kern<<<grid, Ly::NTHREADS, Ly::SMEM_ALLOC, s>>>(tq, tk, tv, tdo, p);
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

template <int D, bool BF16>
static fa_status launch_post(const float* dq_accum, void* dQ, int B, int L, int H, cudaStream_t s) {
  const int Lpad = padded_len(L);
  auto kern = fa_dq_convert_kernel<D, BF16>;
  constexpr size_t smem = conv_smem_bytes<D>();
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
          cudaSuccess)
    return FA_ERR_CUDA;
  kern<<<B * H * (Lpad / kConvRows), kConvThreads, smem, s>>>(
      dq_accum, dQ, B, L, H, Lpad, 1.f / sqrtf(static_cast<float>(D)));
  return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status run_bwd_main(const void* Q, const void* K, const void* V, const void* dO,
                       const float* LSE, const float* Delta, void* dK, void* dV, float* dq_accum,
                       int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                       int dtype, cudaStream_t s) {
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    return bf16 ? launch_bwd<64, true>(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B,
                                       Lq, Lk, H, Hkv, causal, s)
                : launch_bwd<64, false>(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B,
                                        Lq, Lk, H, Hkv, causal, s);
  return bf16 ? launch_bwd<128, true>(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B,
                                      Lq, Lk, H, Hkv, causal, s)
              : launch_bwd<128, false>(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B,
                                       Lq, Lk, H, Hkv, causal, s);
}

template <int D, bool BF16>
static fa_status launch_window_bwd(const void* Q, const void* K, const void* V, const void* dO,
                                   const float* LSE, const float* Delta, void* dQ, void* dK,
                                   void* dV, float* ws, int zero_accum, int B, int Lq, int Lk,
                                   int H, int Hkv, int window, int sinks, cudaStream_t s) {
  BwdParams p = window_plan(B, Lq, Lk, H, Hkv, window, sinks);
  p.dK = dK;
  p.dV = dV;
  p.scale = 1.f / sqrtf(static_cast<float>(D));
  p.sink_part = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + dq_bytes(B, Lq, H, D));
  const fa_status st =
      launch_bwd<D, BF16, true>(Q, K, V, dO, LSE, Delta, dK, dV, ws, zero_accum, B, Lq, Lk, H, Hkv,
                                1, s, window, sinks, p.sink_part);
  if (st != FA_OK) return st;
  if (p.hs > 1) {
    if (!launch_after(fa_head_sum_kernel<D, BF16>, dim3(B * Hkv * p.n_kv, 16), dim3(2 * D), s, p))
      return FA_ERR_CUDA;
  } else if (p.n_rest > 0) {
    if (!launch_after(fa_sink_sum_kernel<D, BF16>, dim3(B * Hkv * p.n_sink, (p.srows + 3) / 4), dim3(2 * D), s, p))
      return FA_ERR_CUDA;
  }
  return launch_post<D, BF16>(ws, dQ, B, Lq, H, s);
}

fa_status run_window_bwd(const void* Q, const void* K, const void* V, const void* dO,
                         const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                         float* ws, size_t ws_bytes, int zero_accum, int B, int Lq, int Lk, int H,
                         int Hkv, int D, int window, int sinks, int dtype, cudaStream_t s) {
  if (ws_bytes < window_bwd_workspace_size(B, Lq, Lk, H, Hkv, D, window, sinks))
    return FA_ERR_SCRATCH_TOO_SMALL;
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    return bf16 ? launch_window_bwd<64, true>(Q, K, V, dO, LSE, Delta, dQ, dK, dV, ws, zero_accum,
                                              B, Lq, Lk, H, Hkv, window, sinks, s)
                : launch_window_bwd<64, false>(Q, K, V, dO, LSE, Delta, dQ, dK, dV, ws, zero_accum,
                                               B, Lq, Lk, H, Hkv, window, sinks, s);
  return bf16 ? launch_window_bwd<128, true>(Q, K, V, dO, LSE, Delta, dQ, dK, dV, ws, zero_accum, B,
                                             Lq, Lk, H, Hkv, window, sinks, s)
              : launch_window_bwd<128, false>(Q, K, V, dO, LSE, Delta, dQ, dK, dV, ws, zero_accum,
                                              B, Lq, Lk, H, Hkv, window, sinks, s);
}

fa_status run_bwd_post(const float* dq_accum, void* dQ, int B, int L, int H, int D, int dtype,
                       cudaStream_t s) {
  const bool bf16 = dtype == FA_BF16;
  if (D == 64)
    return bf16 ? launch_post<64, true>(dq_accum, dQ, B, L, H, s)
                : launch_post<64, false>(dq_accum, dQ, B, L, H, s);
  return bf16 ? launch_post<128, true>(dq_accum, dQ, B, L, H, s)
              : launch_post<128, false>(dq_accum, dQ, B, L, H, s);
}

fa_status run_bwd(const void* Q, const void* K, const void* V, const void* dO, const float* LSE,
                  const float* Delta, void* dQ, void* dK, void* dV, float* dq_accum,
                  int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D, int causal,
                  int dtype, cudaStream_t s) {
  fa_status st = run_bwd_main(Q, K, V, dO, LSE, Delta, dK, dV, dq_accum, zero_accum, B, Lq, Lk, H,
                              Hkv, D, causal, dtype, s);
  if (st != FA_OK) return st;
  return run_bwd_post(dq_accum, dQ, B, Lq, H, D, dtype, s);
}

unsigned int bwd_read_error(cudaStream_t s) { return read_and_clear_error(s); }

// ---------------------------------------------------------------- no-allocation variant
// Scratch for fa_bwd_noalloc's fp32 dQ accumulator.  It is part of this
// module's device image, so every GPU that loads the library holds these
// FA_NOALLOC_SCRATCH_BYTES until the process exits; all calls share it.
static __device__ __align__(256) float g_noalloc_dq_accum[FA_NOALLOC_SCRATCH_BYTES / sizeof(float)];

namespace {
constexpr int kMaxDevices = 64;
std::mutex g_noalloc_mu;
float* g_noalloc_ptr[kMaxDevices] = {};

// Device address of the scratch array on the current device.  In host code
// the array's name is only a host-side stand-in, so the address is looked up
// with the device current.  It is looked up again on every call whose stream
// is not being captured (a device reset reloads the module, possibly at
// another address) and remembered per device for calls made during a
// capture, where the lookup is not attempted.
fa_status noalloc_scratch(cudaStream_t s, float** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return FA_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return FA_ERR_UNSUPPORTED;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  if (cudaStreamIsCapturing(s, &cs) != cudaSuccess) return FA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  if (cs == cudaStreamCaptureStatusNone) {
    void* ptr = nullptr;
    if (cudaGetSymbolAddress(&ptr, g_noalloc_dq_accum) != cudaSuccess || ptr == nullptr)
      return FA_ERR_CUDA;
    g_noalloc_ptr[dev] = static_cast<float*>(ptr);
  } else if (g_noalloc_ptr[dev] == nullptr) {
    return FA_ERR_CUDA;  // first call on this device made during a capture
  }
  *out = g_noalloc_ptr[dev];
  return FA_OK;
}
}  // namespace

fa_status run_bwd_noalloc(const void* Q, const void* K, const void* V, const void* dO,
                          const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                          int B, int L, int H, int Hkv, int D, int causal, int dtype,
                          cudaStream_t s) {
  const size_t need = static_cast<size_t>(B) * H * padded_len(L) * D * sizeof(float);
  if (need > FA_NOALLOC_SCRATCH_BYTES) return FA_ERR_SCRATCH_TOO_SMALL;
  float* acc = nullptr;
  fa_status st = noalloc_scratch(s, &acc);
  if (st != FA_OK) return st;
  // The array keeps the previous call's sums: clear the part this call uses.
  if (cudaMemsetAsync(acc, 0, need, s) != cudaSuccess) return FA_ERR_CUDA;
  return run_bwd(Q, K, V, dO, LSE, Delta, dQ, dK, dV, acc, 0, B, L, L, H, Hkv, D, causal, dtype,
                 s);
}

}  // namespace fa
