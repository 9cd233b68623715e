/*
 * C ABI of the GB300 (sm_103a) tiled online-softmax attention library.
 *
 * Tensors are plain device pointers; sizes are ints; nothing here depends on
 * a framework.  Every call is asynchronous on the given CUDA stream (passed as
 * `void*`, i.e. a cudaStream_t; NULL = the legacy default stream).  Argument
 * errors are reported synchronously by the return value and launch nothing.
 * The caller allocates and owns every buffer, including the backward
 * workspace; the library keeps a per-device SM-count cache, a count of
 * fa_paged_decode calls (each call's number marks its counters in its
 * workspace) and fa_bwd_noalloc's fixed array.
 *
 * Layouts (all contiguous, row-major):
 *   Q, O, dO, dQ   [B, L, H,   D]   fp16 or bf16 ("BSHD")
 *   K, V, dK, dV   [B, L, Hkv, D]   same dtype as Q
 *   LSE, Delta     [B, H, L]        fp32
 * Query head h reads K/V head h / (H / Hkv) (grouped-query attention).
 * The softmax scale is fixed at 1 / sqrt(D).  Causal masking is top-left
 * aligned with one length L for queries and keys: key j is visible to query i
 * iff j <= i.  Every pointer must be 16-byte aligned.
 * Supported: D in {64, 128}; L >= 1; B, H, Hkv >= 1 with H % Hkv == 0;
 * B * H * L and B * L * H * D must fit the kernels' 32-bit coordinates
 * (B, L, H < 2^31 and B * L * H * D < 2^40).
 */
#ifndef TILED_ATTENTION_FA_GB300_FA_H
#define TILED_ATTENTION_FA_GB300_FA_H

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FA_OK = 0,
  FA_ERR_INVALID_ARG = 1,    /* null/misaligned pointer, bad size, H % Hkv != 0 */
  FA_ERR_UNSUPPORTED = 2,    /* D or dtype outside the supported set, or the device or the
                                build cannot run the kernel as designed (too little shared
                                memory per block; a backward kernel compiled with a register
                                allocation other than its warpgroup split assumes);
                                nothing was launched */
  FA_ERR_CUDA = 3,           /* a CUDA runtime call or kernel launch failed */
  FA_ERR_DEVICE_TIMEOUT = 4, /* a kernel gave up a bounded wait (see fa_check_device_error) */
  FA_ERR_SCRATCH_TOO_SMALL = 5 /* fa_bwd_noalloc's fixed scratch or a call's workspace is
                                  smaller than the problem needs; nothing was launched */
} fa_status;

typedef enum { FA_F16 = 0, FA_BF16 = 1 } fa_dtype;

/*
 * Forward attention.  For each batch b and query head h:
 *   S = Q_bh K_bh'^T / sqrt(D)   (h' = h / (H / Hkv)), causal: S_ij = -inf for j > i
 *   O_bh = softmax_rows(S) V_bh'                 -> O   [B, L, H, D]
 *   LSE_bh,i = ln sum_j exp(S_ij)                -> LSE [B, H, L], fp32
 * Page "使用 TileLang 在 AMD GPU 上快速开发高性能 Flash Attention", sections
 * 核心公式与计算流程 (the formulas) and K/V Tile 遍历与核心计算 (the tiled
 * online-softmax loop this kernel implements); the LSE is the per-row
 * statistic the backward kernel of page "TileLang与机器学习训练：反向传播算子优化案例"
 * takes as input (section 算子拆分与流水线设计).
 * Q, K, V are read only.  O and LSE are written in full (LSE may not be NULL).
 */
fa_status fa_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int L,
                 int H, int Hkv, int D, int causal, int dtype, void* stream);

/*
 * Forward with fewer queries than keys (prefill against a key/value cache):
 * Q, O [B, Lq, H, D]; K, V [B, Lk, Hkv, D]; LSE [B, H, Lq].  Under causal
 * masking the queries are the last Lq positions of the Lk-long sequence:
 * query i sees key j iff j <= i + past_len with past_len = Lk - Lq (page
 * "TileLang性能分析报告：H100上FlashAttention吞吐量达1.2PFlops", section
 * 因果掩码优化, where the query index is the row plus past_len); causal
 * calls need Lk >= Lq.  Non-causal calls accept any Lq, Lk >= 1.  With
 * Lq == Lk this is fa_fwd.
 */
fa_status fa_fwd_kv(const void* Q, const void* K, const void* V, void* O, float* LSE, int B, int Lq,
                    int Lk, int H, int Hkv, int D, int causal, int dtype, void* stream);

/*
 * Forward on 8-bit inputs: Q8, K8, V8 hold E4M3 codes (one byte per element,
 * the OCP 8-bit floating point E4M3 format without infinities), in the
 * layouts above, each with one fp32 scale: the call computes the fa_fwd_kv
 * result (same masking rule, past_len = Lk - Lq) for the dequantised inputs
 *   Q = decode(Q8) * q_scale,  K = decode(K8) * k_scale,  V = decode(V8) * v_scale,
 * writing O [B, Lq, H, D] in `out_dtype` (FA_F16 or FA_BF16) and LSE
 * [B, H, Lq] in fp32.  Page "TileLang性能分析报告：H100上FlashAttention吞吐量达
 * 1.2PFlops", section 生产环境部署建议, item 1 (FP8 mixed-precision compute);
 * the loop is the online softmax of page "使用 TileLang 在 AMD GPU 上快速开发
 * 高性能 Flash Attention", section K/V Tile 遍历与核心计算, with P rounded to
 * E4M3 before the PV product, as that page rounds P to the input type.
 * Scores accumulate in fp32 from exact products; the rounding of P is the
 * one approximation (relative error at most 2^-4 per probability, absolute
 * 2^-10 below 2^-6).  Requires D = 128 (FA_ERR_UNSUPPORTED otherwise) and
 * finite scales > 0 (FA_ERR_INVALID_ARG otherwise).
 */
fa_status fa_fwd_fp8(const void* Q8, const void* K8, const void* V8, float q_scale,
                     float k_scale, float v_scale, void* O, float* LSE, int B, int Lq, int Lk,
                     int H, int Hkv, int D, int causal, int out_dtype, void* stream);

/*
 * Split-KV decoding: the forward of fa_fwd_kv (same result, layouts, masking
 * rule and causal past_len = Lk - Lq) computed for few queries against many
 * keys.  The keys of each (batch, K/V head) are cut into equal slices of
 * 128-key tiles, one CTA per slice, sized so the slices fill the GPU; each
 * slice yields a partial output and log-sum-exp in fp32, and a second kernel
 * merges them: LSE = ln sum_s exp(LSE_s), O = sum_s exp(LSE_s - LSE) O_s.
 * Page "TileLang性能分析报告：H100上FlashAttention吞吐量达1.2PFlops", section
 * 生产环境部署建议 (item 2 names flash_decoding for inference; the slicing and
 * merge are the plain reading of that name); the per-slice loop is the online
 * softmax of page "使用 TileLang 在 AMD GPU 上快速开发高性能 Flash Attention",
 * section K/V Tile 遍历与核心计算.
 * The g = H / Hkv query heads of a K/V head and all Lq queries share one
 * 128-row tile, so the call requires g * Lq <= 128 (FA_ERR_UNSUPPORTED
 * otherwise; use fa_fwd_kv).  `workspace` is the caller's device buffer of
 * `workspace_bytes` (16-byte aligned) holding the partials; it needs
 * fa_decode_workspace_size(...) bytes, asked with the same sizes and with the
 * device that will run the call current (the slice count depends on its SM
 * count).  Smaller buffers return FA_ERR_SCRATCH_TOO_SMALL and launch nothing.
 * Its contents need no initialisation and are unspecified afterwards; calls
 * that overlap on the GPU must not share one workspace.
 */
size_t fa_decode_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D);
fa_status fa_decode(const void* Q, const void* K, const void* V, void* O, float* LSE,
                    void* workspace, size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv,
                    int D, int causal, int dtype, void* stream);

/*
 * The two stages fa_decode runs, for callers that schedule or time them
 * apart: fa_decode_slices writes every slice's partial O and LSE into the
 * workspace; fa_decode_merge reads them and writes O and LSE.  Give both the
 * same sizes and run them on the same device, so that they derive the same
 * slice plan; the merge must run after the slices on the stream.
 */
fa_status fa_decode_slices(const void* Q, const void* K, const void* V, void* workspace,
                           size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv, int D,
                           int causal, int dtype, void* stream);
fa_status fa_decode_merge(const void* workspace, size_t workspace_bytes, void* O, float* LSE, int B,
                          int Lq, int Lk, int H, int Hkv, int D, int dtype, void* stream);

/*
 * Paged key/value cache.  K and V live in two pools of pages,
 * [num_pages, page, Hkv, D] (page in {16, 32, 64, 128, 256},
 * FA_ERR_UNSUPPORTED otherwise), whose pages are page_stride elements apart
 * (a multiple of 8, at least page * Hkv * D: both pools may be halves of one
 * tensor).  Row b of block_table [B, max_pages] int32 lists the pages of
 * sequence b in order: its key t lies in page block_table[b, t / page], row
 * t % page.  Tables and lengths are read on the device when the kernels run.
 * A page id outside [0, num_pages) reads as zero keys and values and is never
 * written; lengths are clamped to [0, max_pages * page].
 * Tables, lengths and the like need the alignment of an int only.
 * Key weights, where given, are fp32 [B, Hkv, *]: the weight of key t of
 * sequence b and K/V head h is weights[(b * Hkv + h) * weights_stride + t],
 * with weights_stride >= max_pages * page.
 *
 * fa_paged_write: put the new keys and values K, V [B, L, Hkv, D] into the
 * pages.  Token j of sequence b goes to position start[b] + j; only the first
 * counts[b] tokens when counts [B] is given (a padded batch).  Positions
 * outside the table are skipped.  With `weights`, the weights of the slots
 * written become new_weights [B, Hkv, L] (fa_key_weights of the prompt), or 0
 * when that is NULL; the two must not share memory (FA_ERR_INVALID_ARG).  Two
 * tokens of one call must not share a slot.
 */
fa_status fa_paged_write(const void* K, const void* V, void* K_pool, void* V_pool,
                         long long k_page_stride, long long v_page_stride, const int* block_table,
                         const int* start, const int* counts, float* weights,
                         long long weights_stride, const float* new_weights, int B, int L, int Hkv,
                         int D, int page, int max_pages, int num_pages, int dtype, void* stream);

/*
 * fa_paged_decode: attention of the last Lq tokens of every sequence over its
 * paged keys and values (already written).  lens [B] counts all keys, the new
 * ones included: query i of sequence b has position a = lens[b] - Lq + i and
 * sees key j iff j <= a and (window == 0, or j > a - window, or j < sinks).
 * A length beyond the table (max_pages * page) counts as the table's, one
 * below 0 as 0.  A query that sees nothing (a negative position, an empty
 * sequence) gives O = 0, LSE = -inf.  Keys that no query of the call sees are
 * never used, whatever their slots hold; pages wholly behind the length or
 * before the window are not read and may be absent from the table.  V must be
 * finite at a key that some query of the call sees: for the queries that do not
 * see it, it is multiplied by a zero weight.  NaN in a query or in a key it sees
 * gives that row NaN in O and LSE (and in the weights it adds).
 * Q, O [B, Lq, H, D]; LSE [B, H, Lq]; (H / Hkv) * Lq <= 128
 * (FA_ERR_UNSUPPORTED otherwise).  With `weights` the call adds to each
 * visible key's weight sum over the group's heads and the queries of
 * exp(q . k / sqrt(D) - LSE).  Every key is added to once, by one thread:
 * results do not depend on any order, and sequences may share pages.
 * `workspace`: fa_paged_decode_workspace_size bytes, asked with the device
 * that runs the call current (FA_ERR_SCRATCH_TOO_SMALL when smaller); with
 * `weights` it holds a raw score for every slot of the table and query head
 * (B * Hkv * ceil(max_pages * page / 128) * (H / Hkv) * Lq * 512 bytes), whatever
 * the lengths are, so a table no wider than needed saves memory.  Its
 * contents need no initialisation; calls (and replayed graphs) that overlap
 * on the GPU must not share one.  (After a device error in a replayed graph,
 * zero its workspace or capture it again before the next replay: the counts of
 * the parts that did finish are still in it.)  FA_ERR_UNSUPPORTED also for
 * 2^31 or more tiles of 128 keys (B * Hkv * ceil(max_pages * page / 128)), and
 * with `weights` for B * Hkv > 65535.
 */
size_t fa_paged_decode_workspace_size(int B, int Lq, int H, int Hkv, int D, int page, int max_pages,
                                      int weights);
fa_status fa_paged_decode(const void* Q, const void* K_pool, const void* V_pool,
                          long long k_page_stride, long long v_page_stride, const int* block_table,
                          const int* lens, void* O, float* LSE, float* weights,
                          long long weights_stride, void* workspace, size_t workspace_bytes, int B,
                          int Lq, int H, int Hkv, int D, int page, int max_pages, int num_pages,
                          int window, int sinks, int dtype, void* stream);

/*
 * Rotary positions.  A table of rotary / 2 entries, one per pair of a head's
 * dims, 16-byte aligned: entry i holds in its low 8 bits the pair's axis and
 * above them the turns that a position adds, f_i / (2 pi), as a fraction of 2^56
 * modulo 1 (two's complement: negative frequencies turn backwards).  The first
 * `rotary` dims of a head (a multiple of 16 up to D, FA_ERR_UNSUPPORTED
 * otherwise) are the pairs: dims i and i + rotary / 2, or with `interleaved` dims
 * 2 i and 2 i + 1; the others are copied.  Pair i (x, y) of a token at position n
 * on the pair's axis becomes
 *   (x cos t - y sin t, x sin t + y cos t),   t = n f_i,
 * with angles within 2^-23 rad of the entry's turns times n at every int32
 * position, computed in fp32, each result rounded once.  positions [axes, B, L] int32 (1 to 256 axes;
 * a table's axis beyond the last counts as the last), or NULL with one axis: the
 * token's number 0 .. L - 1.
 *
 * fa_rope: queries Q [B, L, H, D] and keys K [B, L, Hkv, D], turned, into Q_out
 * and K_out; K and K_out NULL with Hkv = 0 for queries alone.  With `backward`
 * it turns by -t: the gradients of Q and K from those of Q_out and K_out.  All four
 * have free strides between batch entries and tokens, in elements and multiples
 * of 8 (parts of a fused projection's rows; inputs may repeat, outputs may not);
 * the last two dims are contiguous.  An output may be its input itself (the same
 * pointer and strides); otherwise the two must not share memory
 * (FA_ERR_INVALID_ARG), nor may an output share an element with the other
 * tensor's operands.  H need not be a multiple of Hkv.
 */
fa_status fa_rope(const void* Q, long long q_batch, long long q_token, const void* K,
                  long long k_batch, long long k_token, void* Q_out, long long q_out_batch,
                  long long q_out_token, void* K_out, long long k_out_batch, long long k_out_token,
                  const long long* table, const int* positions, int axes, int B, int L, int H,
                  int Hkv, int D, int rotary, int interleaved, int backward, int dtype,
                  void* stream);

/*
 * fa_paged_append: fa_rope and fa_paged_write in one pass.  Queries Q [B, L, H, D]
 * are turned into Q_out, all of them; keys K and values V [B, L, Hkv, D] of the
 * tokens that count go into the pages, the keys turned.  Slots, counts, pages and
 * weights are fa_paged_write's, table and rotation fa_rope's; with positions NULL
 * (one axis) a token's position is its slot, start[b] + j.  Q, K, V and Q_out have
 * fa_rope's strides; Q_out may be Q itself, and shares no memory with anything
 * else of the call.
 */
fa_status fa_paged_append(const void* Q, long long q_batch, long long q_token, const void* K,
                          long long k_batch, long long k_token, const void* V, long long v_batch,
                          long long v_token, void* Q_out, long long q_out_batch,
                          long long q_out_token, void* K_pool, void* V_pool,
                          long long k_page_stride, long long v_page_stride, const int* block_table,
                          const int* start, const int* counts, const long long* table,
                          const int* positions, int axes, float* weights, long long weights_stride,
                          const float* new_weights, int B, int L, int H, int Hkv, int D, int rotary,
                          int interleaved, int page, int max_pages, int num_pages, int dtype,
                          void* stream);

/*
 * fa_paged_prefix_decode: fa_paged_decode (no window, no weights) for sequences
 * that share key/value prefixes, each prefix read once for every two tiles of
 * 128 / (H / Hkv) tokens of its sequences, not once a sequence.  Group i
 * is the sequences group_starts[i] .. group_starts[i + 1] - 1 (group_starts
 * [groups + 1] int32, never falling; NULL with one group: all of them); its
 * prefix is the first prefix_lens[i] keys of the pages in row i of prefix_table
 * [groups, prefix_pages].  block_table [B, max_pages] and lens [B] are the
 * sequences' own keys behind the prefix, the new tokens' included: query i of
 * sequence b sees its group's whole prefix and its own keys
 * j <= lens[b] - Lq + i.  A query whose own position lens[b] - Lq + i is
 * negative (an unused slot) is padding and gives O = 0, LSE = -inf.  A sequence
 * of no group, or with a prefix of length 0, has its own keys alone.  Prefixes
 * and own keys lie in the same two pools; tables, lengths and group_starts are
 * read on the device, lengths clamped to their tables and starts to [0, B]
 * (starts that fall anywhere give unspecified results).  Slots behind a length
 * are never used, whatever they hold; V must be finite at a key that some query
 * of the call sees, and NaN in a query or in a key it sees gives that row NaN.
 * As in all calls on 16-bit inputs, probabilities are rounded to their type before
 * the product with V (half a step, relative), sums take them unrounded.
 * (H / Hkv) * Lq <= 128 (FA_ERR_UNSUPPORTED otherwise).
 * Results do not depend on timing.  `workspace`:
 * fa_paged_prefix_decode_workspace_size bytes, asked with the device that runs
 * the call current (FA_ERR_SCRATCH_TOO_SMALL when smaller), under
 * fa_paged_decode's rules; it holds D + 1 floats for twice every query row
 * (B * Lq * H) and for 256 + (H / Hkv) * Lq rows of every SM, and 8 bytes for every
 * group, sequence and pair of tiles of 128 / (H / Hkv) tokens and K/V head.
 * FA_ERR_UNSUPPORTED where three times (D = 64: four times) the
 * 128-key tiles of all prefixes (at their tables' lengths, for each K/V head and
 * two tiles of tokens) and twice those of all own keys could add up to 2^32 or
 * more.
 */
size_t fa_paged_prefix_decode_workspace_size(int B, int Lq, int H, int Hkv, int D, int page,
                                             int groups, int prefix_pages, int max_pages);
fa_status fa_paged_prefix_decode(const void* Q, const void* K_pool, const void* V_pool,
                                 long long k_page_stride, long long v_page_stride,
                                 const int* prefix_table, const int* prefix_lens,
                                 const int* group_starts, const int* block_table, const int* lens,
                                 void* O, float* LSE, void* workspace, size_t workspace_bytes,
                                 int B, int Lq, int H, int Hkv, int D, int page, int groups,
                                 int prefix_pages, int max_pages, int num_pages, int dtype,
                                 void* stream);

/*
 * Key weights: how much attention each key of a prompt has received,
 *   W[b, hkv, j] = sum over the heads h of the group and the queries i that
 *                  see key j of exp(q_i . k_j / sqrt(D) - LSE[b, h, i]),
 * the column sums of the softmax whose LSE a forward call left (fa_fwd,
 * fa_fwd_kv, fa_window_fwd).  Q [B, Lq, H, D], K [B, Lk, Hkv, D], LSE
 * [B, H, Lq], W [B, Hkv, Lk] fp32, written in full.  The mask is fa_fwd_kv's,
 * or with window > 0 (causal calls only, FA_ERR_INVALID_ARG otherwise)
 * fa_window_fwd's.  A query whose LSE is -inf adds nothing.  All sums are fp32
 * in a fixed order: the result does not depend on timing.  `workspace`:
 * fa_key_weights_workspace_size() bytes, asked with the device that runs the
 * call current; no initialisation needed, not shared between calls that
 * overlap on the GPU.  FA_ERR_UNSUPPORTED for 2^31 or more steps (query head, Q
 * tile, K/V tile) per SM.
 */
size_t fa_key_weights_workspace_size(void);
fa_status fa_key_weights(const void* Q, const void* K, const float* LSE, float* W, void* workspace,
                         size_t workspace_bytes, int B, int Lq, int Lk, int H, int Hkv, int D,
                         int causal, int window, int sinks, int dtype, void* stream);

/*
 * Cut the paged caches of a batch down to `keep` keys per sequence and K/V
 * head by accumulated attention weight.  A sequence of n = lens[b] <= keep
 * keys survives whole; of a longer one each head keeps its first `sinks` keys,
 * its last `recent`, and of those between the keep - sinks - recent heaviest
 * by `weights` (NaN counts as heaviest, ties go to the lower position);
 * sinks + recent <= keep.  The survivors move, in their order, to positions
 * 0, 1, ... of the pages in dst_table [B, dst_pages] (dst_pages * page >=
 * keep) of the same pools.  The old pages and `weights` stay as they are, so
 * pages that sequences share are safe; the pages of dst_table must be pages
 * that no sequence of the call reads, each listed once.
 * Written in full: kept [B, Hkv, keep] int32 (old positions, ascending; -1
 * behind the last), new_lens [B] int32 = min(n, keep), new_weights
 * [B, Hkv, dst_pages * page] fp32 (the survivors' weights, 0 behind them).
 * new_lens may be lens itself (a cut in place); other than that no output may
 * share memory with the tables, lens, weights or another output
 * (FA_ERR_INVALID_ARG).
 * No workspace.  B * Hkv <= 65535 (FA_ERR_UNSUPPORTED otherwise).
 */
fa_status fa_paged_evict(void* K_pool, void* V_pool, long long k_page_stride,
                         long long v_page_stride, const int* block_table, const int* lens,
                         const float* weights, long long weights_stride, const int* dst_table,
                         int keep, int sinks, int recent, int* kept, int* new_lens,
                         float* new_weights, int B, int Hkv, int D, int page, int max_pages,
                         int dst_pages, int num_pages, int dtype, void* stream);

/*
 * Backward preprocess: Delta[b, h, i] = sum_d O[b, i, h, d] * dO[b, i, h, d]
 * (fp32 accumulation), the per-row term of the softmax gradient.  Page
 * "TileLang与机器学习训练：反向传播算子优化案例", section 算子拆分与流水线设计
 * (the "Delta" preprocessing stage; its printed block product is read as this
 * per-row dot product).  When `dq_accum` is not NULL it must point to
 * fa_bwd_workspace_size(B, L, H, D) bytes, which this call sets to zero in
 * the same pass, ready for fa_bwd.
 */
fa_status fa_bwd_preprocess(const void* O, const void* dO, float* Delta, float* dq_accum, int B,
                            int L, int H, int D, int dtype, void* stream);

/* Bytes of the fp32 dQ accumulator fa_bwd needs: B * H * ceil(L/128)*128 * D * 4. */
size_t fa_bwd_workspace_size(int B, int L, int H, int D);

/*
 * Backward attention: dQ, dK, dV of the forward above, given dO, the forward's
 * LSE and fa_bwd_preprocess's Delta.  With P = exp(S - LSE):
 *   dV = P^T dO,  dP = dO V^T,  dS = P o (dP - Delta),
 *   dQ = dS K / sqrt(D),  dK = dS^T Q / sqrt(D),
 * with dK, dV of a K/V head summed over its query heads.  Page
 * "TileLang与机器学习训练：反向传播算子优化案例", sections 算子拆分与流水线设计
 * (one K/V tile per CTA looping over Q tiles, dV accumulated from the
 * transposed probabilities) and 内存布局优化 (dQ accumulated in fp32 through
 * atomics into a layout matched to the accumulator fragments, then a
 * post-processing pass).
 * `dq_accum` is the caller's workspace (fa_bwd_workspace_size bytes, 16-byte
 * aligned); it must hold zeros on entry unless `zero_accum` is non-zero, in
 * which case this call zeroes it first.  Its contents afterwards are
 * unspecified.  O is accepted for interface symmetry and is not read (Delta
 * carries it); it may be NULL.  dQ, dK, dV are written in full.
 */
fa_status fa_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                 const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                 float* dq_accum, int zero_accum, int B, int L, int H, int Hkv, int D, int causal,
                 int dtype, void* stream);

/*
 * Backward of fa_fwd_kv: Q, O, dO, dQ [B, Lq, H, D]; K, V, dK, dV
 * [B, Lk, Hkv, D]; LSE, Delta [B, H, Lq]; dq_accum of
 * fa_bwd_workspace_size(B, Lq, H, D) bytes (fa_bwd_preprocess with L = Lq
 * computes Delta and zeroes it).  Same masking rule and limits as fa_fwd_kv.
 */
fa_status fa_bwd_kv(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                    const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                    float* dq_accum, int zero_accum, int B, int Lq, int Lk, int H, int Hkv, int D,
                    int causal, int dtype, void* stream);

/*
 * Sliding-window attention with sinks, forward and backward.  The masks of
 * fa_fwd_kv's causal rule (past_len = Lk - Lq, Lk >= Lq) narrowed to a window:
 * the query at position a = i + past_len sees key j iff
 *   j <= a  and  (j > a - window  or  j < sinks),
 * that is itself, the window - 1 keys before it, and the first `sinks` keys of
 * the sequence.  window >= 1 and sinks >= 0 (FA_ERR_INVALID_ARG otherwise); a
 * window of Lk or more is plain causal attention.  Every query sees at least
 * itself, so no row is empty.  Work and reads grow with
 * Lq * (window + sinks), not with Lq * Lk.  K and V must be finite in every
 * position, as for fa_fwd: a hidden key's V is multiplied by a zero weight.
 * Everything else (layouts, dtypes, limits, Delta from fa_bwd_preprocess) is
 * as for fa_fwd_kv and fa_bwd_kv; dK and dV of keys that no query sees are
 * zero.  The backward's workspace holds fa_window_bwd_workspace_size bytes
 * (FA_ERR_SCRATCH_TOO_SMALL when smaller): first the fp32 dQ accumulator of
 * fa_bwd_workspace_size(B, Lq, H, D) bytes, which must hold zeros on entry
 * (fa_bwd_preprocess sets them) unless zero_accum, then fp32 parts of dK and
 * dV, which need no initialisation.  Ask for the size with the device that runs
 * the call current: how the work is cut depends on its SMs.  dK and dV do not
 * depend on timing; dQ is summed by fp32 atomics, as in fa_bwd.
 */
fa_status fa_window_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE, int B,
                        int Lq, int Lk, int H, int Hkv, int D, int window, int sinks, int dtype,
                        void* stream);
size_t fa_window_bwd_workspace_size(int B, int Lq, int Lk, int H, int Hkv, int D, int window,
                                    int sinks);
fa_status fa_window_bwd(const void* Q, const void* K, const void* V, const void* dO,
                        const float* LSE, const float* Delta, void* dQ, void* dK, void* dV,
                        float* workspace, size_t workspace_bytes, int zero_accum, int B, int Lq,
                        int Lk, int H, int Hkv, int D, int window, int sinks, int dtype,
                        void* stream);

/*
 * The two stages fa_bwd runs, for callers that schedule or time them apart:
 *   fa_bwd_main        dK, dV (written in full) and the dQ accumulator (added
 *                      into; it must hold zeros on entry unless zero_accum);
 *   fa_bwd_postprocess dQ = dq_accum / sqrt(D), converted back to BSHD.
 * Page "TileLang与机器学习训练：反向传播算子优化案例", section
 * 算子拆分与流水线设计 (the core gradient stage and the post-processing stage
 * that reorders the dQ gradient).  Arguments mean what they mean for fa_bwd.
 */
fa_status fa_bwd_main(const void* Q, const void* K, const void* V, const void* dO,
                      const float* LSE, const float* Delta, void* dK, void* dV, float* dq_accum,
                      int zero_accum, int B, int L, int H, int Hkv, int D, int causal, int dtype,
                      void* stream);
fa_status fa_bwd_postprocess(const float* dq_accum, void* dQ, int B, int L, int H, int D,
                             int dtype, void* stream);

/*
 * fa_bwd for callers that cannot allocate device memory at call time: a
 * plugin running inside a host application that owns all GPU memory through
 * its own pool and hands out no allocator, or a serving path that must not
 * allocate once it has started.  This is a library facility; the pages have
 * no counterpart.
 * Same arguments and results as fa_bwd, minus the workspace.  Such a caller
 * gets Delta from fa_bwd_preprocess with a NULL dq_accum (which needs no
 * workspace either).  The fp32 dQ
 * accumulator lives in a fixed device array of FA_NOALLOC_SCRATCH_BYTES that
 * the library's module holds on every GPU that loads it, until exit.  The
 * call allocates nothing (no cudaMalloc, cudaFree or allocating library
 * routine); it clears the part of the array it uses, then runs the backward.
 * Limits and rules:
 *   - B * H * ceil(L/128)*128 * D * 4 bytes must not exceed
 *     FA_NOALLOC_SCRATCH_BYTES (64 MiB, e.g. B=1, H=32, L=4096, D=128);
 *     larger problems return FA_ERR_SCRATCH_TOO_SMALL and launch nothing.
 *   - Every call on a device shares the one array: calls whose work overlaps
 *     on the GPU (other streams, other host threads) race and corrupt each
 *     other's dQ.  Serialise them.
 *   - Each call looks up the array's device address on the current device
 *     (the address can change if the device is reset and the module loaded
 *     again) and remembers it; a call made while its stream is being
 *     captured uses the remembered address instead.  Make the first call on
 *     each device before any stream capture on that device.
 */
#define FA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
fa_status fa_bwd_noalloc(const void* Q, const void* K, const void* V, const void* O,
                         const void* dO, const float* LSE, const float* Delta, void* dQ,
                         void* dK, void* dV, int B, int L, int H, int Hkv, int D, int causal,
                         int dtype, void* stream);

/*
 * Synchronise `stream` and report whether any kernel of this library gave up
 * a bounded wait since the last check (FA_ERR_DEVICE_TIMEOUT; the word is then
 * cleared).  Kernels never trap or spin forever: a wait that exceeds about one
 * second records its site id, unwinds the CTA and returns.
 */
fa_status fa_check_device_error(void* stream);

/*
 * Exercise the bounded-wait failure path without any fault: launches one
 * thread that waits on an mbarrier nothing ever completes.  After
 * `limit_ns` (clamped to 1 ms .. 1 s) the wait gives up, records site 900 in
 * the device error word and the kernel returns; the next
 * fa_check_device_error on the stream then returns FA_ERR_DEVICE_TIMEOUT and
 * the CUDA context stays usable.  A library facility with no counterpart on
 * the pages.
 */
fa_status fa_selftest_bounded_wait(unsigned long long limit_ns, void* stream);

/* Site id recorded by the last FA_ERR_DEVICE_TIMEOUT (0 if none). */
unsigned int fa_last_error_site(void);

/* Static, human-readable text for a status value. */
const char* fa_status_string(fa_status status);

/* Library version string. */
const char* fa_version(void);

#ifdef __cplusplus
}
#endif

#endif /* TILED_ATTENTION_FA_GB300_FA_H */
