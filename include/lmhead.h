/*
 * lmhead.h -- C ABI of the B200 (sm_100a) LM-head loss path.
 *
 * The library computes, on one GPU:
 *   lmhead_fwd     logits[M,V] = X[M,K] . W[V,K]^T, FP32 accumulator stored
 *                  unrounded (or a BF16 copy of it, for comparison)
 *   ce_fwd         per-row cross-entropy statistics {m, d, x_y, loss}
 *   ce_bwd         dlogits = (softmax - onehot(target)) * grad_loss, in FP32,
 *                  rounded to the output dtype only at the store
 *   lmhead_bwd_dx  dX[M,K] = dlogits[M,V] . W[V,K]
 *   lmhead_bwd_dw  dW[V,K] = dlogits[M,V]^T . X[M,K]
 * and, for serving and fine-tuning beside it, the same projection with a
 * low-rank adapter per token (lmhead_fwd_lora, lmhead_bwd_dx_lora,
 * lmhead_bwd_lora) and beam search over its logits (beam_select, beam_reorder).
 *
 * Sources (page title, section):
 *   [P1] Megatron-LM PR #6252 "Add mixed-precision (FP32) LM output logits":
 *        "What does this PR do?" (FP32 GEMM output instead of BF16-rounded
 *        logits; gradients cast back to BF16 under the GEMM contract),
 *        "Tests" (only bf16 and fp32 logit dtypes are accepted, fp16 is
 *        rejected), "Integer bitwise exactness results".
 *   [P2] TransformerEngine #2325 "[Pytorch] change fused cross entropy
 *        backward grad to fp32 and reduce one read": "Description" and
 *        "Changes" (backward computed in FP32, one fewer read of the logits)
 *        and the review discussion (the forward saves the target, n_rows x 1,
 *        and m_d_X_y, n_rows x 4).
 *
 * Conventions shared by every call
 *   - All array arguments are DEVICE pointers into row-major, contiguous
 *     buffers owned by the caller.  The library allocates nothing, keeps no
 *     per-call state and never synchronises: every call only enqueues work on
 *     `stream` (NULL = legacy default stream) and returns.
 *   - BF16 data is IEEE binary32's upper 16 bits; FP32 is IEEE binary32.
 *   - Errors are returned, never raised: arguments are validated on the host
 *     before anything is launched, and a failing launch maps to LMH_ERR_CUDA.
 *   - `status` (nullable) is a device int32 word that kernels OR condition
 *     bits into (LMH_DEV_*).  The caller zeroes it, and reads it after the
 *     stream has been synchronised.  Nothing is trapped on the device.
 *   - Sizes are int64; every size must be >= 1 unless stated otherwise.
 */
#ifndef LMHEAD_H_
#define LMHEAD_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported from liblmhead.so (everything else in the library is hidden). */
#if defined(__GNUC__)
#define LMH_API __attribute__((visibility("default")))
#else
#define LMH_API
#endif

/* Host-side result of a call. */
typedef enum {
    LMH_OK = 0,
    LMH_ERR_INVALID_ARG = 1,  /* null pointer, size < 1, size too large   */
    LMH_ERR_MISALIGNED = 2,   /* pointer or row stride breaks the layout  */
    LMH_ERR_UNSUPPORTED = 3,  /* dtype or stride value not supported      */
    LMH_ERR_CUDA = 4          /* the CUDA runtime reported an error       */
} lmh_status_t;

/* Element types.  As with the logit-dtype option of [P1] "Tests", only FP32
 * and BF16 are accepted; LMH_F16 (and any other value) is rejected with
 * LMH_ERR_UNSUPPORTED. */
typedef enum { LMH_F32 = 0, LMH_BF16 = 1, LMH_F16 = 2 } lmh_dtype_t;

/* Bits ORed into *status by the kernels. */
#define LMH_DEV_BAD_TARGET 0x1   /* a target neither ignore_index nor in [0,V);
                                    the row was treated as ignored          */
#define LMH_DEV_PIPE_TIMEOUT 0x2 /* a pipeline wait gave up (bounded spin);
                                    the output of that call is not valid    */
#define LMH_DEV_BAD_LOGIT 0x4    /* beam_select met a logit that is NaN or not
                                    below 1e38, or a score of NaN or +inf; each
                                    was taken as -inf                       */
#define LMH_DEV_BAD_ADAPTER 0x8  /* an adapter id neither -1 nor in [0, N); the
                                    token was treated as having none        */
#define LMH_DEV_BAD_PARENT 0x10  /* beam_reorder met a parent outside [0, W);
                                    that beam's state was left as it was    */

/* Same type as cudaStream_t. */
typedef struct CUstream_st *lmh_stream_t;

/* logits = X . W^T  ([P1] "What does this PR do?").
 *   X       [M,K] BF16, K contiguous.         W [V,K] BF16, K contiguous.
 *   logits  [M,V] FP32 (out_dtype LMH_F32: the accumulator, unrounded) or
 *           BF16 (LMH_BF16: the accumulator rounded to nearest even).
 *   Requirements: K % 8 == 0 (16-byte rows for the tensor-memory copies),
 *   X and W 16-byte aligned, logits 4-byte aligned; M, V, K <= 2^31 - 1.
 *   Accumulation is FP32 inside the tensor cores; when every partial sum is
 *   an exactly representable integer (BF16 integers in [-8,8] with
 *   K * 64 < 2^24, [P1] "Integer bitwise exactness results") the FP32 output
 *   is exact.  Deterministic: repeated calls give identical bits. */
LMH_API lmh_status_t lmhead_fwd(const void *X, const void *W, void *logits, int32_t out_dtype,
                        int64_t M, int64_t K, int64_t V, int32_t *status,
                        lmh_stream_t stream);

/* Cross-entropy forward statistics ([P2] discussion: target and m_d_X_y).
 *   logits  [M,V] FP32.   target [M] int64.
 *   stats   [M,4] FP32, per row {m, d, x_y, loss}:
 *             m = max_j x_j, d = sum_j exp(x_j - m), x_y = x[target],
 *             loss = -log softmax(x)_target = m + log(d) - x_y, computed as
 *             log1p(s exp(m - x_y)) with s = d - exp(x_y - m) summed over the
 *             other columns, so that it keeps its precision when the target
 *             holds nearly all of the row's mass.
 *   A row whose target equals ignore_index is not read and gets
 *   {0,0,0,0}.  A target outside [0,V) that is not ignore_index sets
 *   LMH_DEV_BAD_TARGET in *status and the row is treated as ignored.
 *   Any V >= 1; no alignment beyond the element size. */
LMH_API lmh_status_t ce_fwd(const float *logits, const int64_t *target, float *stats,
                    int64_t M, int64_t V, int64_t ignore_index, int32_t *status,
                    lmh_stream_t stream);

/* Cross-entropy backward in FP32 ([P2] "Description", "Changes"; the BF16
 * cast at the end is the one of [P1] "What does this PR do?").
 *   logits     [M,V] FP32, the same buffer ce_fwd read.
 *   target     [M] int64.   stats [M,4] FP32 from ce_fwd.
 *   grad_loss  FP32 upstream gradient of the per-row loss:
 *              grad_loss_stride 0 = one scalar for every row,
 *              1 = one value per row ([M]); anything else is unsupported.
 *   dlogits    [M,V], dl_dtype LMH_F32 or LMH_BF16 (round to nearest even):
 *              dl[i,j] = (exp(x_ij - m_i) / d_i - [j == target_i]) * g_i;
 *              at the target, softmax - 1 = exp(-loss_i) - 1 is taken as
 *              expm1(-loss_i) from the saved loss (no cancellation).
 *              Ignored and bad-target rows are written as zeros.
 *              With LMH_F32, dlogits may be the logits buffer itself
 *              (in-place; each element is read before it is overwritten).
 *   Any V >= 1. */
LMH_API lmh_status_t ce_bwd(const float *logits, const int64_t *target, const float *stats,
                    const float *grad_loss, int64_t grad_loss_stride, void *dlogits,
                    int32_t dl_dtype, int64_t M, int64_t V, int64_t ignore_index,
                    int32_t *status, lmh_stream_t stream);

/* logits = X . W^T (FP32) and the cross-entropy forward statistics of those
 * logits in one pass over them: the vocabulary GEMM's epilogue reduces every
 * 128-wide vocabulary block of each token row to a partial (max, sum-exp,
 * the sum leaving out the target's own term) in
 * `workspace` and records the target logit while the tile is still on chip,
 * and a second kernel merges each token's partials (in a fixed order) into
 * stats[M,4] = {m, d, x_y, loss}.  The logits are written but not read back
 * -- the "one fewer read of the logits" of [P2] "Changes", taken one step
 * further than a separate ce_fwd.
 *   Arguments and results as lmhead_fwd (out_dtype FP32) followed by ce_fwd
 *   (same tolerances; the statistics are merged in a different order, so they
 *   need not be bitwise equal to ce_fwd's).
 *   workspace: device scratch of at least lmhead_fwd_ce_workspace_bytes(M, V)
 *   bytes, 16-byte aligned, owned by the caller; its contents on entry do not
 *   matter and on return are unspecified.  When V % 4 != 0 or logits is not
 *   16-byte aligned the call runs lmhead_fwd then ce_fwd and does not touch
 *   the workspace (which may then be NULL). */
LMH_API lmh_status_t lmhead_fwd_ce(const void *X, const void *W, const int64_t *target,
                                   float *logits, float *stats, void *workspace,
                                   int64_t workspace_bytes, int64_t M, int64_t K, int64_t V,
                                   int64_t ignore_index, int32_t *status, lmh_stream_t stream);

/* Scratch bytes lmhead_fwd_ce needs: 2 * ceil(V / 256) blocks x M tokens x
 * 8 bytes (2 MB for M = 1024, V = 32768).  -1 for sizes out of range. */
LMH_API int64_t lmhead_fwd_ce_workspace_bytes(int64_t M, int64_t V);

/* lmhead_fwd_ce for callers that cannot allocate device memory (no
 * counterpart on the pages).  Some callers cannot give the library a scratch
 * buffer: plug-ins whose host framework owns all device memory and offers
 * them no allocator, and code on paths where calling cudaMalloc (which may
 * synchronise the device) is not allowed.  This call computes exactly what
 * lmhead_fwd_ce computes (same arguments minus the workspace) but keeps the
 * partial statistics in a fixed 8 MiB array inside the library, which every
 * GPU that loads the library holds until the process exits.  It allocates
 * nothing and calls no allocating routine.
 *   Limit: M * 2 * ceil(V / 256) <= 1048576 (e.g. M = 4096 with V up to
 *   32768); larger problems return LMH_ERR_INVALID_ARG before anything is
 *   launched.  (When V % 4 != 0 or logits is not 16-byte aligned the call
 *   runs lmhead_fwd then ce_fwd, which need no scratch, at any size.)
 *   The first call on each device looks up the array's device address
 *   (cudaGetSymbolAddress, with that device current); make that first call
 *   before any stream capture.  The address is kept for the life of the
 *   process: do not use this call on a device after cudaDeviceReset (or
 *   after its primary context has been destroyed), when the library's
 *   device image, and the array with it, may be loaded at another address.
 *   Every call shares the one array per device: calls that may run at the
 *   same time on the GPU (different streams, or different host threads)
 *   race and corrupt each other's results.  Nothing in the array has to start
 *   at zero: each call writes every entry it later reads. */
LMH_API lmh_status_t lmhead_fwd_ce_noalloc(const void *X, const void *W, const int64_t *target,
                                           float *logits, float *stats, int64_t M, int64_t K,
                                           int64_t V, int64_t ignore_index, int32_t *status,
                                           lmh_stream_t stream);

/* Vocabulary-parallel cross-entropy (the vocabulary split across devices, as
 * Megatron's VocabParallelCrossEntropy does, named in [P2] "Description").
 * Device r holds logits[M, V_r] for vocabulary entries [offset_r, offset_r +
 * V_r) of a vocabulary of vocab_total; targets are global ids.  The three
 * calls below are the per-device parts; the exchange between devices (an
 * all-gather of the [M,4] shard records) is the caller's.
 *
 * ce_fwd_shard: per row of this shard, shard_stats[M,4] = {m_r, d_r, x_y or 0,
 *   1 if the target is in this shard else 0}: m_r = the max over the shard's
 *   columns, d_r = sum of exp(x - m_r) over them, leaving out the target's own
 *   term in the shard that holds it; ignored rows (target ==
 *   ignore_index) and bad targets (outside [0, vocab_total)) give zeros, bad
 *   targets also set LMH_DEV_BAD_TARGET.
 *   Requirements: 0 <= vocab_offset, vocab_offset + V <= vocab_total. */
LMH_API lmh_status_t ce_fwd_shard(const float *logits, const int64_t *target, float *shard_stats,
                                  int64_t M, int64_t V, int64_t vocab_offset, int64_t vocab_total,
                                  int64_t ignore_index, int32_t *status, lmh_stream_t stream);

/* ce_merge_shards: stats[M,4] = {m, d, x_y, loss} of the whole vocabulary
 * from the num_shards records of every shard, laid out shard-major
 * (shard_stats[r][M][4]): m = max_r m_r, s = sum_r d_r exp(m_r - m) taken in
 * shard order (deterministic; every column but the target), x_y from the
 * owning shard, d = s + exp(x_y - m), loss = log1p(s exp(m - x_y)).  The
 * result is what ce_fwd gives on the whole rows, up to the order of the sums. */
LMH_API lmh_status_t ce_merge_shards(const float *shard_stats, int64_t num_shards,
                                     const int64_t *target, float *stats, int64_t M,
                                     int64_t vocab_total, int64_t ignore_index, int32_t *status,
                                     lmh_stream_t stream);

/* ce_bwd_shard: ce_bwd on a shard, with the merged stats: dl[i,j] =
 * (exp(x_ij - m_i) / d_i - [vocab_offset + j == target_i]) * g_i, the target's
 * entry as in ce_bwd. */
LMH_API lmh_status_t ce_bwd_shard(const float *logits, const int64_t *target, const float *stats,
                                  const float *grad_loss, int64_t grad_loss_stride, void *dlogits,
                                  int32_t dl_dtype, int64_t M, int64_t V, int64_t vocab_offset,
                                  int64_t vocab_total, int64_t ignore_index, int32_t *status,
                                  lmh_stream_t stream);

/* dX = dlogits . W, the input gradient of logits = X . W^T
 * ([P1] "What does this PR do?", backward under the GEMM contract: the
 * gradient GEMMs take the BF16 dlogits cast from the FP32 backward).
 *   dlogits [M,V] BF16.  W [V,K] BF16.
 *   dX      [M,K] FP32 (LMH_F32) or BF16 (LMH_BF16).
 *   Requirements: V % 8 == 0 and K % 8 == 0 (16-byte rows), inputs 16-byte
 *   aligned.  Deterministic.  With an FP32 dX the output tiles of a last
 *   wave that would leave most SMs idle are computed as two halves of the
 *   reduction that are both added into rows of dX the call first zeroes on
 *   the stream; with two addends the order of the additions does not change
 *   the result. */
LMH_API lmh_status_t lmhead_bwd_dx(const void *dlogits, const void *W, void *dX, int32_t out_dtype,
                           int64_t M, int64_t K, int64_t V, int32_t *status,
                           lmh_stream_t stream);

/* dW = dlogits^T . X, the weight gradient of logits = X . W^T
 * ([P1] "What does this PR do?", backward under the GEMM contract: the
 * gradient GEMMs take the BF16 dlogits cast from the FP32 backward).
 *   dlogits [M,V] BF16.  X [M,K] BF16.
 *   dW      [V,K] FP32 (LMH_F32) or BF16 (LMH_BF16).
 *   Requirements: V % 8 == 0 and K % 8 == 0, inputs 16-byte aligned.
 *   Deterministic. */
LMH_API lmh_status_t lmhead_bwd_dw(const void *dlogits, const void *X, void *dW, int32_t out_dtype,
                           int64_t M, int64_t K, int64_t V, int32_t *status,
                           lmh_stream_t stream);

/* dW += dlogits^T . X: the weight gradient accumulated into an FP32 main
 * gradient (beta = 1), as when gradients of several micro-batches are summed
 * before the optimizer step.
 *   dlogits [M,V] BF16, X [M,K] BF16, dW [V,K] FP32 (read and written).
 *   Each dW element receives exactly one FP32 addition per call (performed
 *   by the TMA reduce-add of the epilogue, or one atomic add where a tensor
 *   map cannot describe dW), so the result does not depend on scheduling:
 *   dW_out = fl(dW_in + fl32-accumulated product).
 *   Requirements as lmhead_bwd_dw. */
LMH_API lmh_status_t lmhead_bwd_dw_acc(const void *dlogits, const void *X, float *dW, int64_t M,
                                       int64_t K, int64_t V, int32_t *status, lmh_stream_t stream);

/* The LM head with low-rank adapters, one per token (no counterpart on the
 * pages): the tokens of many requests share W, and each has its own adapter
 * (A_a [R,K], B_a [V,R]) beside it, or none.
 *   u[i,:]      = scale[a] X[i,:] . A_a^T                       a = adapter[i]
 *   logits[i,:] = X[i,:] . W^T + u[i,:] . B_a^T
 *   A [N,R,K] BF16, B [N,V,R] BF16, scale [N] FP32, of N adapters of rank R
 *   (adapters of lower rank padded with zeros).   adapter [M] int32: -1 for a
 *   token without one; any other value outside [0,N) sets LMH_DEV_BAD_ADAPTER
 *   and counts as -1.
 *   u       [M,R] FP32, written (0 for a token without adapter); the backward
 *           calls take it.   logits as lmhead_fwd.
 *   One kernel forms both products in the same sums, FP32 rounded to nearest
 *   every 768 terms of K or fewer (4096 for BF16 logits, where the tiles are not cut
 *   along K), so the base part is as
 *   lmhead_fwd's but with a smaller error and not bitwise equal to it.  u enters the
 *   second product with FP32's 24 bits (above 128 tokens as three BF16 parts), for
 *   BF16 logits too.  An adapter's values reach the tokens that use it and no
 *   others, infinities and NaN included (for its own tokens an infinity may come
 *   out as NaN, since the parts of u multiply it one by one).  Any order of the
 *   tokens; those of one adapter next to each other cost least (each 256-token
 *   tile reads the adapters that occur in it).
 *   workspace: device scratch of lmhead_lora_workspace_bytes(M, K, V, R, N)
 *   bytes, 256-byte aligned; its contents do not matter before or after.
 *   Requirements: K % 8 == 0, R % 8 == 0, R <= 256, N <= 65535, M <= 4194240, M N <= 2^34;
 *   X, W, A, B, u 16-byte aligned; logits aligned to its element.
 *   Deterministic. */
LMH_API lmh_status_t lmhead_fwd_lora(const void *X, const void *W, const void *A, const void *B,
                                     const float *scale, const int32_t *adapter, float *u,
                                     void *logits, int32_t out_dtype, void *workspace,
                                     int64_t workspace_bytes, int64_t M, int64_t K, int64_t V,
                                     int64_t R, int64_t N, int32_t *status, lmh_stream_t stream);

/* Scratch bytes each of the three adapter calls needs at most.  -1 for sizes out
 * of range. */
LMH_API int64_t lmhead_lora_workspace_bytes(int64_t M, int64_t K, int64_t V, int64_t R, int64_t N);

/* The input gradient of lmhead_fwd_lora:
 *   g[i,:]  = scale[a] dlogits[i,:] . B_a          (written, [M,R] FP32)
 *   dX[i,:] = dlogits[i,:] . W + g[i,:] . A_a      (FP32 or BF16)
 * summed as in lmhead_fwd_lora (FP32 dX: every 512 terms of V, BF16 dX: every 4096),
 * g with FP32's 24 bits.  Requirements as there, and V % 8 == 0, dlogits, g and dX
 * 16-byte aligned.  Deterministic. */
LMH_API lmh_status_t lmhead_bwd_dx_lora(const void *dlogits, const void *W, const void *A,
                                        const void *B, const float *scale, const int32_t *adapter,
                                        float *g, void *dX, int32_t out_dtype, void *workspace,
                                        int64_t workspace_bytes, int64_t M, int64_t K, int64_t V,
                                        int64_t R, int64_t N, int32_t *status, lmh_stream_t stream);

/* The adapters' gradients, from the u of lmhead_fwd_lora and the g of
 * lmhead_bwd_dx_lora:
 *   dA_a = sum over its tokens of g[i,:]^T . X[i,:]        [N,R,K] FP32
 *   dB_a = sum over its tokens of dlogits[i,:]^T . u[i,:]  [N,V,R] FP32
 * zeros for an adapter without tokens.  u and g enter as three BF16 parts
 * (FP32's 24 bits).  Requirements as lmhead_bwd_dx_lora; dA and dB 16-byte
 * aligned.  Deterministic. */
LMH_API lmh_status_t lmhead_bwd_lora(const void *dlogits, const void *X, const float *u,
                                     const float *g, const int32_t *adapter, float *dA, float *dB,
                                     void *workspace, int64_t workspace_bytes, int64_t M, int64_t K,
                                     int64_t V, int64_t R, int64_t N, int32_t *status,
                                     lmh_stream_t stream);

/* One step of beam search over the logits: of all continuations of the W beams
 * of each of N batch entries, the C best, and the W beams that go on (no
 * counterpart on the pages; the log-softmax is that of ce_fwd).
 *   logits  [N,W,V] FP32 or BF16 (logits_dtype), as lmhead_fwd or
 *           lmhead_fwd_lora store them.   scores [N,W] FP32, log-probability
 *           of each beam so far.
 *   total[w,v] = scores[w] + logits[w,v] - log sum_v exp(logits[w,v]).
 *   done    [N] int32 or NULL: an entry with done != 0 is not read and keeps
 *           its beams (next_score = scores, next_beam = w); its candidates are
 *           (-inf, -1, -1).
 *   cand_score / cand_beam / cand_token [N,C] (FP32, int32, int64): the C best
 *           continuations, best first, compared by the FP64 value of total and,
 *           where equal, by the lower w, the higher logit, the lower v.  The
 *           logarithm of a row's sum is off by at most 2^-20 of the probability that
 *           lies outside its C best (1e-9 where they hold nearly all, 4e-8 measured on
 *           rows of many likely tokens); beams closer than that may change places.
 *           A logit or score of -inf
 *           forbids a continuation: where fewer than C are possible the rest is
 *           (-inf, -1, -1).  Logits as low as the type goes are continuations like
 *           any other; a total below FP32's range counts as -inf.
 *   next_score / next_beam / next_token [N,W], all three or none (NULL): the
 *           first W candidates whose token is not eos (eos = -1: none is), in
 *           order.  Places that no candidate fills get (-inf, w, eos, or 0 for
 *           eos = -1), w being the place itself.  next_score may be scores.
 *   workspace: device scratch of beam_select_workspace_bytes(N, W, V, C) bytes,
 *           16-byte aligned; its contents do not matter before or after.
 *   Limits: W <= 64, C <= 128, and with next_*: C >= 2 W (C >= W for eos = -1),
 *   so that W candidates go on however many end; -1 <= eos < V.  Any V >= 1;
 *   logits aligned to its element.  Deterministic.  Logits that are NaN or not
 *   below 1e38 set LMH_DEV_BAD_LOGIT and count as -inf. */
LMH_API lmh_status_t beam_select(const void *logits, int32_t logits_dtype, const float *scores,
                                 const int32_t *done, float *cand_score, int32_t *cand_beam,
                                 int64_t *cand_token, float *next_score, int32_t *next_beam,
                                 int64_t *next_token, void *workspace, int64_t workspace_bytes,
                                 int64_t N, int64_t W, int64_t V, int64_t C, int64_t eos,
                                 int32_t *status, lmh_stream_t stream);

/* Scratch bytes beam_select needs: 16 + 8 C bytes per part of a row, a part being
 * 4096 to 32768 logits, the longer the more rows there are.  -1 for sizes out of
 * range. */
LMH_API int64_t beam_select_workspace_bytes(int64_t N, int64_t W, int64_t V, int64_t C);

/* Puts the beams' states (caches, token histories) in the order of their
 * parents, in place: state[.., n, w, ..] = old state[.., n, parents[n,w], ..].
 * Beams whose parent is their own place are not touched.
 *   states   HOST array of num_states (1..128) device pointers to states of one
 *            geometry: element (o, n, w) starts at
 *            sum_i o_i outer_stride[i] + n entry_stride + w beam_stride and has
 *            run_bytes contiguous bytes; outer and outer_stride are HOST arrays
 *            of num_outer (0..3) extents and strides.  All strides in bytes.
 *            Elements of a state must not overlap, nor different states: both are
 *            checked, from the strides and the pointers, and refused
 *            (LMH_ERR_INVALID_ARG).  States that lie between each other's rows are fine.
 *   parents  [N,W] int32 (beam_select's next_beam).  A parent outside [0, W)
 *            sets LMH_DEV_BAD_PARENT and leaves that beam's state as it was.
 *   Limits: N <= 65535, W <= 64.  Any alignment: 16-byte copies where the
 *   pointers, strides and run_bytes allow them, narrower ones otherwise. */
LMH_API lmh_status_t beam_reorder(void *const *states, int64_t num_states, const int32_t *parents,
                                  int64_t N, int64_t W, int64_t entry_stride, int64_t beam_stride,
                                  int64_t run_bytes, const int64_t *outer,
                                  const int64_t *outer_stride, int64_t num_outer, int32_t *status,
                                  lmh_stream_t stream);

/* Static, NUL-terminated description of a status value. */
LMH_API const char *lmh_status_string(lmh_status_t s);

/* Library version, major * 10000 + minor * 100 + patch. */
LMH_API int32_t lmh_version(void);

/* Self-test of the pipeline watchdog (failure detection; no counterpart on
 * the pages).  Launches one CTA whose thread waits, with the same bounded
 * wait the GEMM pipelines use, on a shared-memory barrier that nothing
 * arrives at, with a limit of `limit_us` microseconds (1..1000000).  The wait
 * gives up, the CTA unwinds and LMH_DEV_PIPE_TIMEOUT is ORed into *status
 * (device int32, required).  Nothing faults or hangs; the context stays
 * usable.  Asynchronous like every other call. */
LMH_API lmh_status_t lmh_watchdog_selftest(int32_t *status, int64_t limit_us, lmh_stream_t stream);

/* Self-test of the GEMM's own failure path (failure detection; no
 * counterpart on the pages).  Runs lmhead_fwd with FP32 logits, the same
 * kernel selection and arguments, but with every pipeline wait limited to
 * `limit_ns` nanoseconds (1..1000000000) instead of two seconds.  With a limit
 * far below the time one output tile takes (1 ns, say), a wait runs out: the
 * CTA stops, lets every operand copy it issued land and every MMA it issued
 * finish, frees its tensor memory and ORs LMH_DEV_PIPE_TIMEOUT into *status
 * (device int32, required).  The logits are then not valid.  Nothing faults
 * or hangs, and later calls on the stream run normally. */
LMH_API lmh_status_t lmh_gemm_watchdog_selftest(const void *X, const void *W, float *logits,
                                                int64_t M, int64_t K, int64_t V, int64_t limit_ns,
                                                int32_t *status, lmh_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LMHEAD_H_ */
