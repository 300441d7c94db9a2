/*
 * tt_ops.h -- op-level C ABI: the individual kernels tt_gpt2_step is built
 * from, callable on their own (tests check each one against a CPU reference;
 * small programs can build their own training steps from them).
 *
 * Every call enqueues on the context's stream and takes device pointers.
 * `dtype` selects the storage type of activations and weights: TT_FP32 (all
 * fp32) or TT_BF16 (bf16 storage, fp32 arithmetic), and in the calls over
 * lists of logits TT_FP16 as well.  Parameter gradients,
 * LayerNorm statistics, log-sum-exp values and losses are always fp32.
 * Scratch memory, where a call needs it, is bump-allocated from the context's
 * arena (reset the arena between calls to reclaim it); TT_ERR_ARENA_OOM if
 * it does not fit.  All matrices are row-major and contiguous.
 */
#ifndef TT_OPS_H
#define TT_OPS_H

#include "tt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* GEMM engine selection: 0 = automatic (tcgen05 tensor cores whenever the
 * operands allow: bf16, 16-byte aligned rows; else SIMT, and the two-CTA
 * pair form wherever the M-tile count allows), 1 = SIMT only, 2 = tensor
 * cores with one CTA per 128-row tile (no pair form).  Returns TT_ERR_ARG
 * for any other value. */
tt_status tt_ctx_set_gemm_backend(tt_ctx* ctx, int backend);

/* Limit of every bounded device-side wait of the tensor-core kernels
 * launched through this context, in SM clock cycles (clock64).  cycles <= 0
 * restores the default, 4e9 cycles (about 2 s).  A wait that runs out sets
 * the context's timeout flag and a code naming the wait; the kernel lets its
 * copies and MMAs already issued finish, frees its tensor memory and returns;
 * every kernel that sees the flag gives up at its next wait; and the next
 * call that synchronises (tt_ctx_sync, a step with a loss pointer) returns
 * TT_ERR_TIMEOUT with the code in tt_last_error.  tt_ctx_reset clears the
 * flag; the context is usable again.  Below 1e6 cycles the waits look at
 * the clock on every poll, so a wait that is not complete within a few
 * hundred cycles of its start runs out (the form used to exercise the
 * timeout path).  The pages' boundary reports failure by status codes
 * (microcrad page, 反向传播); this is how a device-side wait reports one. */
tt_status tt_ctx_set_wait_limit(tt_ctx* ctx, long long cycles);

/* Linear layer forward (tinytorch 三.3 MatMul with the [out, in] weight
 * layout of 八.5):  u = x W^T + b;  y = gelu(u) if gelu (tanh form, tinytorch
 * 三.4) else u;  y += residual if residual != NULL.
 *   x [M,K], W [N,K], b [N] or NULL, residual [M,N] or NULL, y [M,N];
 *   pre [M,N]: receives u when gelu != 0 (required then), else ignored. */
tt_status tt_op_linear_fwd(tt_ctx* ctx, tt_dtype dtype, const void* x, const void* W,
                           const void* b, const void* residual, void* y, void* pre,
                           int M, int K, int N, int gelu);

/* Input gradient of a linear layer (tinytorch 三.3: dA = dC B^T):
 *   dx = dy W, times gelu'(pre) elementwise if pre != NULL (the gradient is
 *   then taken through the GELU that produced this layer's input from pre);
 *   accumulate != 0 adds into dx instead of overwriting.
 *   dy [M,N], W [N,K], pre [M,K] or NULL, dx [M,K]. */
tt_status tt_op_linear_bwd_dx(tt_ctx* ctx, tt_dtype dtype, const void* dy, const void* W,
                              const void* pre, void* dx, int M, int K, int N, int accumulate);

/* Weight and bias gradients (tinytorch 三.3: dB = A^T dC), fp32, overwritten:
 *   dW[N,K] = dy^T x,  db[N] = column sums of dy (db may be NULL).
 *   Deterministic: fixed split of the token dimension and fixed-order sums. */
tt_status tt_op_linear_bwd_dw(tt_ctx* ctx, tt_dtype dtype, const void* dy, const void* x,
                              float* dW, float* db, int M, int K, int N);

/* Causal self-attention forward (Forge page, 最硬的一关: scores scaled by
 * 1/sqrt(d_k), future masked with -inf).  qkv [B*T, 3C] with columns
 * [q | k | v] each [H, C/H]; y [B*T, C]; lse [B, H, T] fp32 receives the
 * log-sum-exp of each score row (saved for the backward). */
tt_status tt_op_attention_fwd(tt_ctx* ctx, tt_dtype dtype, const void* qkv, void* y,
                              float* lse, int B, int T, int C, int H);

/* Attention backward: dqkv [B*T, 3C] is overwritten.  Needs the forward's
 * y and lse; probabilities are recomputed, no T x T matrix is stored. */
tt_status tt_op_attention_bwd(tt_ctx* ctx, tt_dtype dtype, const void* qkv, const void* y,
                              const float* lse, const void* dy, void* dqkv,
                              int B, int T, int C, int H);

/* LayerNorm forward over the last dimension (biased variance, eps = 1e-5):
 *   y = (x - mean) * rstd * w + b;  mean, rstd [M] fp32. */
tt_status tt_op_layernorm_fwd(tt_ctx* ctx, tt_dtype dtype, const void* x, const void* w,
                              const void* b, void* y, float* mean, float* rstd, int M, int C);

/* LayerNorm backward: dx (+)= rstd (g - mean(g) - xhat mean(g xhat)), g = dy w;
 * dw = sum_rows dy xhat, db = sum_rows dy (fp32, overwritten, deterministic). */
tt_status tt_op_layernorm_bwd(tt_ctx* ctx, tt_dtype dtype, const void* x, const void* w,
                              const float* mean, const float* rstd, const void* dy, void* dx,
                              float* dw, float* db, int M, int C, int accumulate);

/* Fused log-softmax cross entropy, forward and backward in one pass over the
 * logits (tinytorch 三.5, Forge 核心组件清单).  logits [M, ld] (ld >= V; the
 * columns V..ld-1 are padding and are masked out) are REPLACED by
 *   dlogits = (softmax(z) - onehot(target)) * dscale      (pad columns: 0)
 * row_loss [M] receives log-sum-exp - z[target]; mean_loss[0] receives the
 * mean over the M rows (deterministic fixed-order sum).  dscale is usually 1/M. */
tt_status tt_op_xent(tt_ctx* ctx, tt_dtype dtype, void* logits, const int32_t* targets,
                     float* row_loss, float* mean_loss, int M, int V, int ld, float dscale);

/* Token + position embedding: x[b*T+t] = wte[tokens[b*T+t]] + wpe[t]. */
tt_status tt_op_embed_fwd(tt_ctx* ctx, tt_dtype dtype, const void* wte, const void* wpe,
                          const int32_t* tokens, void* x, int B, int T, int C, int V);

/* Embedding backward, deterministic (no floating-point atomics):
 *   dwte[v] += sum of dx rows whose token is v, in increasing position order
 *   (dwte is ACCUMULATED into, so that a tied LM-head gradient written first
 *   is kept); dwpe[t] = sum_b dx[b*T+t] for t < T and 0 for T <= t < maxT. */
tt_status tt_op_embed_bwd(tt_ctx* ctx, tt_dtype dtype, const void* dx, const int32_t* tokens,
                          float* dwte, float* dwpe, int B, int T, int C, int V, int maxT);

/* ------------------------------------------------------ lists over the logits
 * Operators on the LM head's logits that deal in lists of columns: the top
 * logits of a row, distillation from a teacher's list of them, and the
 * selection and reordering steps of a beam search.  They take TT_FP32,
 * TT_BF16 and TT_FP16 storage; lists, statistics, losses and scores are fp32.
 * Rows are ld elements apart, the columns V..ld-1 are padding that no result
 * depends on; neither ld nor the pointers need more than the element's
 * alignment, 4 bytes for lists, indices, scores and losses (without it:
 * TT_ERR_ARG).  They can be recorded (tt_graph.h); a
 * recorded call keeps its scratch until the reset.  The context's device has
 * to be the current one (else TT_ERR_STATE).  The pages have no counterpart to these calls: they extend the
 * fused cross entropy (tinytorch 三.5) and the greedy choice (八.3). */

#define TT_TOP_MAX 128  /* longest list of a row */
#define TT_BEAM_MAX 32  /* most beams of a sequence */
#define TT_TOP_SCRATCH_BYTES (4u << 20) /* most arena scratch of tt_op_top_logits */
#define TT_ROW_BYTES_MAX 1600000  /* most bytes of the V logits of a row (few rows are held on chip) */

/* The k largest logits of each row, in descending order, equal ones by
 * ascending column (-0 equals +0):
 *   vals [M, k] fp32, idx [M, k];  lse [M] fp32 or NULL: log sum_v exp(z_v / tau)
 * over the V columns.  1 <= k <= min(V, TT_TOP_MAX), tau > 0 (log2(e) / tau within fp32).  A NaN logit
 * stands in the list as -inf and makes the row's lse NaN; a row of -inf has
 * lse = -inf, one with +inf has lse = +inf.  Scratch from the arena where
 * there are few rows: at most TT_TOP_SCRATCH_BYTES. */
tt_status tt_op_top_logits(tt_ctx* ctx, tt_dtype dtype, const void* logits, float* vals, int32_t* idx, float* lse,
                           int M, int V, int ld, int k, float tau);

/* Distillation from a teacher's top logits, loss and gradient in one call.
 * The teacher's list of row r: logits t_vals [M, k] at the columns t_idx
 * [M, k]; an index of -1 is an unused entry.  With q = softmax(z / tau):
 *   t_lse == NULL:  p_j = softmax of t_j / tau over the list's entries,
 *     KL = sum_j p_j (ln p_j - ln q_ij)
 *   t_lse [M] (the teacher's log sum exp(t / tau) over its whole vocabulary,
 *   as tt_op_top_logits gives it):  p_j = exp(t_j / tau - t_lse), and the
 *   teacher's remaining mass p_r = max(0, 1 - sum_j p_j) is compared with the
 *   student's mass off the list, q_r:
 *     KL = sum_j p_j (ln p_j - ln q_ij) + p_r (ln p_r - ln q_r)
 *   (the last term is left out where q_r is below e^-700: no column off the list,
 *   or all of them masked)
 *   row_loss[r] = alpha tau^2 KL + (1 - alpha) (log sum exp(z) - z[target_r])
 *   dlogits = d row_loss / d z * dscale, pad columns 0
 * mean_loss (may be NULL) receives the mean over the M rows; dscale is
 * usually 1/M.  dlogits [M, ld] may be logits itself (the call is then in
 * place, as tt_op_xent) or NULL (loss only); any other overlap is not
 * allowed.  A row whose entries are all unused has no KL term; a target of -1
 * means that the row has no cross entropy term (targets may be NULL when
 * alpha is 1).  A row with neither has loss 0 and gradient 0, whatever its
 * logits hold.  A target or index outside these ranges, or an index that a row
 * lists twice, raises the bad token flag (tt_ctx_sync: TT_ERR_ARG); what the
 * row then receives is undefined.  0 <= alpha <= 1, tau > 0 (tau^2 and log2(e) / tau within fp32),
 * 1 <= k <= min(V, TT_TOP_MAX).
 * Deterministic. */
tt_status tt_op_distill(tt_ctx* ctx, tt_dtype dtype, const void* logits, const float* t_vals, const int32_t* t_idx,
                        const float* t_lse, const int32_t* targets, void* dlogits, float* row_loss,
                        float* mean_loss, int M, int V, int ld, int k, float alpha, float tau, float dscale);

/* One selection step of a beam search.  logits [B * K, ld]: row b K + j is
 * beam j of sequence b; scores [B, K] are the beams' cumulative log
 * probabilities (finite, or -inf for a slot that holds no hypothesis).  The n
 * best of the K V candidates
 *   scores[b, j] + z_v - log sum exp(z)
 * of each sequence, best first, equal ones by ascending j V + v:
 *   parent [B, n] (j), token [B, n] (v), out_scores [B, n];
 *   out_done [B, n] or NULL: 1 where the parent was done or token == eos.
 * done [B, K] or NULL: a beam with done != 0 has the one candidate eos at its
 * unchanged score (its logits are not read); the others count as -inf.  eos:
 * the end token, or -1 for none (done must then be NULL).  Candidates are
 * compared in 64 bits; within a beam they are ordered by logit.  Beams of equal
 * score with the same n best tokens and logits count as equal, and their
 * candidates tie, where their log-sum-exps differ by no more than 1e-5 (what
 * fp32 sums can differ by with the place of a row in memory).  A beam whose
 * logits hold NaN or +inf raises the non-finite flag (tt_ctx_sync:
 * TT_ERR_NONFINITE); it, a beam whose logits are all -inf and one whose score
 * is not finite have candidates of -inf only.  1 <= K <= TT_BEAM_MAX,
 * 1 <= n <= min(2 TT_BEAM_MAX, K V).  out_scores and out_done may be scores
 * and done when n == K.  Scratch from the arena: 8 B K (n + 1) bytes, times
 * the parts that few rows are cut into; at most TT_TOP_SCRATCH_BYTES more. */
tt_status tt_op_beam_select(tt_ctx* ctx, tt_dtype dtype, const void* logits, const float* scores,
                            const int32_t* done, int32_t* parent, int32_t* token, float* out_scores,
                            int32_t* out_done, int B, int K, int V, int ld, int n, int eos);

/* Reorder per-beam state in place after a selection step: in each of the N
 * blocks (for example a layer's cache) of B K rows of row_bytes bytes, the
 * bytes [first, first + count) of row b K + j become those that row
 * b K + parents[b, j] held before the call.  parents [B, K] in [0, K): any
 * mapping; a value out of range raises the bad token flag and its row stays.
 * Rows that are their own parent are not touched.  1 <= K <= TT_BEAM_MAX. */
tt_status tt_op_beam_reorder(tt_ctx* ctx, void* state, const int32_t* parents, int N, int B, int K,
                             size_t row_bytes, size_t first, size_t count);

/* ------------------------------------------------------ allocation-free call
 * The pages have no counterpart to this entry point.  It serves callers of
 * this library that cannot allocate device memory: a program whose GPU memory
 * is owned by another allocator (for example a framework's caching allocator
 * or a server that budgets all memory when it starts) must not have a library
 * call cudaMalloc behind its back, and such a caller cannot create a tt_ctx
 * either, because a context's arena is one cudaMalloc.
 *
 * tt_linear_bwd_dw_noalloc computes the same weight and bias gradients as
 * tt_op_linear_bwd_dw in bf16 mode (tensor cores, deterministic split-K):
 *   dW[N,K] = dy^T x (fp32, overwritten),  db[N] = column sums of dy (fp32,
 *   overwritten; db may be NULL),  dy [M,N] and x [M,K] bf16 row-major,
 *   16-byte aligned, N and K multiples of 8.
 * It takes a stream (a cudaStream_t; NULL = legacy default stream) instead
 * of a context and allocates nothing -- no cudaMalloc, no cudaFree, no
 * allocating library routine.  Its scratch is one fixed array of
 * TT_NOALLOC_SCRATCH_BYTES (32 MiB + 256 B) of device memory inside this
 * library, held by every GPU that loads the library until the process exits:
 * 256 B of device flags, TT_NOALLOC_SPLIT_FLOATS floats of split-K partial
 * sums (always enough on GPUs with up to 192 SMs) and TT_NOALLOC_BIAS_FLOATS
 * floats of bias partial sums.
 * Returns TT_ERR_ARG for a NULL pointer, a non-positive size, operands the
 * tensor-core path cannot take, or when db != NULL and the bias partial sums,
 * ceil(M / 256) * N floats, exceed TT_NOALLOC_BIAS_FLOATS (for M = 32768 that
 * allows N <= 16384); TT_ERR_CUDA if a CUDA call fails.  It returns before the
 * GPU finishes; a device-side wait that times out leaves dW undefined and is
 * not reported by this call.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, once per device, with that device current); make
 * that first call before any stream capture begins.  Every call shares the
 * one array and it keeps the last call's contents: nothing in it needs to
 * start at zero except the flags, which each call clears on its stream, since
 * every scratch element a call reads is written earlier in that call.  Calls
 * that overlap on the GPU (on different streams, or from threads without
 * ordering between them) race on the array: issue them on one stream. */
#define TT_NOALLOC_SPLIT_FLOATS 6291456u
#define TT_NOALLOC_BIAS_FLOATS 2097152u
#define TT_NOALLOC_SCRATCH_BYTES (256u + 4u * (TT_NOALLOC_SPLIT_FLOATS + TT_NOALLOC_BIAS_FLOATS))
tt_status tt_linear_bwd_dw_noalloc(void* stream, const void* dy, const void* x, float* dW,
                                   float* db, int M, int K, int N);

#ifdef __cplusplus
}
#endif
#endif /* TT_OPS_H */
