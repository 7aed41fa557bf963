/*
 * gpipe_ops.h - kernel-level entry points of libgpipe.
 *
 * Each call enqueues the kernel(s) of one operation of the GPipe step on
 * `stream` (a cudaStream_t passed as void*; NULL = legacy default stream) and
 * returns 0 or a negative GPIPE_ERR_* code from gpipe.h without launching on
 * invalid arguments.  All pointers are caller-owned device addresses unless
 * stated; nothing is allocated or freed.  They exist so that every kernel the
 * step uses can be checked on its own; gpipe_step calls the same launchers.
 * The operations are the pieces of the step of "GPipe technical review"
 * (zzz0906.github.io), section "Pipeline flow": the layers' forward and
 * backward, the loss, the gradient accumulation and the RMSProp update
 * ("Preliminaries 2: the memory wall").
 *
 * dtype: 0 = fp32 operands/activations, 1 = bf16 operands/activations (fp32
 * accumulation and fp32 statistics in both cases).
 */
#ifndef GPIPE_OPS_H
#define GPIPE_OPS_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  GPIPE_EPI_STORE = 0,     /* C = acc (+ bias[n]) (+ resid[m,n])                  */
  GPIPE_EPI_BIAS_GELU = 1, /* C = z = acc + bias[n];  C2 = GELU(z)  (exact erf)    */
  GPIPE_EPI_GELU_BWD = 2,  /* C = acc * GELU'(aux[m,n])                              */
  GPIPE_EPI_ACC_F32 = 3,   /* C (fp32) += acc                                        */
  GPIPE_EPI_STORE_F32 = 4, /* C (fp32) = acc                                         */
  GPIPE_EPI_RESID_F32 = 5  /* C (fp32) = (acc + bias[n]) + resid (fp32)[m,n]         */
};

/* C[m,n] = epilogue( sum_k A(m,k) B(n,k) ), 0 <= m < M, 0 <= n < N.
 * A(m,k) = A[m*lda + k] when a_kmajor, else A[k*lda + m];
 * B(n,k) = B[n*ldb + k] when b_kmajor, else B[k*ldb + n].
 * So x W^T (W [out,in]) is (a_kmajor=1, b_kmajor=1); dY W is (1, 0); the weight
 * gradient dY^T X is (0, 0).  C, C2, resid and aux are row-major with leading
 * dimension ldc (C, C2), ldr (resid), ldaux (aux); element type = dtype except
 * for the fp32 epilogues.  bias is fp32 [N] (read) or NULL for the forward
 * epilogues; for GPIPE_EPI_ACC_F32 a non-NULL bias is an fp32 [M] accumulator
 * that receives += sum_k A(m,k) (the bias gradient that goes with a weight
 * gradient dY^T X, computed by the same launch).  resid may be NULL.
 * dtype 1 runs the tcgen05/TMEM tensor-core kernel fed by TMA and needs every
 * leading dimension a multiple of 8 elements and 16-byte aligned bases; it is
 * built for (1,1) with STORE, BIAS_GELU, STORE_F32, ACC_F32, RESID_F32 (resid
 * required, fp32 like C); (1,0) with STORE,
 * GELU_BWD, ACC_F32; (0,0) with STORE, ACC_F32 (others: GPIPE_ERR_UNSUPPORTED).
 * dtype 0 runs an fp32 FFMA kernel (any layout and epilogue).
 * Requires M, N, K >= 1. */
int gpipe_op_gemm(int dtype, int M, int N, int K,
                  const void* A, int64_t lda, int a_kmajor,
                  const void* B, int64_t ldb, int b_kmajor,
                  int epi, void* C, int64_t ldc,
                  float* bias, const void* resid, int64_t ldr,
                  void* C2, const void* aux, int64_t ldaux, void* stream);

/* SM share of the GEMMs this host thread launches through gpipe_op_gemm from
 * now on: sms > 0 sizes their grids (and so the tile width and kernel) as the
 * step does for a GEMM given that many SMs; 0 (the default) gives each the
 * whole GPU.  Returns 0, or GPIPE_ERR_INVALID_ARG for sms < 0. */
int gpipe_op_gemm_set_sm_share(int sms);

/* Bytes of fp32 scratch the two-stage column reductions below need. */
size_t gpipe_op_scratch_bytes(int rows, int cols);

/* LayerNorm over rows of width d (eps 1e-5, biased variance):
 * y = (x - mean) * rstd * g + b; mean and rstd (fp32 [rows]) are saved.
 * d must be a multiple of 8 and at most 1024 (GPIPE_ERR_INVALID_ARG otherwise). */
int gpipe_op_layernorm_fwd(int dtype, int rows, int d, const void* x, const float* g,
                           const float* b, void* y, float* mean, float* rstd, void* stream);

/* LayerNorm backward: dx = rstd (g dy - mean(g dy) - xhat mean(g dy xhat)) + dres
 * (dres may be NULL); dg_acc += sum_rows dy xhat and db_acc += sum_rows dy,
 * accumulated in a fixed order (two stages through `scratch`, of
 * gpipe_op_scratch_bytes(rows, 2*d) bytes). */
int gpipe_op_layernorm_bwd(int dtype, int rows, int d, const void* dy, const void* x,
                           const float* mean, const float* rstd, const float* g,
                           const void* dres, void* dx, float* dg_acc, float* db_acc,
                           float* scratch, void* stream);

/* The same LayerNorm backward for callers that cannot allocate device memory
 * when they call it: for instance a plugin inside a host framework that owns
 * all device memory through its own pool, or a latency-critical path that must
 * never enter the CUDA allocator.  The paper has no counterpart; this is a
 * convenience of this library.  Instead of a caller `scratch` buffer it uses a
 * fixed array of 2^20 floats (4 MiB) inside the library's device image, which
 * every GPU that loads the library keeps until the process exits; it calls no
 * allocation routine.  Limit: ceil(rows / 8) * 2 * d <= 2^20 (for d = 1024,
 * rows <= 4096); larger sizes return GPIPE_ERR_INVALID_ARG with a message.
 * Every call looks up the array's device address in the current context (no
 * allocation and no stream work), so a context re-created after
 * cudaDeviceReset is served correctly; the first lookup on a device may load
 * the library's device image, so make the first call before any stream
 * capture.  All calls
 * share the one array: every partial sum the call reads is written by the
 * same call, so nothing needs clearing, but calls that overlap on the GPU (on
 * different streams, or from different threads) race on it. */
int gpipe_op_layernorm_bwd_noalloc(int dtype, int rows, int d, const void* dy, const void* x,
                                   const float* mean, const float* rstd, const float* g,
                                   const void* dres, void* dx, float* dg_acc, float* db_acc,
                                   void* stream);

/* out_acc[c] += sum_r y[r*ldy + c] in a fixed order (bias gradients); scratch
 * of gpipe_op_scratch_bytes(rows, cols) bytes. cols % 8 == 0, ldy % 8 == 0. */
int gpipe_op_colsum(int dtype, int rows, int cols, const void* y, int64_t ldy,
                    float* out_acc, float* scratch, void* stream);

/* Causal multi-head attention forward, bf16, head width 64, scale 1/8, on
 * the tcgen05 tensor cores (S and O accumulate in tensor memory).
 * qkv [nseq*seq, 3*heads*64] (query | key | value column blocks), output
 * o [nseq*seq, heads*64], lse [nseq*seq, heads] fp32 natural-log
 * log-sum-exp of the scaled scores.  seq % 64 == 0, nseq * seq <= 2^30. */
int gpipe_op_attention_fwd(int nseq, int seq, int heads, const void* qkv, void* o,
                           float* lse, void* stream);

/* Backward: dqkv [nseq*seq, 3*heads*64] gets dQ | dK | dV.  dvec is fp32
 * [nseq*seq, heads]: rowsum(dO o O), written first by a small kernel, then
 * read by one launch whose dQ blocks and dK/dV blocks run side by side; no
 * atomics, so results are bit-reproducible.  nseq <= 32767. */
int gpipe_op_attention_bwd(int nseq, int seq, int heads, const void* qkv, const void* o,
                           const void* dout, const float* lse, float* dvec, void* dqkv,
                           void* stream);

/* Causal attention with a sliding window, sinks and a learned relative position
 * bias, bf16, head width 64, scale 1/8.  Query i of a sequence sees key j when
 * j <= i and (i - j < window or j < sinks); its score is
 *   q_i . k_j / 8 + table[bucket(i - j), head].
 * qkv [nseq*seq, (heads + 2 kv_heads)*64] (query | key | value column blocks;
 * heads / kv_heads consecutive query heads share a key/value head), o
 * [nseq*seq, heads*64], lse fp32 [nseq*seq, heads] (natural log).
 *   window    >= 1: keys a query sees, itself included (>= seq: every earlier one).
 *   sinks     0..64: first tokens of a sequence that stay visible to all of it.
 *   lens      int32 [nseq] on the device, or NULL for full sequences: tokens of
 *             each sequence (clamped to [0, seq]).  The rows behind them are
 *             padding: nothing of them is used (they may hold anything, NaN
 *             included), and their o and dqkv rows are written as zeros, their
 *             lse as -inf.
 *   table     fp32 [num_buckets, heads], or NULL with num_buckets 0.  An entry
 *             of -1e30 or less (-inf, the lowest finite value) hides its bucket.
 *             Other finite entries may have any size: only how far they are from
 *             the largest one that a query sees is rounded (the lse, which holds
 *             that one, has its own 24 bits).  Heads with entries above 256 in
 *             size take a slower path.
 *             A query that sees nothing has o = 0, lse = -inf, zero gradients.
 *   bucket(d) d itself below e = num_buckets / 2, then e + floor(log(d / e) /
 *             log(max_distance / e) * (num_buckets - e)), at most
 *             num_buckets - 1, decided in exact arithmetic
 *             (gpipe_op_position_bucket_starts); 2 <= num_buckets <= 64,
 *             num_buckets / 2 < max_distance <= 4096.
 * Any seq >= 1; nseq * seq <= 2^30.  Cost grows with the visible pairs.  Outputs
 * that overlap each other or an input are rejected. */
int gpipe_op_attention_window_fwd(int nseq, int seq, int heads, int kv_heads, int window, int sinks,
                                  const int32_t* lens, const float* table, int num_buckets,
                                  int max_distance, const void* qkv, void* o, float* lse, void* stream);

/* Its backward pass: dqkv gets dQ | dK | dV (a shared key/value head's summed
 * over its query heads); dtable_acc fp32 [num_buckets, heads] (or NULL) gets
 * += sum of dS over the pairs of each bucket.  o and lse are the forward's, with
 * the same lens and table.  scratch: gpipe_op_attention_window_scratch_bytes,
 * 256-byte aligned, written before it is read (calls that may overlap on the
 * GPU, captured ones included, need one each, and a dtable_acc each: it is read,
 * added to and written back).  dqkv, dtable_acc and scratch may overlap neither
 * each other nor the inputs (but dtable_acc the table: the gradient is then added
 * to it).  Query heads that share a key/value head follow each other in its dK and
 * dV, so a large group over a short sequence takes longer than its pairs alone would.
 * No atomics: results are bit-reproducible. */
int gpipe_op_attention_window_bwd(int nseq, int seq, int heads, int kv_heads, int window, int sinks,
                                  const int32_t* lens, const float* table, int num_buckets,
                                  int max_distance, const void* qkv, const void* o, const void* dout,
                                  const float* lse, void* dqkv, float* dtable_acc, void* scratch,
                                  void* stream);

/* Bytes of scratch the backward pass needs (num_buckets 0: no table gradient);
 * 0 for sizes that it would reject. */
size_t gpipe_op_attention_window_scratch_bytes(int nseq, int seq, int heads, int window, int sinks,
                                               int num_buckets);

/* starts[b] = the smallest distance of bucket b, or of the next one that is not
 * empty (host memory, num_buckets values; no GPU work). */
int gpipe_op_position_bucket_starts(int num_buckets, int max_distance, int32_t* starts);

/* Next-token softmax cross-entropy on fp32 logits [rows, vocab].
 * Row r is token row0 + r of the mini-batch (tokens [N*seq] int32); its target
 * is tokens[row0 + r + 1] unless (row0 + r) % seq == seq - 1 (no target).
 * loss_rows[r] = (lse - z_target) * inv_count (0 without target).
 * want_grad: writes dz = (softmax - onehot) * inv_count as bf16 IN PLACE over
 * the logits, row r at bf16 offset r * 2 * vocab (so the gradient matrix has
 * leading dimension 2*vocab bf16 elements).  vocab % 4 == 0.  A target id
 * outside [0, vocab) is treated as "no target" and sets the device error flag. */
int gpipe_op_cross_entropy(int rows, int vocab, int seq, const int32_t* tokens, int row0,
                           float inv_count, float* logits, float* loss_rows, int want_grad,
                           void* stream);

/* The same with logit clipping ("GPipe technical review", "Training
 * stability": logits above a threshold are clipped before the softmax).
 * clip > 0: the softmax and the target term see min(max(z, -clip), clip), and
 * dz is zero where |z| > clip (the clamp's derivative; a NaN logit stays NaN in
 * the loss).  clip = 0: no clipping, exactly gpipe_op_cross_entropy.  A
 * negative or NaN clip is rejected (GPIPE_ERR_INVALID_ARG). */
int gpipe_op_cross_entropy_clip(int rows, int vocab, int seq, const int32_t* tokens, int row0,
                                float inv_count, float clip, float* logits, float* loss_rows,
                                int want_grad, void* stream);

/* Distillation from a teacher's top logits, with the hard-label cross-entropy
 * of gpipe_op_cross_entropy beside it.  Per row of student logits z (dtype
 * elements, leading dimension ld >= vocab), teacher logits t_k = top_logit[r,k]
 * (fp32 [rows, topk]) at tokens i_k = top_idx[r,k] (int32 [rows, topk]; i_k < 0:
 * an empty slot, whose logit is not used), p = softmax(t / temperature) over the
 * filled slots and q_T = softmax(z / T):
 *   loss_rows[r] = kd_scale T^2 sum_k p_k (log p_k - log q_T[i_k])
 *                + ce_scale (-log q_1[target])
 *   dz           = kd_scale T (q_T - sum_k p_k onehot(i_k))
 *                + ce_scale (q_1 - onehot(target))
 * (T = temperature >= 2^-126; kd_scale T^2 finite).  The target of row r is that of
 * gpipe_op_cross_entropy: tokens[row0 + r + 1] unless (row0 + r) % seq ==
 * seq - 1; tokens is not read when ce_scale = 0 and may then be NULL.  A row
 * whose slots are all empty (or whose filled teacher logits are all -inf) has
 * no teacher term, a row without a target no label term.  Slots that name the
 * same token count as separate terms of the sum.  A token id of vocab or more
 * is treated as an empty slot, a target outside [0, vocab) as no target; both
 * set the device error flag.  (A padded batch with labels: one call a sequence, with
 * seq and rows its length and row0 0.)
 * dz is bf16 [rows, vocab] with leading dimension lddz, or NULL for the loss
 * alone.  It may be the logits themselves (same address, and the same row
 * stride in bytes: lddz = ld for bf16, 2 ld for fp32); any other overlap of dz
 * or loss_rows with an input or each other is rejected.  Elements of a row behind the vocab-th are neither read nor written.
 * 1 <= topk <= 256, 1 <= rows <= 2^27, 1 <= vocab <= 2^30 (any; rows that start on
 * 16-byte boundaries take wide loads).  No atomics: results are bit-reproducible. */
int gpipe_op_distill(int dtype, int rows, int vocab, const void* logits, int64_t ld, int topk,
                     const int32_t* top_idx, const float* top_logit, float temperature,
                     float kd_scale, int seq, const int32_t* tokens, int row0, float ce_scale,
                     float* loss_rows, void* dz, int64_t lddz, void* stream);

/* Next-token softmax cross-entropy of the tied head without its logits, which are
 * never held: per row of hidden states h (bf16 [rows, d], leading dimension ldh)
 * over the table emb (bf16 [vocab, d]),
 *   z = h E^T in fp32, limited to [-clip, clip] where clip > 0, p = softmax(z),
 *   loss_rows[r] = w_r inv_count (-log p[target])
 *   g    = w_r (p - onehot(target)), 0 where |z| > clip > 0, rounded to bf16 (what the
 *          target's column loses by it is given back to dh, and to demb of up to 64 rows)
 *   dh   = inv_count g E        bf16 [rows, d], leading dimension lddh, or NULL
 *   demb = inv_count g^T h      [vocab, d], or NULL: demb_dtype 0 an fp32
 *                               accumulator that receives it (+=), 1 bf16, written
 * (dh and demb NULL: the loss alone.)  The target of row r is that of
 * gpipe_op_cross_entropy, tokens[row0 + r + 1] unless (row0 + r) % seq == seq - 1;
 * a negative id means that the row has none, one of vocab or more too, and sets
 * the device error flag.  w_r = row_weight[r] (fp32 [rows]; NULL: 1).  A row
 * without a target or of weight 0 has loss 0, a zero row of dh and no part in demb;
 * its h is not used and may hold anything (NaN included).  Logits of other rows keep
 * their differences up to 2^24 in size.  A NaN among a row's logits makes its loss, dh
 * and all of demb NaN.  Without clip so does a logit of +inf; one of -inf counts as
 * p = 0, and as a loss of +inf where it is the target's.  With clip > 0 an infinite
 * logit counts as the limit, without a gradient.  (An infinity of h or E shows in its
 * column of demb or dh besides, as 0 times it.)
 * piece     columns of the vocabulary that a launch works on (rounded up to a multiple
 *           of 256): more scratch and fewer launches with more of them.  g exists for
 *           one piece at a time, for two where the vocabulary takes several.  0: as
 *           many as give g 256 MB in all, but 2048 at least (so more than 32768 rows
 *           over several pieces have two buffers of 4096 bytes a row).  Results
 *           depend on it by their roundings, and where the first piece's p passes
 *           through fp16 (d >= 768, or less where the rows do not fill tiles of 256):
 *           there those below 2^-38 of the largest of 128 columns may count as 0.
 * scratch   gpipe_op_head_loss_scratch_bytes (grads: 1 dh, 2 demb, 3 both), 256-byte
 *           aligned, written before it is read (calls that may overlap on the GPU,
 *           captured ones included, need one each, and outputs each).
 * 1 <= rows <= 2^24, 1 <= vocab <= 2^27 (and at most 2^26 tiles of 256 x 256),
 * d <= 2^16 and the leading dimensions multiples of 8, 16-byte aligned bases.  Outputs
 * and scratch may overlap neither each other nor an input.  Every element receives its
 * additions one launch after the other: results are bit-reproducible. */
int gpipe_op_head_loss(int rows, int d, int vocab, const void* h, int64_t ldh, const void* emb_bf16, int seq,
                       const int32_t* tokens, int row0, const float* row_weight, float inv_count, float clip,
                       int piece, float* loss_rows, void* dh, int64_t lddh, int demb_dtype, void* demb, void* scratch,
                       void* stream);

/* Bytes of scratch; 0 for sizes that the call would reject. */
size_t gpipe_op_head_loss_scratch_bytes(int rows, int d, int vocab, int piece, int grads);

/* MSE rows: loss_rows[r] = sum_j (y - t)^2 * inv_count; dy = 2 (y - t) inv_count. */
int gpipe_op_mse(int rows, int d, const float* y, const float* t, float inv_count,
                 float* loss_rows, float* dy, void* stream);

/* x[r,:] = emb[tokens[r],:] (bf16 rows of width d, d % 8 == 0, vocab rows).
 * A token id outside [0, vocab) gives a zero row and sets the device error
 * flag (read by gpipe_debug_counters) instead of reading out of bounds. */
int gpipe_op_embedding_fwd(int rows, int d, int vocab, const int32_t* tokens, const void* emb_bf16,
                           void* x, void* stream);

/* demb[tokens[r],:] += dx[r,:] (fp32 accumulator, bf16 dx).  Deterministic: each
 * embedding row is owned by one CTA, which adds its tokens in ascending r. */
int gpipe_op_embedding_bwd(int rows, int d, int vocab, const int32_t* tokens,
                           const void* dx_bf16, float* demb, void* stream);

/* x[r,:] = scale emb[tokens[r],:] (bf16 table [vocab, d]), x of dtype elements with
 * leading dimension ldx, rounded once from fp32 (bf16: and once from there).  A
 * negative token is padding: a zero row.  A token id of vocab or more gives a zero
 * row too and sets the device error flag.  1 <= rows <= 2^27, d and ldx multiples
 * of 8, 16-byte aligned bases; x may not overlap an input. */
int gpipe_op_embedding_scaled_fwd(int dtype, int rows, int d, int vocab, const int32_t* tokens, const void* emb_bf16,
                                  float scale, void* x, int64_t ldx, void* stream);

/* Its gradient: demb[tokens[r],:] += scale dx[r,:] (fp32 accumulator, dx of dtype
 * elements with leading dimension lddx), so that many CTAs sum a frequent token's rows.
 * A token's rows are added in ascending r, in parts that are then added in order; the
 * sum is scaled, rounded and added to demb.  The parts: up to 256 rows, quarters of the
 * token's; more rows are sorted by token, stably, and cut into runs of 8 sorted rows (up
 * to 24576) or 64, and a token of more than 16 runs has their sums added in eighths
 * first.  Padding and ids out of range as above, with no gradient.
 * (gpipe_op_embedding_bwd adds one row after the other and needs no scratch; it is
 * quicker for up to some 2000 rows whose tokens hardly repeat.)
 * scratch: gpipe_op_embedding_sorted_bwd_scratch_bytes, 256-byte aligned, written
 * before it is read (calls that may overlap on the GPU, captured ones included, need
 * one each, and a demb each).  demb and scratch may overlap neither each other nor
 * the inputs.  Every element of demb receives at most one addition, by a reduction of
 * the GPU's, which has subnormal operands and results as zero; so results are
 * bit-reproducible. */
int gpipe_op_embedding_sorted_bwd(int dtype, int rows, int d, int vocab, const int32_t* tokens, const void* dx,
                                  int64_t lddx, float scale, float* demb, void* scratch, void* stream);

/* Bytes of scratch; 0 for sizes that the call would reject. */
size_t gpipe_op_embedding_sorted_bwd_scratch_bytes(int rows, int d, int vocab);

/* RMSProp over n parameters: v = decay v + (1-decay) g^2; w -= lr g/(sqrt(v)+eps);
 * w_bf16 (may be NULL) receives the round-to-nearest-even bf16 copy of w;
 * zero_grad != 0 sets g = 0 afterwards. */
int gpipe_op_rmsprop(size_t n, float* w, float* g, float* v, void* w_bf16, float lr,
                     float decay, float eps, int zero_grad, void* stream);

/* dst[i] = bf16(src[i]) (round to nearest even). */
int gpipe_op_cast_bf16(size_t n, const float* src, void* dst, void* stream);

/* Failure detection.  Every wait of the library's kernels on another part of
 * the GPU is bounded (2 s); one that gives up, or a kernel that meets an
 * invalid input it skips (a token id outside [0, vocab)), sets the device error
 * word of the current device: 1-4 a bounded wait (TMA producer, MMA issuer,
 * epilogue, exit drain), 5 an invalid token id, 6 this probe, 7 a kernel whose
 * shared memory was less aligned than its swizzled tiles need (its work is
 * skipped).
 *   gpipe_op_wait_probe: launches one CTA whose bounded wait on an mbarrier
 *     that nothing completes gives up after the limit and sets code 6; the
 *     kernel returns normally and the context stays usable.
 *   gpipe_op_device_error: copies the word to *flag_out (synchronises
 *     `stream`); clear != 0 resets it to 0 afterwards. */
int gpipe_op_wait_probe(void* stream);
int gpipe_op_device_error(int* flag_out, int clear, void* stream);

/* The GELU arithmetic of the GEMM epilogues, in fp32 (for checking it):
 * gelu[i] = z Phi(z) and dgelu[i] = Phi(z) + z phi(z) for z = z_in[i] (exact-erf
 * GELU as the review's Transformer uses it; erf evaluated to within 1.5e-7, see
 * the kernels).  Either output may be NULL. */
int gpipe_op_gelu(size_t n, const float* z_in, float* gelu, float* dgelu, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* GPIPE_OPS_H */
