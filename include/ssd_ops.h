/*
 * libssd kernel-level entry points.
 *
 * Each call runs one kernel of the decoding hot path on caller-provided
 * DEVICE buffers, enqueued on `stream` (a cudaStream_t; NULL = legacy
 * default stream), and returns without waiting.  They exist so that each
 * kernel can be checked on its own against the CPU oracle with seeded
 * inputs; the context API in ssd.h runs the same kernels.
 *
 * Common rules: M (rows, i.e. token positions processed together) is
 * 1..16; weight matrices are bf16 in the packed layout of ssd_pack_weight
 * (shapes are given as those of the row-major matrix, R % 16 == 0 and
 * K % 32 == 0); pointers are 16-byte aligned.  Calls that need scratch memory take it
 * from the stream-ordered allocator (cudaMallocAsync) and free it on the
 * same stream.  Errors: SSD_ERR_INVALID_ARG for a bad size or pointer,
 * SSD_ERR_OOM, SSD_ERR_CUDA for a failed launch; the message is available
 * from ssd_ops_last_error().
 *
 * Every kernel's reduction order is fixed by the element's own position and
 * never depends on M or on the other rows: row m of a call with M rows is
 * bit-identical to the same row computed alone.  ssd_op_tree_attention is the
 * exception (see there).
 */
#ifndef SSD_OPS_H_
#define SSD_OPS_H_

#include <stdint.h>

#include "ssd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Per-row summary of a logits vector z (LM head epilogue). */
typedef struct {
  int32_t top1;   /* argmax z (lowest id on ties)                           */
  int32_t top2;   /* second-largest entry's id                              */
  int32_t sample; /* Gumbel-max sample of softmax(z / T) (T > 0), else top1 */
  int32_t pad;
  float z1;       /* z[top1]                                                */
  float z2;       /* z[top2]                                                */
  float lse;      /* log sum exp z                                          */
  float conf;     /* max softmax(z) = exp(z1 - lse)                         */
  float lse_t;    /* log sum exp (z / T) (T > 0), else lse                  */
  float pad2[3];
} ssd_row_stats;

/* y[m][r] = sum_k W[r][k] * act[m][k].  W bf16 [R][K]; act bf16 [M][K];
 * y fp32 [M][R].  The small-M weight-streaming GEMV of the decoder. */
ssd_status ssd_op_linear(const void* W, int32_t R, int32_t K, const void* act, int32_t M,
                         float* y, void* stream);

/* y = W bf16(rmsnorm(x) * gain): the norm-fused input of the QKV projection
 * and the LM head.  x fp32 [M][K]; gain fp32 [K]; y fp32 [M][R].  When M
 * rows of K do not fit the GEMV's per-CTA activation stage, a RMSNorm pass
 * first writes the bf16 rows (scratch) and the projection reads them; the
 * result is the same.  The same holds for ssd_op_swiglu and ssd_op_lm_head. */
ssd_status ssd_op_rmsnorm_linear(const void* W, int32_t R, int32_t K, const float* x,
                                 const float* gain, float eps, int32_t M, float* y, void* stream);

/* x += W act: o_proj / down_proj with the residual add fused.  x fp32
 * [M][R] (read and written); act bf16 [M][K]. */
ssd_status ssd_op_residual_linear(const void* W, int32_t R, int32_t K, const void* act, int32_t M,
                                  float* x, void* stream);

/* u = bf16(silu(Wg h) * (Wu h)) with h = bf16(rmsnorm(x) * gain).
 * Wg, Wu bf16 [F][K]; x fp32 [M][K]; u bf16 [M][F]. */
ssd_status ssd_op_swiglu(const void* Wg, const void* Wu, int32_t F, int32_t K, const float* x,
                         const float* gain, float eps, int32_t M, void* u, void* stream);

/* Decode / verify attention for M consecutive positions pos0..pos0+M-1.
 * qkv fp32 [M][(H + 2 Hkv) dh] holds the raw projections (q rows, k rows,
 * v rows, before RoPE).  The call applies rotate-half RoPE (base theta) to
 * q and k, stores bf16(k), bf16(v) into k_cache / v_cache ([Hkv][max_seq][dh]
 * bf16) at the M positions, and writes
 *   out[m][h dh ..] = bf16(softmax(q K^T / sqrt(dh), keys <= pos0+m) V)
 * (bf16 [M][H dh]).  Grouped-query: query head h reads K/V head h / (H/Hkv).
 * dh is 64 or 128; pos0 + M <= max_seq. */
ssd_status ssd_op_attention(const float* qkv, int32_t M, int32_t pos0, void* k_cache,
                            void* v_cache, int32_t max_seq, int32_t H, int32_t Hkv, int32_t dh,
                            float theta, void* out, void* stream);

/* Final RMSNorm + LM head with the fused row summary: z = W bf16(rmsnorm(x)
 * * gain) for each of the M rows (W bf16 [V][D], x fp32 [M][D]); writes
 * stats[m] (device) and, if logits is not NULL, z to logits (fp32 [M][V]).
 * At temperature > 0 the row summary includes a Gumbel-max sample drawn with
 * Philox4x32-10 counters (v/4, pos0 + m + 1, round, stream_id), key = seed. */
ssd_status ssd_op_lm_head(const void* W, int32_t V, int32_t D, const float* x, const float* gain,
                          float eps, int32_t M, float temperature, uint64_t seed, int32_t round,
                          int32_t stream_id, int32_t pos0, float* logits, ssd_row_stats* stats,
                          void* stream);

/* LayerSkip §3.3 acceptance at temperature T > 0 for one round.
 * P fp32 [d+1][V] verify logits, Q fp32 [d][V] draft logits, drafts int32 [d]
 * (all device).  Draft j is accepted when u_j < p_j(y_j) / q_j(y_j) with
 * p = softmax(P/T), q = softmax(Q/T) and u_j the Philox uniform at counter
 * (0, n + j, round, 1); on the first rejection a token is drawn from
 * norm(max(0, p_j - q_j)) (from p_j if that is empty), otherwise a bonus
 * from p_d, by Gumbel-max at counters (v/4, n + j, round, 2).
 * Writes emitted (device int32 [d+1]) and n_emitted (device int32 [1]). */
ssd_status ssd_op_accept_stochastic(const float* P, const float* Q, const int32_t* drafts,
                                    int32_t d, int32_t V, float temperature, uint64_t seed,
                                    int32_t round, int32_t n, int32_t* emitted,
                                    int32_t* n_emitted, void* stream);

/* Philox4x32-10 of the library: out[4i..4i+3] = philox(ctr[4i..4i+3], key).
 * ctr, out: device uint32 [4 count]. */
ssd_status ssd_op_philox(const uint32_t* ctr, int32_t count, uint64_t key, uint32_t* out,
                         void* stream);

/* Many-row projection on the tensor cores (the batched candidate-mask
 * scoring forward of SWIFT §4.1.2, where K candidates x N window positions
 * give hundreds of rows): for T >= 1 rows of act (bf16 [T][K]),
 *   epi 0 (store):  out fp32 [T][R] = W act
 *   epi 1 (resid):  out fp32 [*][R]: out[map[t]] += W act[t] (map: device
 *                   int32 [T] of distinct rows, NULL = identity; rows not
 *                   named stay as they are)
 *   epi 2 (swiglu): out bf16 [T][R] = bf16(silu(W act) * (W1 act)), W1 the
 *                   up matrix (same shape as W)
 *   epi 3 (argmax): out int32 [T] = argmax_r (W act)[r], lowest r on ties
 * W, W1 packed (ssd_pack_weight).  With epi | SSD_ROWS_ACT_PACKED, act is
 * already in the packed layout: ssd_pack_weight of the [T'][K] matrix, T'
 * = T rounded up to 16 (the rows beyond T are read and their results
 * dropped); otherwise the call packs a scratch copy first.  Every output
 * sums K in ascending 32-wide steps, whatever T.  This call has no limit of
 * 16 rows. */
#define SSD_ROWS_ACT_PACKED 16
ssd_status ssd_op_linear_rows(const void* W, const void* W1, int32_t R, int32_t K,
                              const void* act, int32_t T, int32_t epi, void* out,
                              const int32_t* map, void* stream);

/* Attention of candidate-mask scoring windows.  For each candidate k in
 * cand (device int32 [n_cand]) and window row i < N (query position
 * split + i), with q bf16 [n_cand N][H][dh] (RoPE applied, row ja N + i for
 * the ja-th candidate of the list):
 *   out[ja N + i][h dh ..] = bf16(softmax(q K^T / sqrt(dh)) V)
 * over the keys of the shared cache k_cache / v_cache ([Hkv][max_seq][dh]
 * bf16) at positions 0..split-1, then candidate k's own window keys
 * wk / wv (bf16 [w_rows][Hkv][dh], row k N + w) for w <= i; every k in cand
 * has k N + N <= w_rows.  split >= 1, split <= max_seq; dh 64 or 128. */
ssd_status ssd_op_score_attention(const void* q, const int32_t* cand, int32_t n_cand, int32_t N,
                                  int32_t split, const void* k_cache, const void* v_cache,
                                  int32_t max_seq, const void* wk, const void* wv, int32_t w_rows,
                                  int32_t H, int32_t Hkv, int32_t dh, void* out, void* stream);

/* ---- Decoding with a tree of drafts: attention of the tree over the cache,
 * eviction from the cache by accumulated attention weight, beam selection
 * and the reordering of the beams' caches.  These calls allocate nothing:
 * where a call needs scratch memory, the caller gives a workspace of device
 * memory (256-byte aligned, at least what the call's _workspace function
 * returns for the current device; fewer bytes are SSD_ERR_CAPACITY; 0 for
 * sizes that need none, or that the call refuses).  Its contents need no
 * initialisation and mean nothing afterwards; calls that may overlap on the GPU
 * need one each.  Each call can be captured into a CUDA graph.  Buffers overlap
 * only where a call says so.  Inputs that these calls read from device memory
 * (parents, done) may hold any values, with the meanings below. */

/* Attention of T drafted nodes over a cache of n_ctx rows.  1 <= T <= 1024,
 * n_ctx >= 0, n_ctx + T <= max_seq, pos0 >= 0; dh 64 or 128.
 * parents (device int32 [T]): parents[t] is the node that t follows,
 * 0 <= parents[t] < t, or -1 where t follows the context itself.  Any other
 * value makes t absent, and with it every node below it: padding rows.
 * qkv fp32 [T][(H + 2 Hkv) dh] holds the raw projections (q, k, v rows,
 * before RoPE; what ssd_op_linear_rows stores).  The call rotates q and k by
 * rotate-half RoPE (base theta) to position pos0 + depth(t), depth(t) = the
 * number of nodes above t, stores bf16(k), bf16(v) into row n_ctx + t of
 * k_cache / v_cache ([Hkv][max_seq][dh] bf16; zeros for an absent node), and
 * writes
 *   out[t][h dh ..] = bf16(softmax(q K^T / sqrt(dh)) V)      (bf16 [T][H dh])
 * over cache rows 0..n_ctx-1, the nodes above t, and t itself; query head h
 * reads K/V head h / (H/Hkv).  An absent node's row is zeros.  Keys that a
 * row does not see take no part in it, whatever they hold.  n_ctx and pos0
 * differ when rows have been evicted.  Cache rows >= n_ctx + T are neither
 * read nor written.
 * weight_out (fp32 [Hkv][max_seq], nullable): the attention weight that each
 * key received, summed over the present rows that see it and the query heads
 * of its group: rows j < n_ctx get weight_in[j] (fp32 [Hkv][max_seq]; NULL: zeros;
 * may be weight_out itself, no other overlap) plus this call's sum, rows
 * n_ctx..n_ctx+T-1 this call's sum alone; other rows stay as they are.
 * q enters the scores as two bf16 parts, which leaves a score
 *   (2^-16 + 2 dh 2^-24) sum |q_i k_i| / sqrt(dh)
 * off at most; an infinite element of K gives the infinity that it gives q.
 * Probabilities are rounded to bf16 for the product with V.  A row whose every
 * score is -infinity gives no key weight.  The result of a call does not depend
 * on timing (no floating-point atomics): equal calls give equal bits.  But keys
 * are summed in blocks from row 0 and from row n_ctx on, split and interleaved
 * as T, n_ctx, the heads and the device's SMs suggest, so that a node's row may
 * differ in its last bits from the same node's in another tree or alone, and
 * from ssd_op_attention's: the greedy choice between near ties is not held to
 * that of one token at a time. */
/* (Of calls with and without weights: with up to 16 rows per K/V head, 4 bytes
 * for each row and key are those of the weights.) */
size_t ssd_op_tree_attention_workspace(int32_t T, int32_t n_ctx, int32_t H, int32_t Hkv,
                                       int32_t dh);
ssd_status ssd_op_tree_attention(const float* qkv, const int32_t* parents, int32_t T,
                                 int32_t n_ctx, int32_t pos0, void* k_cache, void* v_cache,
                                 int32_t max_seq, int32_t H, int32_t Hkv, int32_t dh, float theta,
                                 const float* weight_in, float* weight_out, void* out,
                                 void* workspace, size_t workspace_bytes, void* stream);

/* Eviction from a cache by accumulated attention weight: of rows 0..n-1 of
 * each K/V head, keeps the first `sinks`, the last `recent` and, of those
 * between, the ones with the largest weight (ties: the lower row; NaN counts
 * as -infinity), `keep` rows in all, in their order:
 *   kept[h][j]       the j-th kept row's index        (int32 [Hkv][keep])
 *   k_out[h][j], v_out[h][j], weight_out[h][j] = its K, V and weight.
 * sinks, recent >= 0; sinks + recent <= keep <= n <= max_seq;
 * 1 <= keep <= max_out.  k, v [Hkv][max_seq][dh] and weight fp32
 * [Hkv][max_seq]; k_out, v_out [Hkv][max_out][dh] and weight_out fp32
 * [Hkv][max_out] (nullable), no overlap with the inputs; rows >= keep of the
 * outputs stay as they are.  dtype: SSD_DTYPE_BF16 or SSD_DTYPE_FP32, the
 * element type of the four caches; a row's bytes are a multiple of 16. */
ssd_status ssd_op_cache_evict(const void* k, const void* v, const float* weight, int32_t n,
                              int32_t keep, int32_t sinks, int32_t recent, int32_t max_seq,
                              int32_t Hkv, int32_t dh, int32_t dtype, void* k_out, void* v_out,
                              float* weight_out, int32_t max_out, int32_t* kept, void* stream);

/* Beam selection: the W best candidates (b, v) of B beams by
 *   scores[b] + (logits[b][v] - lse[b])
 * (computed in 64 bits, so that no rounding reorders them; within a beam by
 * logit; ties: the lower beam, then the lower token), best first:
 *   tokens[w] = v, parents[w] = b, scores_out[w] = the score in fp32.
 * logits fp32 [B][V]; lse: row b's log sum exp at lse[b * lse_stride]
 * (&stats[0].lse with a stride of 12 reads ssd_row_stats records), NULL
 * where logits are log-probabilities already.  done (int32 [B], nullable):
 * beam b with done[b] != 0 has ended and stands for itself, one candidate
 * with token end_id and score scores[b]; its logits are not read.
 * done_out (int32 [W], nullable): 1 where the token is end_id (or nothing was
 * left), else 0.  NaN and -infinity scores are no candidates; where fewer
 * than W are left, the rest is tokens = parents = -1, scores_out = -infinity.
 * 1 <= B <= 256, 1 <= W <= 256, V >= 1, -1 <= end_id < V, and end_id >= 0
 * with done; logits, lse and scores 4-byte aligned, no other alignment. */
size_t ssd_op_beam_select_workspace(int32_t B, int32_t V, int32_t W);
ssd_status ssd_op_beam_select(const float* logits, int32_t B, int32_t V, const float* lse,
                              int32_t lse_stride, const float* scores, const int32_t* done,
                              int32_t end_id, int32_t W, int32_t* tokens, int32_t* parents,
                              float* scores_out, int32_t* done_out, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Reordering of the beams' caches after a selection: state w of the output
 * takes rows start..stop-1 of every group of state parents[w] of the input.
 * k, v [B][groups][max_seq][row_bytes] (groups = layers x K/V heads; v and
 * v_out may both be NULL), k_out, v_out [W][groups][max_seq][row_bytes], no
 * overlap; row_bytes a multiple of 16.  0 <= start <= stop <= max_seq; all
 * other rows stay as they are, and so does state w where parents[w] (device
 * int32 [W]) is outside 0..B-1. */
ssd_status ssd_op_beam_reorder(const void* k, const void* v, const int32_t* parents, int32_t B,
                               int32_t W, int32_t groups, int32_t max_seq, int32_t start,
                               int32_t stop, int32_t row_bytes, void* k_out, void* v_out,
                               void* stream);

/* Description of the most recent failed op call on this host thread. */
const char* ssd_ops_last_error(void);

/* Failure detection self-test: runs the device-side bounded waits the
 * kernels use (an mbarrier wait, a global-counter wait) against conditions
 * that never come true, each limited to `polls` polls (1..2^20).  Every wait
 * must give up and report instead of hanging: *code_out (host) receives bit
 * 0 if the mbarrier wait gave up and bit 1 if the counter wait did (3 when
 * both behave).  Synchronises the stream.  Errors: INVALID_ARG, CUDA. */
ssd_status ssd_op_wait_selftest(int32_t polls, int32_t* code_out, void* stream);

/* The same of the tree attention, for the later calls of this host thread:
 * CTA `attention` of its attention kernel acts as after a wait that gave up,
 * and the waits of CTA `weights` of the kernel that sums the weights of many
 * rows give up at once (-1: none, as at the start).  Such a call ends, still
 * returns SSD_OK, and has NaN in every row of out (in every key's weight) that
 * may be incomplete.  Errors: INVALID_ARG (below -1). */
ssd_status ssd_debug_tree_give_up(int32_t attention, int32_t weights);

/* ssd_op_linear for callers that cannot allocate device memory (the pages
 * have no counterpart; this is a library convenience).  Same arguments,
 * layout and result as ssd_op_linear, but the GEMV's scratch (partial sums of
 * row groups split across CTAs, completion counters) comes from a fixed
 * 1 MiB + 4.25 KiB array that the library reserves on every GPU that loads it,
 * held until the process exits; no cudaMalloc, cudaFree or other allocating
 * routine is called.  R must be <= 8192 (SSD_ERR_CAPACITY otherwise).
 * The first call on a device looks up the array's device address with that
 * device current and keeps it; make that first call before any stream
 * capture, and make no call on a device after cudaDeviceReset on it (the
 * reset destroys the array the kept address points to).  Every
 * call on a device shares the one array and clears its counters on entry, so
 * calls whose kernels overlap on the GPU (different streams, or different
 * host threads) race and must be serialised by the caller.  Errors are
 * described by ssd_op_linear_noalloc_last_error(). */
ssd_status ssd_op_linear_noalloc(const void* W, int32_t R, int32_t K, const void* act, int32_t M,
                                 float* y, void* stream);
const char* ssd_op_linear_noalloc_last_error(void);

#ifdef __cplusplus
}
#endif
#endif /* SSD_OPS_H_ */
