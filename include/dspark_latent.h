/*
 * dspark_latent.h — C ABI of the draft attention in the latent space of MLA
 * (page "GLM 5.2 DSpark speculative-training design", parameter summary: the
 * inference cache holds 576 numbers per token and layer, a 512-wide latent and
 * a 64-wide rope key; §4 "MLA": keys and values are linear maps of the latent).
 *
 * Absorbed form. With the key half of the kv expansion folded into the query
 * (q_l = W_UK^T q^C per head) and the value half applied after the attention
 * (o_head = W_UV O), all heads attend to the same latent vectors:
 *   s = scale * (q_l . c_p + rope(q_r, pos_q) . rope(k_r_p, p)),
 *   O = softmax(s) C,
 * which equals the attention of dspark_attn.h over the expanded keys and values
 * of the same latents (scale = (d_c + d_r)^(-1/2) of the expanded head).
 * Here: the training operators over the draft mask (forward and backward), the
 * paged cache of latents (write, read), and the attention of new tokens over
 * that cache.
 *
 * Conventions (ownership, streams, statuses, dspark_get_error, the launch
 * counter and the wait limit) are those of dspark_attn.h. RoPE turns adjacent
 * pairs (2i, 2i+1) of the d_r-wide parts by pos * rope_base^(-2i/d_r).
 */
#ifndef DSPARK_LATENT_H
#define DSPARK_LATENT_H

#include "dspark_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- training: attention over the draft mask -------------------------------
 * Layouts (contiguous, row-major):
 *   q   [B, n_h, 5N, d_l + d_r] dtype   absorbed query, rope slice last, NOT rotated
 *   c   [B, S + 5N, d_l]        dtype   latents, shared by the heads: keys and values
 *   kr  [B, S + 5N, d_r]        dtype   rope keys, NOT rotated
 *   o   [B, n_h, 5N, d_l]       dtype;  lse [B, n_h, 5N] fp32 (natural log)
 *   do_ like o; dq like q; dc like c; dkr like kr
 * The mask, anchors, keep, padding rows (O = 0, LSE = -inf, zero gradients) and
 * the check of anchors are those of dspark_attn_fwd. Every element of every
 * output is written.
 * Limits checked on the host: 0 <= B <= 65535, n_h >= 1, 1 <= S < 2^30 - 8,
 *   0 <= N <= 8192, 1 <= W <= 4096, 1 <= d_l <= 512, d_r even, 0 <= d_r <= 128,
 *   (S + 5N) * max(d_l, d_r) < 2^31, 5N * n_h * (d_l + d_r) < 2^31,
 *   B * n_h * 5N < 2^31, rope_base and scale finite and > 0. */
typedef struct {
    int32_t B;         /* batch */
    int32_t n_h;       /* heads */
    int32_t S;         /* context positions */
    int32_t N;         /* draft blocks (5 positions each) */
    int32_t W;         /* sliding window: W-1 context positions visible */
    int32_t d_l;       /* latent width */
    int32_t d_r;       /* rope width */
    int32_t dtype;     /* dspark_dtype of every non-integer tensor but lse */
    double rope_base;  /* RoPE base, e.g. 10000 */
    double scale;      /* softmax scale */
    int32_t reserved[2]; /* must be 0 */
} dspark_latent_problem;

/* Bytes of device workspace (0 if *p is invalid): the size the backward
 * requires; the forward uses a leading part of it. 256-byte aligned. */
DSPARK_API size_t dspark_latent_workspace_size(const dspark_latent_problem *p);

/* Forward: o and lse. flags as dspark_attn_fwd (DSPARK_FLAG_REUSE_DESCRIPTOR:
 * the workspace holds the descriptor of an earlier latent call with the same
 * anchors, keep, sizes and rope_base). */
DSPARK_API dspark_status dspark_latent_attn_fwd(const dspark_latent_problem *p, const void *q, const void *c,
                                                const void *kr, const int32_t *anchors, const uint8_t *keep, void *o,
                                                float *lse, void *workspace, size_t workspace_bytes, uint32_t flags,
                                                void *stream);

/* Backward for a loss L with dL/dO = do_: writes dq, dc (the latent's gradient
 * as key and as value) and dkr, with respect to the un-rotated inputs. lse is
 * the forward's. The forward's O is not needed: rowsum(dO o O) is formed as
 * sum_k P_k dP_k. dc and dkr are fp32 sums over heads and blocks, in an order that
 * may differ between runs, rounded once. */
DSPARK_API dspark_status dspark_latent_attn_bwd(const dspark_latent_problem *p, const void *q, const void *c,
                                                const void *kr, const int32_t *anchors, const uint8_t *keep,
                                                const float *lse, const void *do_, void *dq, void *dc, void *dkr,
                                                void *workspace, size_t workspace_bytes, uint32_t flags,
                                                void *stream);

/* ---- the paged latent cache --------------------------------------------------
 * A cache is [n_pages, page_size] rows of one token each; slot s is row
 * s % page_size of page s / page_size. Rows by kind:
 *   DSPARK_CACHE_F32, DSPARK_CACHE_BF16: d_l latent then d_r rotated rope-key
 *     values of that type;
 *   DSPARK_CACHE_FP8: d_l e4m3 values; d_r bf16 rotated rope-key values; one
 *     fp32 scale per 128 latent values; zero bytes up to a multiple of 16. A
 *     latent value is its e4m3 value times its scale. The scale is the least
 *     power of two 2^e, e >= -117, with |x| <= 448 * 2^e for the group's finite
 *     values (1 where they are all 0), so the values it stands for are bf16
 *     numbers (but 2^128, what 248 * 2^120 and more is rounded to: infinity when
 *     read); values that are not finite are stored as NaN.
 * Rows and caches are 16-byte aligned: d_l and d_r multiples of 8 (d_l of 128
 * for FP8). */
typedef enum { DSPARK_CACHE_F32 = 0, DSPARK_CACHE_BF16 = 1, DSPARK_CACHE_FP8 = 2 } dspark_cache_kind;

/* Bytes of one cache row (0 for an unknown kind or widths it does not take:
 * d_l in 8 .. 512, d_r in 0 .. 128, multiples as above, d_r even). */
DSPARK_API size_t dspark_latent_row_bytes(int32_t kind, int32_t d_l, int32_t d_r);

typedef struct {
    int32_t T;          /* tokens, at most 2^31 - 64 */
    int32_t d_l, d_r;   /* widths */
    int32_t kind;       /* dspark_cache_kind */
    int32_t n_pages, page_size;
    int32_t dtype;      /* dspark_dtype of c, kr, norm_weight (write) or of the outputs (read) */
    int32_t reserved;   /* must be 0 */
} dspark_latent_cache;

/* Writes T tokens' rows into row slots[t]: y = c * (mean(c^2) + eps)^(-1/2) *
 * norm_weight (y = c when norm_weight is NULL), rounded once to the cache's type,
 * and the rope key turned to its position (the angle in 64 bits, sine, cosine and
 * products in fp32: within 8 * 2^-24 of the pair's size), rounded to the cache's
 * type of rope keys. A slot outside
 * [0, n_pages * page_size) (such as -1, a padded token) writes nothing; the
 * other slots of a call have to be distinct. Other rows stay as they were.
 *   c [T, d_l], kr [T, d_r], norm_weight [d_l] or NULL: dtype, 16-byte aligned;
 *   positions [T] int32; slots [T] int64. Launches one kernel; eps >= 0. */
DSPARK_API dspark_status dspark_latent_cache_write(const dspark_latent_cache *p, const void *c, const void *kr,
                                                   const void *norm_weight, double eps, double rope_base,
                                                   const int32_t *positions, const int64_t *slots, void *cache,
                                                   void *stream);

/* Reads T rows back as the values that they stand for (rounded to dtype):
 * c_out [T, d_l], kr_out [T, d_r] (the rotated rope key; NULL = not wanted).
 * A slot out of range reads as zeros; slots may repeat. Launches one kernel. */
DSPARK_API dspark_status dspark_latent_cache_read(const dspark_latent_cache *p, const void *cache,
                                                  const int64_t *slots, void *c_out, void *kr_out, void *stream);

/* ---- serving: new tokens over the paged cache ----------------------------------
 * Sequence s has the new tokens q_start[s] .. q_start[s+1] - 1 of q and
 * kv_len[s] cached keys, its new tokens (already written) last: token i of q_len
 * is at position kv_len - q_len + i. Key p is row p % page_size of page
 * block_table[s][p / page_size]. A token at position t sees
 *   causal = 1: keys p <= t, and p > t - window when window > 0;
 *   causal = 0 (a draft block: its tokens see one another, page §3): every key
 *     p < kv_len, and p > kv_len - q_len - window when window > 0, the same
 *     window [A - W + 1, A) as in training for a block at anchor A.
 * A row that sees no key gives O = 0, LSE = -inf. Rows of o and lse behind the
 * last sequence's tokens are left as they were.
 *   q [T, n_h, d_l + d_r], o [T, n_h, d_l]: dtype, rope slice last and NOT
 *     rotated, with the given strides in elements (multiples of 16 bytes, positive
 *     and below 2^39; both 0 = contiguous); lse [T, n_h] fp32 contiguous
 *   q_start [n_seq + 1], kv_len [n_seq], block_table [n_seq, max_pages]: int32
 * A page outside [0, n_pages), a kv_len outside [0, max_pages * page_size] or a
 * q_start that is not ascending within [0, T] is only visible on the device, and
 * dspark_get_error returns DSPARK_ERR_PAGE: the page's keys are skipped; a sequence
 * of such a kv_len gives O = 0 and LSE = -inf; one whose two q_start entries descend
 * or leave [0, T], or that begins before the end of an earlier sequence whose
 * entries do not, attends nothing and leaves rows as they were. The other
 * sequences are not affected.
 * kind F32 goes with dtype F32, BF16 and FP8 with dtype BF16.
 * Limits: n_h >= 1, n_seq >= 0, T >= 0, page_size >= 1, widths as the cache,
 *   T * n_h < 2^31, max_pages * page_size < 2^31, n_pages * page_size < 2^31,
 *   n_seq < 2^24, window >= 0.
 * max_kv_len, a bound of kv_len known to the caller (0 = max_pages * page_size),
 * only guides the choice of kernels: a wrong one costs time, not results. */
typedef struct {
    int32_t n_seq, T, n_h, d_l, d_r;
    int32_t page_size, n_pages, max_pages;
    int32_t max_kv_len;
    int32_t window, causal;
    int32_t dtype, kind;
    int32_t reserved;  /* must be 0 */
    int64_t q_token_stride, q_head_stride, o_token_stride, o_head_stride;
    double rope_base, scale;
} dspark_latent_paged;

/* Bytes of device workspace (0 if *p is invalid), 256-byte aligned. Its first
 * word is the error word that dspark_get_error reads; each call clears it. */
DSPARK_API size_t dspark_latent_paged_workspace_size(const dspark_latent_paged *p);

DSPARK_API dspark_status dspark_latent_attn_paged(const dspark_latent_paged *p, const void *q, const void *cache,
                                                  const int32_t *block_table, const int32_t *q_start,
                                                  const int32_t *kv_len, void *o, float *lse, void *workspace,
                                                  size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_LATENT_H */
