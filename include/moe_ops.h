/*
 * moe_ops.h -- operators beside the MoE layer forward of moe.h (same library, same
 * conventions: caller-owned device pointers, checks before any launch, moe_status
 * codes, moe_last_error(), no allocation, no host synchronisation, work enqueued on
 * `stream` of the current device, outputs fully overwritten, bitwise repeatable):
 *
 *   - the products of a few tokens with 4-bit expert weights (moe_matvec_int4,
 *     moe_ffn_int4): decoding, where every weight is read once and no row is padded,
 *     gathered or dispatched;
 *   - the training side of the router: the load-balance loss with the per-expert counts
 *     (moe_balance_loss) and the gradient of the gate weights and of that loss with
 *     respect to the logits (moe_route_bwd).
 *
 * Limits shared with the router: 1 <= k <= min(E, 64), E <= 1024.
 */
#ifndef FP8GG_MOE_OPS_H
#define FP8GG_MOE_OPS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Slots (token, expert pairs) one few-token call takes; larger batches belong to the
 * dispatched grouped GEMMs of moe.h. */
#define MOE_FEW_SLOTS_MAX 1024

/* moe_quant_weight_int4 with blocks of `group` (32, 64 or 128) weights along K: for each
 * row n and block, scale = max|w| (1 if 0), q = rne(fl32(fl32(w/scale)*7)) in [-7, 7],
 * s7 = fl32(scale/7).  w [G, N, K] fp32 -> q [G, N, K/2] packed as MOE_INT4 describes,
 * s7 [G, N, K/group] fp32.  K a multiple of group; w and q 16-byte aligned.  With
 * group = 128 the outputs are those of moe_quant_weight_int4. */
int moe_quant_weight_int4_group(const float *w, int G, int N, int K, int group, uint8_t *q,
                                float *s7, void *stream);

/* Matrix-vector products of a few rows with 4-bit weights and group scales.  Slot s
 * multiplies row s / x_div of x with expert e = idx[s]'s matrix (e = 0 for every slot
 * when idx is NULL):
 *   v[s, n] = sum_g s7[e, n, g] * ( sum_{k in group g} q[e, n, k] * x[s / x_div, k] )
 *   MOE_EPI_PLAIN:  y[s, n] = v[s, n],                                 n < N
 *   MOE_EPI_SWIGLU: y[s, n] = silu(v[s, n]) * v[s, N + n]   (2N weight rows), n < N
 * The products q x are exact (below 2^-115 in magnitude to a multiple of 2^-139), the sums
 * and the SwiGLU are taken in fp32, and y is rounded once.  The weights are used as q * s7 (grouped_gemm_w4a16 rounds that product to bf16
 * first).  A slot whose expert lies outside [0, G) (a dropped slot, a padding row) gets
 * a row of zeros and its x row is not used.
 *   x [ceil(S / x_div), K] of dtype x_dt and y [S, N] of dtype y_dt (MOE_BF16 or MOE_F32
 *   each); q [G, Nb, K/2] and s7 [G, Nb, K/group] as moe_quant_weight_int4 or
 *   moe_quant_weight_int4_group write them, Nb = N or 2N; group 32, 64 or 128; K a
 *   positive multiple of group, K <= 2^24; 1 <= N <= 2^24; 1 <= G <= 65536;
 *   0 <= S <= MOE_FEW_SLOTS_MAX; x_div >= 1 (1 without idx).  x and q 16-byte aligned.  y
 *   must not overlap an input (not checked).
 * Slots may name the same expert (its weights are then read once for up to 16 or 48 rows of
 * x, an fp32 row counting as three) and the same row. */
int moe_matvec_int4(const void *x, moe_dtype x_dt, int x_div, const uint8_t *q, const float *s7,
                    int group, const int32_t *idx, int S, int G, int N, int K, int epilogue,
                    void *y, moe_dtype y_dt, void *stream);

/* Bytes of device workspace moe_ffn_int4 needs (0 on bad sizes or T = 0). */
size_t moe_ffn_int4_workspace_size(int T, int k, int d, int I);

/* The routed experts' FFN of a few tokens with 4-bit weights, after the router:
 *   y[t] = sum_j topk_w[t, j] * W2_e ( silu(Wgate_e x_t) * (Wup_e x_t) ),  e = topk_idx[t, j]
 * with the products of moe_matvec_int4; the SwiGLU output stays in fp32, the k terms are
 * added in fp32 in an order fixed by the sizes, and y is rounded once.  Slots whose expert lies
 * outside [0, E) are skipped (their weight is not used); a token without any gets zeros.
 *   x [T, d] and y [T, d] of dtype dt (MOE_BF16 or MOE_F32); w13 [E, 2I, d/2] (rows [0, I)
 *   gate, [I, 2I) up), s13 [E, 2I, d/group]; w2 [E, d, I/2], s2 [E, d, I/group]; topk_idx
 *   [T, k] int32, topk_w [T, k] fp32 as moe_route writes them; d and I positive multiples
 *   of group (32, 64 or 128), at most 2^24; T >= 0, T * k <= MOE_FEW_SLOTS_MAX; 1 <= E <= 65536;
 *   x, w13, w2 and ws 16-byte aligned; ws_bytes >= moe_ffn_int4_workspace_size().  y must
 *   not overlap an input (not checked). */
int moe_ffn_int4(const void *x, moe_dtype dt, const uint8_t *w13, const float *s13,
                 const uint8_t *w2, const float *s2, int group, const int32_t *topk_idx,
                 const float *topk_w, int T, int k, int E, int d, int I, void *y, void *ws,
                 size_t ws_bytes, void *stream);

/* Balance losses.  Over the tokens of a segment that count (n of them), with
 * p[t] = softmax(logits[t] + bias), P_e = mean_t p[t, e] and f_e = counts_e / (k n): */
#define MOE_BALANCE_SWITCH 0  /* coef * E * sum_e f_e P_e, f taken as a constant            */
#define MOE_BALANCE_SQUARE 1  /* coef * sum_e (P_e - 1/E)^2; E times it is (std/mean)^2 of P */

/* Bytes of device workspace moe_balance_loss and moe_route_bwd need (0 on bad sizes). */
size_t moe_balance_workspace_size(int T, int E, int B);
size_t moe_route_bwd_workspace_size(int T, int E);

/* The load-balance loss of a routed batch, the per-expert counts and what the loss's
 * gradient needs.  Segment b holds the tokens [offsets[b], offsets[b+1]) (device int32
 * [B+1], non-decreasing, within [0, T]; NULL: B = 1 and all T tokens).  A token counts
 * if it lies in a segment and its mask byte is nonzero (mask NULL: all); the logits and
 * indices of other tokens have no influence, whatever they hold.
 *   counts [B, E] int32  counting tokens' slots per expert; indices outside [0, E) not
 *   probs  [B, E] fp32   P_e (0 for a segment without counting tokens)
 *   grad   [B, E] fp32   dloss / dp[t, e] of a counting token of segment b, less its mean
 *                        over e for MOE_BALANCE_SWITCH (a constant that the softmax's
 *                        gradient cancels): what moe_route_bwd takes
 *   loss   [1] fp32      mean of the losses of the segments that have counting tokens
 *                        (0 if none has)
 * The softmax is the router's (key = fl32(logit + bias), fp32); sums over tokens are
 * carried on in fp64.  -inf logits are experts with probability 0; a token whose logits
 * are all -inf has p = 0.  NaN or +inf in a counting token's row gives NaN probs and loss
 * (and grad, for MOE_BALANCE_SQUARE).  logits [T, E] fp32, bias [E] fp32 or NULL (0),
 * topk_idx [T, k] int32; 1 <= B <= 65535; pointers to [T, ...] inputs may be NULL when T = 0. */
int moe_balance_loss(const float *logits, const float *bias, const int32_t *topk_idx,
                     const uint8_t *mask, const int32_t *offsets, int T, int E, int k, int B,
                     int kind, float coef, int32_t *counts, float *probs, float *grad,
                     float *loss, void *ws, size_t ws_bytes, void *stream);

/* Gradient of the router's outputs with respect to its logits (and bias):
 *   dlogits[t] = sum_j dtopk_w[t, j] dtopk_w_j/dlogits  +  dloss * dL/dlogits[t]
 * for the gate weights that moe_route / moe_route_from_logits return for topk_idx with the
 * same flags (the choice of experts is a constant) and the loss of moe_balance_loss.
 * With p = softmax(logits + bias), D_e the sum of dtopk_w over the slots that chose e and
 * G = D + dloss * grad[b]:  dlogits_e = p_e (G_e - sum_i p_i G_i); with MOE_ROUTE_RENORM
 * the gate part is instead w_j (dtopk_w_j - sum_l w_l dtopk_w_l) at the chosen experts.
 *   dtopk_w [T, k] fp32 or NULL (no gate part); balance_grad [B, E] fp32 (moe_balance_loss's
 *   grad) or NULL (no loss part); dloss [1] fp32 on the device or NULL (1); mask and
 *   offsets as in moe_balance_loss: rows of tokens that do not count are written as zeros
 *   and their inputs have no influence.  Slots with an index outside [0, E) have no part.
 *   dlogits [T, E] fp32; dbias [E] fp32, the sum of dlogits over the tokens, or NULL.
 *   ws is used for dbias only (NULL without it); ws_bytes >= moe_route_bwd_workspace_size. */
int moe_route_bwd(const float *logits, const float *bias, const int32_t *topk_idx,
                  const float *dtopk_w, const uint8_t *mask, const int32_t *offsets,
                  const float *balance_grad, const float *dloss, int T, int E, int k, int B,
                  unsigned flags, float *dlogits, float *dbias, void *ws, size_t ws_bytes,
                  void *stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8GG_MOE_OPS_H */
