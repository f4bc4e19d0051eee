/*
 * moe_training.h -- C ABI of the training operators beside moe.h's on MI355X
 * (gfx950): the gradients of the experts' feed-forward on grouped rows, and
 * activation checkpoints in 8 bits with the forward that writes and the
 * backward that reads them.  Part of libmoe.so; types, status codes and
 * conventions are moe.h's (device pointers, work enqueued on `stream`,
 * arguments checked on the host first, nothing allocated, values read on the
 * device clamped to what they index).
 *
 * Rows, weights, gradients, codes and workspaces begin at multiples of 16
 * bytes (MOE_ERR_ARG otherwise); scales, indices and routing weights at
 * multiples of their own 4.  No output overlaps an input, another output or the
 * workspace.  Limits beside moe.h's: d and I below 2^21, grouped
 * rows * max(d, 2I) below 2^31, E * 2*d*I below 2^34, a layer's T*d below 2^30.
 *
 * A workspace size holds for its arguments alone: fewer rows can need a larger
 * one (the products of few rows are cut into ranges, summed from there).
 *
 * The 8-bit checkpoint.  What the backward needs of the forward, beside x and
 * the weights, are the pre-activations g | u = x Wgu of every grouped row;
 * h = silu(g) u is formed from them again and y is not needed.  They are kept
 * as whole multiples of a scale, one float32 scale for 64 consecutive columns:
 *   s = max(amax, 2^-100) / 127,  code = v / s to the nearest whole number,
 *   amax the largest magnitude of the 64; the value kept is code * s
 *   gu_q [rows, 2I] int8 (gate columns first)
 *   gu_s [rows, 2, I/64] float32 (gate blocks first)
 * 2.125 I bytes a row, where the bf16 intermediates of moe_forward_train take
 * 4d + 6I.  A value is off by at most s / 2 = amax / 254: 0.57% of the
 * standard deviation for normally distributed values (e4m3 codes: 2.6%).  A
 * block that holds an infinity or a NaN gets a NaN scale, and its values are
 * NaN; every finite block is kept, up to the largest float32.  Gradients from a
 * checkpoint are those of the formulas below at the kept values of g and u; the
 * forward's own output does not pass through them.
 */
#ifndef TRE_MOE_TRAINING_H
#define TRE_MOE_TRAINING_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- the experts' feed-forward on grouped rows ---------------------------------
 * moe_grouped_ffn for a training step, for rows that were grouped elsewhere
 * (the rows an expert-parallel rank received).
 *
 * moe_grouped_ffn_train: y_perm by moe_grouped_ffn's formula and roundings (g
 * and u unrounded into h, h to bf16, y once; the order of sums may differ, and
 * h stays float32 where it does in the backward), and
 * the 8-bit checkpoint of the rows' g | u.
 *
 * moe_grouped_ffn_backward: gradients of <dy_perm, y_perm>.  For row r of
 * expert e, with s = sigmoid(g) and h = g s u:
 *   dh = dy Wd[e]^T;  dg = dh u s (1 + g (1 - s));  du = dh g s
 *   dx = [dg | du] Wgu[e]^T;  dW_gate_up[e] = sum_r x^T [dg | du]
 *   dW_down[e] = sum_r h^T dy           (zero for an expert without rows)
 * gu_q and gu_s: a checkpoint, or both NULL: g | u are computed again from x
 * (MOE_BF16: held meanwhile as whole multiples of a scale as above, of 16 bits,
 * off by at most amax / 65534: closer than bf16 for values down to 1 / 128 of
 * their block's largest, coarser below).  MOE_BF16: float32 accumulation; h, dg
 * and du are rounded to bf16 before the products that read them (in calls of few
 * rows whose sums are not long they stay float32, by a rule on the sizes), and
 * every gradient once; MOE_F32: float32 throughout.  The order of every sum
 * depends on the sizes only, so equal calls give equal bits.
 *   x_perm, dy_perm [max_rows, d] dt; expert_offsets [E+1]
 *   y_perm, dx_perm [max_rows, d] dt (outputs; rows >= expert_offsets[E], of
 *     the checkpoint too, are untouched)
 *   dw_gate_up [E, d, 2I], dw_down [E, I, d] dt (outputs, overwritten)
 *   workspace >= the matching *_workspace_size(); max_rows == 0 zeroes the
 *     weight gradients only                                                 */
size_t moe_grouped_ffn_train_workspace_size(int32_t max_rows, int32_t E, int32_t d, int32_t I, moe_dtype dt);
moe_status moe_grouped_ffn_train(const void* x_perm, const int32_t* expert_offsets, int32_t max_rows, int32_t E,
                                 int32_t d, int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt,
                                 void* y_perm, void* gu_q, float* gu_s, void* workspace, size_t workspace_bytes,
                                 void* stream);
size_t moe_grouped_ffn_backward_workspace_size(int32_t max_rows, int32_t E, int32_t d, int32_t I, moe_dtype dt);
moe_status moe_grouped_ffn_backward(const void* x_perm, const int32_t* expert_offsets, int32_t max_rows, int32_t E,
                                    int32_t d, int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt,
                                    const void* gu_q, const float* gu_s, const void* dy_perm, void* dx_perm,
                                    void* dw_gate_up, void* dw_down, void* workspace, size_t workspace_bytes,
                                    void* stream);

/* ---- the whole layer with an 8-bit checkpoint ------------------------------------
 * moe_forward_train_q8: topk_idx and topk_w exactly as moe_forward computes
 * them (from logits, or given pairs), out by its formula, the grouping and the
 * checkpoint.  MOE_BF16 rounds h (where the backward does) and then out: the
 * experts' rows y stay float32 up to out's one rounding, where moe_forward
 * rounds them too.
 * The caller keeps expert_offsets [E+1], row_token [T*k], pair_row [T*k],
 * gu_q [T*k, 2I] and gu_s [T*k, 2, I/64] for the backward; the workspace is
 * free again when the call's work has run.
 *
 * moe_backward_q8: gradients of <dout, out>, as moe_backward defines them, at
 * the checkpoint's g and u.  The routing weight goes into h and [dg | du] before
 * they are rounded, so that every product reads dout as it is, and a token's dx
 * is summed from float32 rows and rounded once.  With y not kept, a routing weight's gradient is
 * taken on the other side of the down projection:
 *   dtopk_w[p] = <dout_t, h_p Wd[e]> = <dout_t Wd[e]^T, h_p>
 *   dlogits[t, e_j] = w_j (dtopk_w_j - sum_i w_i dtopk_w_i) for the weights of
 *   moe_route_topk, zero for experts not selected (NULL to skip)
 *   x, dout [T, d] dt; topk_idx, topk_w [T, k] and the five kept arrays: as
 *     the forward filled or read them (rows of a checkpoint beyond
 *     expert_offsets[E] are not read; row_token has to be given, and is not
 *     read either: pair_row says where a token's rows are)
 *   dx [T, d], dw_gate_up [E, d, 2I], dw_down [E, I, d] dt, dtopk_w [T, k]
 *     float32 (outputs, overwritten; dtopk_w is 0 for dropped pairs)
 *   workspace >= the matching *_workspace_size(); T == 0 zeroes the weight
 *     gradients only                                                        */
size_t moe_forward_train_q8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I, moe_dtype dt);
moe_status moe_forward_train_q8(const void* x, const float* logits, int32_t T, int32_t d, int32_t E, int32_t k,
                                int32_t I, const void* w_gate_up, const void* w_down, moe_dtype dt, int32_t* topk_idx,
                                float* topk_w, int32_t* expert_offsets, int32_t* row_token, int32_t* pair_row,
                                void* gu_q, float* gu_s, void* out, void* workspace, size_t workspace_bytes,
                                void* stream);
size_t moe_backward_q8_workspace_size(int32_t T, int32_t d, int32_t E, int32_t k, int32_t I, moe_dtype dt);
moe_status moe_backward_q8(const void* x, int32_t T, int32_t d, int32_t E, int32_t k, int32_t I,
                           const void* w_gate_up, const void* w_down, moe_dtype dt, const int32_t* topk_idx,
                           const float* topk_w, const int32_t* expert_offsets, const int32_t* row_token,
                           const int32_t* pair_row, const void* gu_q, const float* gu_s, const void* dout, void* dx,
                           void* dw_gate_up, void* dw_down, float* dtopk_w, float* dlogits, void* workspace,
                           size_t workspace_bytes, void* stream);

/* The pre-activations a checkpoint stands for, gu [rows, 2I] dt (output):
 * code * scale, rounded to dt once.                                          */
moe_status moe_checkpoint_values(const void* gu_q, const float* gu_s, int32_t rows, int32_t I, moe_dtype dt, void* gu,
                                 void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TRE_MOE_TRAINING_H */
