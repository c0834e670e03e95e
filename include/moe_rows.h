/*
 * moe_rows.h -- C ABI of the rows around an expert stage (sm_103a): tokens sorted by expert, for any
 * router's choice, the way back with gates applied, and the gradients of both.
 *
 * T tokens, k slots a token (slot s = t * k + j), E experts.  What expert a slot chose is idx[t, j]; a
 * value outside [0, E) is a slot without a row (dropped, or an expert of another rank).  The other
 * slots' rows lie expert by expert, inside an expert in slot order:
 *   counts[e]       rows of expert e (what moe_expert_forward and moe_fp8_expert_forward take)
 *   slot_pos[t, j]  the row of slot (t, j), -1 where it has none
 *   row_slot[p]     the slot of row p, -1 for p from the sum of the counts on
 * The buffers of rows have R of them.  Wherever slot_pos is read, a slot whose value lies outside [0, R)
 * has no row: nothing is read or written for it.  The values inside [0, R) have to be different ones
 * (as the sort writes them); rows that no slot names are left as they were.
 *
 * Conventions are those of moe.h, but that every array needs only the alignment of its type (the
 * workspace: 256 bytes).  Arrays that a call writes overlap no other ones of the call, unless said
 * otherwise.
 */
#ifndef MOE_ROWS_H
#define MOE_ROWS_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Bytes of workspace that a sort of T tokens needs: 0 where it needs none (up to 6144 slots), and for sizes that no call
 * takes. */
size_t moe_rows_workspace(int64_t T, int32_t k, int32_t n_experts);

/* counts [E], slot_pos [T, k] and row_slot [T k] (may be NULL) from idx [T, k], whose values have
 * idx_bytes bytes, 4 or 8.  T >= 0, 1 <= k <= 64, 1 <= E <= 1024, T k < 2^31.  T = 0 sets counts
 * to 0. */
moe_status moe_rows_sort(const void* idx, int32_t idx_bytes, int64_t T, int32_t k, int32_t n_experts, int32_t* counts,
                         int32_t* slot_pos, int32_t* row_slot, void* workspace, size_t workspace_bytes, void* stream);

/* x_rows[slot_pos[t, j]] = x[t], with gates (may be NULL) row_gates[slot_pos[t, j]] = gates[t, j].
 * x [T, d] of elem_bytes (1, 2 or 4) bytes a value with a pitch of ldx values, x_rows [R, d].  x_scales
 * [T, scale_bytes] and row_scales [R, scale_bytes] (4-byte aligned, scale_bytes a multiple of 4; both or
 * neither) go with the rows: the block factors of 8-bit rows. */
moe_status moe_rows_gather(const int32_t* slot_pos, int64_t T, int32_t k, const void* x, int32_t elem_bytes, int64_t d,
                           int64_t ldx, int64_t R, void* x_rows, const uint8_t* x_scales, uint8_t* row_scales,
                           int64_t scale_bytes, const float* gates, float* row_gates, void* stream);

/* moe_rows_sort and moe_rows_gather in one call: one launch for few slots, three else. */
moe_status moe_rows_dispatch(const void* idx, int32_t idx_bytes, int64_t T, int32_t k, int32_t n_experts, int32_t* counts,
                             int32_t* slot_pos, int32_t* row_slot, const void* x, int32_t elem_bytes, int64_t d,
                             int64_t ldx, int64_t R, void* x_rows, const uint8_t* x_scales, uint8_t* row_scales,
                             int64_t scale_bytes, const float* gates, float* row_gates, void* workspace,
                             size_t workspace_bytes, void* stream);

/* out[t] = residual[t] + sum_j gates[t, j] * y_rows[slot_pos[t, j]], the sum over j in fp32 and in order,
 * rounded once.  gates [T, k] fp32, NULL for ones (the gradient of moe_rows_gather: x's from the rows');
 * residual [T, d] in out_dtype, NULL for none; out [T, d], which may be residual itself.  y_rows
 * [R, d] in y_dtype. */
moe_status moe_rows_combine(const void* y_rows, int32_t y_dtype, int64_t R, const int32_t* slot_pos, const float* gates,
                            int64_t T, int32_t k, int64_t d, const void* residual, void* out, int32_t out_dtype,
                            void* stream);

/* Its gradients, from dout = dL/dout [T, d] (that of residual is dout):
 *   dy_rows[slot_pos[t, j]] = gates[t, j] * dout[t]                  [R, d] in y_dtype, NULL: not wanted
 *   dgates[t, j] = sum_c dout[t, c] * y_rows[slot_pos[t, j], c]      [T, k] fp32, NULL: not wanted; 0
 *                                                                    for a slot without a row
 * The sums are fp32 ones in a fixed order.  gates NULL: ones.  y_rows [R, d] may be NULL without
 * dgates; dy_rows may be y_rows itself. */
moe_status moe_rows_combine_backward(const void* dout, int32_t dout_dtype, const int32_t* slot_pos, const float* gates,
                                     int64_t T, int32_t k, int64_t d, int64_t R, const void* y_rows, void* dy_rows,
                                     int32_t y_dtype, float* dgates, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ROWS_H */
