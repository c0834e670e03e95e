/*
 * moe_fp8.h -- C ABI of the 8-bit operators around the expert layer (sm_103a).
 *
 * Number format.  An 8-bit tensor is e4m3 values (one byte each, largest finite value 448)
 * with one power-of-two factor for each block of 128 values along its rows, stored as an
 * e8m0 byte b standing for 2^(b-127) (255 stands for NaN):
 *   value[i,j] = e4m3[i,j] * 2^(scale[i', j/128] - 127)
 * Activations have a factor for every 128 columns of a row (i' = i, "1 x 128"), weights one
 * for every 128 x 128 block (i' = i/128, counted from each expert's first row).  The last
 * block of a row may be short.  A row of c values has moe_fp8_scale_cols(c) scale bytes:
 * ceil(c/128) rounded up to a multiple of 4; the library writes the padding bytes as 0.
 *
 * Quantising a block: amax = its largest |value|, b - 127 = the least integer e with
 * amax <= 448 * 2^e (b clamped to [0, 254]; b = 0 for a block of zeros), and each value is
 * v * 2^-e rounded to the nearest e4m3, ties to even.  A block that holds an infinity or a
 * NaN gets b = 255 (NaN), and what multiplies it becomes NaN.
 *
 * The powers of two are the tensor cores' own block factors: the products below apply them
 * inside the matrix instruction, and every sum is accumulated in fp32.
 *
 * Conventions are those of moe.h: device pointers, 16-byte aligned unless stated otherwise;
 * row-major; a call only enqueues work on its stream; the caller owns all memory; every
 * argument is checked on the host before any CUDA call; errors are moe_status values and
 * moe_last_error() describes them.  "ld" arguments are row pitches in elements.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Scale bytes of a row of `cols` values (0 for cols < 1). */
int64_t moe_fp8_scale_cols(int64_t cols);

/* Quantise x [rows, cols] (fp32 or bf16, row pitch ldx) to q [rows, cols] (contiguous) and
 * scales.  block_rows = 1: a factor per 128 columns of a row, scales
 * [rows, moe_fp8_scale_cols(cols)].  block_rows = 128: a factor per 128 x 128 block of each of
 * rows / expert_rows experts (rows a multiple of expert_rows >= 1), scales
 * [rows / expert_rows, ceil(expert_rows / 128), moe_fp8_scale_cols(cols)]; expert_rows is
 * ignored when block_rows = 1.  rows = 0 is allowed and does nothing.  x needs only the
 * alignment of its type. */
moe_status moe_fp8_quantize(const void* x, int32_t x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                            int32_t block_rows, int64_t expert_rows, void* q, uint8_t* scales, void* stream);

/* ---------------------------------------------------------------------------------------
 * RMS norm with the residual's addition, for the residual block around the layer:
 *   r[t] = x[t] + residual[t]       (rounded to the stream's type, fp32 or bf16)
 *   n[t] = r[t] * rstd[t] * weight,  rstd[t] = 1 / sqrt(mean_j r[t,j]^2 + eps)
 * --------------------------------------------------------------------------------------- */

/* rows >= 0, d >= 1, eps >= 0.  x, residual (may be NULL: r = x), residual_out [rows, d] in
 * `dtype` with pitches ldx, ldr and d; residual_out may be NULL only when residual is NULL
 * or r is not wanted.  weight [d] fp32, or NULL for ones.
 * Outputs, each NULL if not wanted, at least one wanted: out [rows, d] in `dtype` (n rounded
 * once); q [rows, d] with scales [rows, moe_fp8_scale_cols(d)] (n quantised from fp32, both or
 * neither); rstd [rows] fp32 (what the backward needs).  x, residual, residual_out and out need
 * only the alignment of their type.  residual_out may be x or residual itself (in place). */
moe_status moe_rmsnorm(const void* x, const void* residual, const float* weight, int32_t dtype, int64_t rows, int32_t d,
                       int64_t ldx, int64_t ldr, float eps, void* residual_out, void* out, void* q, uint8_t* scales,
                       float* rstd, void* stream);

/* Backward: from dout = dL/dn [rows, d] (fp32 or bf16, dout_dtype), r (what the forward
 * normalised: residual_out, or x without a residual; pitch ldr), its rstd, and dresidual (may
 * be NULL): the gradient that reaches r on its other way [rows, d] in `dtype`:
 *   g = dout * weight,  xhat = r * rstd
 *   dx[t]   = rstd (g - xhat * mean_j(g xhat)) + dresidual        [rows, d] in `dtype`
 *   dweight = sum_t dout[t] * xhat[t]                             [d] fp32, may be NULL
 * dx is the gradient of x and of the residual alike.  It may be dresidual, dout (where both have one
 * type) or r (where ldr is d) itself; a dx that overlaps one of them otherwise is refused.  The sum
 * over rows is taken in a fixed order (results do not depend on timing).  workspace: device,
 * 256-byte aligned, moe_rmsnorm_backward_workspace(rows, d) bytes (when dweight is wanted; may
 * be NULL where that is 0, as with few rows). */
size_t moe_rmsnorm_backward_workspace(int64_t rows, int32_t d);
moe_status moe_rmsnorm_backward(const void* dout, int32_t dout_dtype, const void* r, const float* weight,
                                const float* rstd, const void* dresidual, int32_t dtype, int64_t rows, int32_t d,
                                int64_t ldr, void* dx, float* dweight, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------------------
 * Products of 8-bit rows with 8-bit weights, the rows grouped by expert.
 *
 * Rows lie in n_sources * n_experts segments, source-major, as moe_expert_forward has them
 * (segment s: the rows of expert s % n_experts from source s / n_experts); seg_counts gives
 * their lengths on the device.  A negative count or a sum above max_rows is recorded as
 * MOE_ERR_INTERNAL (moe_fp8_get_device_status) and no row is computed; rows past the sum are
 * not written.  seg_counts may be NULL when there is one segment: all max_rows rows.
 * --------------------------------------------------------------------------------------- */

typedef struct moe_fp8_plan_s* moe_fp8_plan_t;

typedef struct {
  int64_t max_rows;        /* R: capacity of the row buffers, >= 1 */
  int32_t k;               /* K: columns of a row (the sum's length), >= 1 */
  int32_t n;               /* output columns, >= 1 */
  int32_t n_experts;       /* E */
  int32_t n_sources;       /* W; W * E <= 256 */
  int32_t out_dtype;       /* moe_dtype of the output rows */
  int32_t path;            /* MOE_PATH_AUTO (K, n multiples of 16) or MOE_PATH_SIMT (any size) */
  int64_t wait_timeout_ns; /* bound on any device-side wait, 1 ms at least; <= 0 selects 2 s */
} moe_fp8_matmul_config;

/* out[p] = A[p] . W_e^T for the rows p of expert e.  A [R, K] with scales 1 x 128; W
 * [E, n, K] with scales 128 x 128: [E, ceil(n/128), moe_fp8_scale_cols(K)]; out [R, n]. */
moe_status moe_fp8_matmul_plan(const moe_fp8_matmul_config* cfg, moe_fp8_plan_t* plan, size_t* workspace_bytes);
moe_status moe_fp8_matmul(moe_fp8_plan_t plan, const int32_t* seg_counts, const void* a, const uint8_t* a_scales,
                          const void* w, const uint8_t* w_scales, void* out, void* workspace, size_t workspace_bytes,
                          void* stream);

/* The expert stage in 8 bits, with moe_expert_config as moe_expert_plan takes it (act_dtype
 * ignored; d_model and d_expert multiples of 16 unless MOE_PATH_SIMT):
 *   h[p] = SiLU(W1_e x[p]) * (W3_e x[p])   quantised to 8 bits, 1 x 128, out of fp32
 *   y_rows[p] = gates[p] * (W2_e h[p])     bf16 [R, d]
 * x_rows [R, d] with scales [R, moe_fp8_scale_cols(d)]; gates [R] fp32; w1, w3 [E_l, F, d]
 * and w2 [E_l, d, F] with 128 x 128 scales.  On MOE_PATH_AUTO SiLU(a) is 0 for a < -87.3 (it is at most
 * 1.03e-36 in magnitude there). */
moe_status moe_fp8_expert_plan(const moe_expert_config* cfg, moe_fp8_plan_t* plan, size_t* workspace_bytes);
moe_status moe_fp8_expert_forward(moe_fp8_plan_t plan, const int32_t* seg_counts, const void* x_rows,
                                  const uint8_t* x_scales, const float* gates, const void* w1, const uint8_t* w1_scales,
                                  const void* w3, const uint8_t* w3_scales, const void* w2, const uint8_t* w2_scales,
                                  void* y_rows, void* workspace, size_t workspace_bytes, void* stream);

/* The whole layer with its experts in 8 bits, for a plan made by moe_plan with
 * MOE_FLAG_FP8_EXPERTS: the router on x (bf16 [T, d]), the dispatch of the 8-bit rows x_q [T, d]
 * with factors x_scales [T, moe_fp8_scale_cols(d)] (moe_rmsnorm writes both out of one read),
 * the experts as in moe_fp8_expert_forward, and the combine into y [T, d] in the plan's
 * out_dtype.  The workspace's views are those of moe_forward, but that xp and h hold e4m3.  The
 * plan's wait_timeout_ns is 1 ms at least, as in moe_fp8_matmul_config. */
moe_status moe_fp8_forward(moe_plan_t plan, const void* x, const void* x_q, const uint8_t* x_scales, const void* w_router,
                           const float* router_bias, const void* w1, const uint8_t* w1_scales, const void* w3,
                           const uint8_t* w3_scales, const void* w2, const uint8_t* w2_scales, void* y, void* workspace,
                           size_t workspace_bytes, void* stream);

void moe_fp8_plan_destroy(moe_fp8_plan_t plan);

/* SYNCHRONISES `stream`, then reads the workspace's status word (as moe_get_device_status). */
moe_status moe_fp8_get_device_status(moe_fp8_plan_t plan, const void* workspace, void* stream);

/* ---------------------------------------------------------------------------------------
 * Activation checkpoints in 8 bits: the SwiGLU's two pre-activations a = W1 x and b = W3 x
 * (bf16, [rows, F]) are most of what a training forward keeps.  Kept as e4m3 with a factor
 * per 128 columns they take a little over half of that.
 * --------------------------------------------------------------------------------------- */

/* a, b [rows, F] bf16 -> qa, sa, qb, sb (1 x 128), in one pass over each. */
moe_status moe_checkpoint_save_rows(const void* a, const void* b, int64_t rows, int32_t F, void* qa, uint8_t* sa,
                                    void* qb, uint8_t* sb, void* stream);

/* The values that a checkpoint holds, a and b (exact in bf16), and h = silu(a) * b; outputs
 * [rows, F] bf16, each NULL if not wanted. */
moe_status moe_checkpoint_restore_rows(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb, int64_t rows,
                                       int32_t F, void* a, void* b, void* h, void* stream);

/* The SwiGLU's backward out of the checkpoint, with a, b the values it holds:
 *   da = dh * b * silu'(a),  db = dh * silu(a),  h = silu(a) * b
 * dh, da, db, h [rows, F] bf16, computed in fp32 and rounded once.  h (for the gradient of
 * the down-projection's weights) may be NULL.  da or db may be dh itself. */
moe_status moe_checkpoint_backward_rows(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                        const void* dh, int64_t rows, int32_t F, void* da, void* db, void* h,
                                        void* stream);

/* Checkpoints of a training layer: L layers of one shape train with one workspace and L
 * checkpoints.  A checkpoint has 2 F (1 + 1/32) bytes a routed row and the routing, where a forward leaves
 * 6 F + 2 d for moe_backward: a little over a quarter at F = d, a fifth at F = d / 2.  After moe_forward, moe_checkpoint_save copies the routing and the router
 * softmax and quantises the pre-activations; before moe_backward, moe_checkpoint_restore puts
 * them back, rebuilds the hidden rows from them and the dispatched rows from x (the forward's
 * input).  The backward is then that of the layer with the pre-activations as they were kept.
 * moe_checkpoint_bytes: 0 for a plan without MOE_FLAG_TRAINING.  Checkpoint and workspace are
 * 256-byte aligned device memory; both calls are asynchronous on `stream`. */
size_t moe_checkpoint_bytes(moe_plan_t plan);
moe_status moe_checkpoint_save(moe_plan_t plan, const void* workspace, size_t workspace_bytes, void* checkpoint,
                               size_t checkpoint_bytes, void* stream);
moe_status moe_checkpoint_restore(moe_plan_t plan, const void* x, const void* checkpoint, size_t checkpoint_bytes,
                                  void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_FP8_H */
