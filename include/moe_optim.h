/*
 * moe_optim.h -- C ABI of the optimiser's step over many tensors (sm_103a): the gradients' norm with the
 * factor that clips it, and AdamW with moments in 32 or in 8 bits.
 *
 * One step of AdamW, with f the clipping factor, t the number of the step (1 the first):
 *   g = f * grad,   m = b1 m + (1 - b1) g,   v = b2 v + (1 - b2) g^2
 *   p = p - lr wd p - lr (m / (1 - b1^t)) / (sqrt(v / (1 - b2^t)) + eps)
 * in fp32, with 1 - lr wd taken to 2^-48; the square root and the quotient are good to two of its steps, and a v below 2^-126 counts as 0 in them.
 * Where (1 - b2) g^2 is 2^128 or more (|g| of 5.8e20 with a b2 of 0.999), v becomes infinite and the parameter may then become NaN.
 * A parameter is fp32; or bf16 with an fp32 master, which the step is taken on and the
 * parameter rounded from (to nearest); or bf16 alone, rounded stochastically.
 *
 * Moments in 8 bits are m and r = sqrt(v), e4m3 values with an e8m0 factor for each 128 consecutive ones of
 * the tensor (the last block may be short), as moe_fp8.h describes the format; they are rounded stochastically
 * too: m to one of its two neighbours with the probability that makes its mean right, r with the one
 * that makes the mean of r^2, that is of v, right.  (v moves by 1 - b2 = 0.1 % a step.  A step from one e4m3
 * value to the next is 6 to 12 %: rounded to nearest, v would stay where it is.)  A v above 0 is never
 * rounded to 0, so that no update is divided by eps alone.
 *
 * The random words are a hash of the seed, t, the tensor's index in the list and the value's index:
 * a step gives the same bits wherever its arrays lie and however it is launched.  With words of 32 bits,
 *   mix(x):  x *= 0x9E3779B1; x ^= x >> 16;  x *= 0x6A09E667; x ^= x >> 15;  x *= 0xBB67AE85; x ^= x >> 16
 *   key = mix(mix(mix(mix(seed_low) + seed_high) + t_low) + tensor)
 *   r_0 = mix(i / 8 + key),  r_{j+1} = r_j * 0x3C6EF375 + 0xA54FF53B,  the word of value i is r_{i mod 8}
 * whose bits 31-16 round m, 23-8 r and 15-0 a bf16 parameter.
 *
 * Conventions are those of moe.h, but that every array needs only the alignment of its type (arrays on
 * 16-byte boundaries are faster) and no two arrays of a call overlap.
 */
#ifndef MOE_OPTIM_H
#define MOE_OPTIM_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* param;         /* n values of param_dtype */
  float* master;       /* n values, or NULL; only with MOE_BF16 */
  const void* grad;    /* n values of grad_dtype */
  void* m;             /* n values: fp32, or e4m3 */
  void* v;             /* n values: v in fp32, or r = sqrt(v) in e4m3 */
  uint8_t* m_scales;   /* NULL: moments in fp32; else ceil(n / 128) bytes */
  uint8_t* v_scales;
  int64_t n;           /* 0 .. 2^35 */
  float weight_decay;  /* >= 0 */
  int32_t param_dtype, grad_dtype; /* moe_dtype */
} moe_adamw_tensor;

typedef struct {
  double lr;              /* >= 0 */
  const float* lr_device; /* NULL, or a device value that is used for lr (a captured step reads it at each replay) */
  double beta1, beta2;    /* [0, 1); 1 - beta is taken in 64 bits */
  double eps;             /* >= 2^-126 */
  uint64_t seed;
} moe_adamw_config;

/* One step over n_tensors tensors.  `steps` (device, 8-byte aligned): the steps taken so far, which the call
 * raises by one.  `ticket` (device): a word that is 0 before the first call and that the calls leave 0;
 * calls in flight at the same time need words of their own.  grad_factor (device, may be NULL: 1) is f;
 * where it is infinite or NaN nothing is changed, steps neither.  The list is read during the call. */
moe_status moe_adamw(const moe_adamw_tensor* tensors, int32_t n_tensors, const moe_adamw_config* cfg,
                     const float* grad_factor, int64_t* steps, uint32_t* ticket, void* stream);

typedef struct {
  const void* grad;
  int64_t n;
  int32_t dtype;
} moe_grad_tensor;

/* Bytes of workspace for moe_grad_norm over n_tensors tensors. */
size_t moe_grad_norm_workspace(int32_t n_tensors);

/* *norm = sqrt(sum over all values g^2) and, where factor is not NULL, *factor = min(1, max_norm / *norm), NaN
 * where the norm is infinite or NaN.  Squares are taken in fp32 (a |g| above 1.8e19 gives an infinite
 * norm, values below 1e-19 count with few bits or not at all), summed in fp32 over 1024 values at most, pairwise,
 * then with 48 bits or more, in an order that the sizes fix; in 64 bits from the squares on where fp32 does not hold a sum.
 * max_norm > 0.  workspace: 256-byte aligned; its first 4 bytes are 0
 * before the first call, and the calls leave them 0.  Calls in flight at the same time need workspaces of their own. */
moe_status moe_grad_norm(const moe_grad_tensor* tensors, int32_t n_tensors, float max_norm, float* norm, float* factor,
                         void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_OPTIM_H */
