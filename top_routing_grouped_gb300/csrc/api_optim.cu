// api_optim.cu -- the C ABI of the optimiser's step (include/moe_optim.h): argument checks and launches.
#include <float.h>
#include <math.h>

#include "host_checks.h"
#include "optim_internal.h"

namespace {

using namespace moe;

moe_status check_count(const void* tensors, int32_t n) {
  if (n < 0 || n > 1 << 20) return fail(MOE_ERR_INVALID_ARG, "n_tensors must be 0 to 2^20");
  if (n > 0 && !tensors) return fail(MOE_ERR_INVALID_ARG, "tensors is null");
  return MOE_OK;
}

moe_status check_tensor(int i, const moe_adamw_tensor& t) {
  if (!is_dtype(t.param_dtype) || !is_dtype(t.grad_dtype)) return fail(MOE_ERR_INVALID_ARG, "tensor %d: bad dtype", i);
  if (t.n < 0 || t.n > optim::kMostValues) return fail(MOE_ERR_INVALID_ARG, "tensor %d: n must be 0 to 2^35", i);
  if (!(t.weight_decay >= 0.f) || !isfinite(t.weight_decay)) return fail(MOE_ERR_INVALID_ARG, "tensor %d: weight_decay must be finite and >= 0", i);
  if (t.master && t.param_dtype != MOE_BF16) return fail(MOE_ERR_INVALID_ARG, "tensor %d: only a bf16 parameter has a master", i);
  if (!t.m_scales != !t.v_scales) return fail(MOE_ERR_INVALID_ARG, "tensor %d: m_scales and v_scales go together", i);
  if (t.n == 0) return MOE_OK;
  if (!t.param || !t.grad || !t.m || !t.v) return fail(MOE_ERR_INVALID_ARG, "tensor %d: an array is null", i);
  const size_t moments = t.m_scales ? 1 : 4;
  if (!aligned(t.param, esize(t.param_dtype)) || !aligned(t.master, 4) || !aligned(t.grad, esize(t.grad_dtype)) || !aligned(t.m, moments) ||
      !aligned(t.v, moments))
    return fail(MOE_ERR_INVALID_ARG, "tensor %d: an array is not aligned to its type", i);
  const size_t n = (size_t)t.n, blocks = (n + 127) / 128;
  const struct {
    const void* p;
    size_t bytes;
    const char* name;
  } a[] = {{t.param, n * esize(t.param_dtype), "param"}, {t.master, n * 4, "master"}, {t.m, n * moments, "m"}, {t.v, n * moments, "v"},
           {t.m_scales, blocks, "m_scales"},             {t.v_scales, blocks, "v_scales"}, {t.grad, n * esize(t.grad_dtype), "grad"}};
  for (int x = 0; x < 7; ++x)
    for (int y = x + 1; y < 7; ++y)
      if (a[x].p && a[y].p && overlap(a[x].p, a[x].bytes, a[y].p, a[y].bytes))
        return fail(MOE_ERR_INVALID_ARG, "tensor %d: %s overlaps %s", i, a[x].name, a[y].name);
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_adamw(const moe_adamw_tensor* tensors, int32_t n_tensors, const moe_adamw_config* cfg, const float* grad_factor,
                     int64_t* steps, uint32_t* ticket, void* stream) {
  moe_status s = check_count(tensors, n_tensors);
  if (s != MOE_OK) return s;
  if (!cfg) return fail(MOE_ERR_INVALID_ARG, "cfg is null");
  if (!(cfg->lr >= 0) || !isfinite((float)cfg->lr)) return fail(MOE_ERR_INVALID_ARG, "lr must be finite and >= 0");
  if (!(cfg->beta1 >= 0 && cfg->beta1 < 1 && cfg->beta2 >= 0 && cfg->beta2 < 1))
    return fail(MOE_ERR_INVALID_ARG, "beta1 and beta2 must be in [0, 1)");
  if (!((float)cfg->eps >= FLT_MIN) || !isfinite((float)cfg->eps)) return fail(MOE_ERR_INVALID_ARG, "eps must be finite and at least 2^-126");
  const Ptr ptrs[] = {{cfg->lr_device, "lr_device", 4, true}, {grad_factor, "grad_factor", 4, true}, {steps, "steps", 8, false},
                      {ticket, "ticket", 4, false}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  for (int32_t i = 0; i < n_tensors; ++i)
    if ((s = check_tensor(i, tensors[i])) != MOE_OK) return s;
  return cuda_status(optim::launch_adamw(tensors, n_tensors, *cfg, grad_factor, steps, ticket, static_cast<cudaStream_t>(stream)),
                     "launching the step");
}

size_t moe_grad_norm_workspace(int32_t n_tensors) {
  if (n_tensors < 0 || n_tensors > 1 << 20) return 0;
  // the ticket, and a sum for each CTA of each launch
  const size_t launches = n_tensors == 0 ? 1 : (size_t)(n_tensors + optim::kMostTensors - 1) / optim::kMostTensors;
  return ((1 + launches * optim::kNormCtas) * sizeof(double) + 255) / 256 * 256;
}

moe_status moe_grad_norm(const moe_grad_tensor* tensors, int32_t n_tensors, float max_norm, float* norm, float* factor, void* workspace,
                         size_t workspace_bytes, void* stream) {
  moe_status s = check_count(tensors, n_tensors);
  if (s != MOE_OK) return s;
  if (!(max_norm > 0.f) || !isfinite(max_norm)) return fail(MOE_ERR_INVALID_ARG, "max_norm must be finite and above 0");
  const Ptr ptrs[] = {{norm, "norm", 4, false}, {factor, "factor", 4, true}};
  if ((s = check(ptrs)) != MOE_OK) return s;
  if (norm == factor) return fail(MOE_ERR_INVALID_ARG, "norm and factor are one value");
  for (int32_t i = 0; i < n_tensors; ++i) {
    const moe_grad_tensor& t = tensors[i];
    if (!is_dtype(t.dtype)) return fail(MOE_ERR_INVALID_ARG, "tensor %d: bad dtype", i);
    if (t.n < 0 || t.n > optim::kMostValues) return fail(MOE_ERR_INVALID_ARG, "tensor %d: n must be 0 to 2^35", i);
    if (t.n > 0 && (!t.grad || !aligned(t.grad, esize(t.dtype)))) return fail(MOE_ERR_INVALID_ARG, "tensor %d: grad is null or not aligned to its type", i);
  }
  const size_t need = moe_grad_norm_workspace(n_tensors);
  if (!workspace || !aligned(workspace, 256)) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (workspace_bytes < need) return fail(MOE_ERR_INVALID_ARG, "workspace too small: %zu < %zu", workspace_bytes, need);
  return cuda_status(optim::launch_grad_norm(tensors, n_tensors, max_norm, norm, factor, workspace,
                                             static_cast<cudaStream_t>(stream)),
                     "launching the norm");
}

}  // extern "C"
