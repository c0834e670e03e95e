// optim_internal.h -- what the host side of the optimiser's step (api_optim.cu) and its kernels share.
#pragma once
#include "../../include/moe_optim.h"
#include "moe_internal.h"

namespace moe {
namespace optim {

constexpr int kMostTensors = 420;  // of one launch: their list is a kernel argument (32 KB at most)
constexpr int kNormCtas = 152 * 8;
constexpr int64_t kMostValues = (int64_t)1 << 35;  // of a tensor

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int n, const moe_adamw_config& cfg, const float* factor, int64_t* steps,
                         uint32_t* ticket, cudaStream_t st);
cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int n, float max_norm, float* norm, float* factor, void* workspace,
                             cudaStream_t st);

}  // namespace optim
}  // namespace moe
