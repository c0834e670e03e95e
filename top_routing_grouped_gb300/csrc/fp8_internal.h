// fp8_internal.h -- what the host side of the 8-bit operators (api_fp8.cu) and their kernels
// share.
#pragma once
#include "../../include/moe_fp8.h"
#include "moe_internal.h"

namespace moe {
namespace fp8 {

constexpr int kBlock = 128;  // values per scale
constexpr uint64_t kMinTimeoutNs = 1000000;  // the shortest limit of a device-side wait
constexpr int kMaxNormCols = 49152;  // the widest row that the norms hold in shared memory
__host__ __device__ inline int64_t scale_cols(int64_t cols) { return (cols + 511) / 512 * 4; }

// One grouped product as its kernels see it.
struct GemmArgs {
  const uint8_t* a;     // [rows, K] e4m3
  const uint8_t* sa;    // [rows, scale_cols(K)]
  const uint8_t* b;     // [E, n, K] (SwiGLU: W1)
  const uint8_t* sb;    // [E, ceil(n/128), scale_cols(K)]
  const uint8_t* b3;    // SwiGLU: W3 and its scales
  const uint8_t* sb3;
  const float* gate;    // [rows] factor of each output row, or null
  void* out;            // [rows, n]: bf16 or fp32; SwiGLU: e4m3
  uint8_t* out_scales;  // SwiGLU: [rows, scale_cols(n)]
  int64_t rows;         // capacity of the row buffers
  int n, K, E;
};
enum : int { kSwiGLU = 1, kOutBf16 = 2, kOutF32 = 3 };

cudaError_t launch_quantize_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx, void* q,
                                 uint8_t* scales, cudaStream_t st);
cudaError_t launch_quantize_blocks(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                   int64_t expert_rows, void* q, uint8_t* scales, cudaStream_t st);
cudaError_t launch_checkpoint_save(const void* a, const void* b, int64_t rows, int F, void* qa, uint8_t* sa, void* qb,
                                   uint8_t* sb, cudaStream_t st);
cudaError_t launch_checkpoint_backward(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                       const void* dh, int64_t rows, int F, void* da, void* db, void* h,
                                       cudaStream_t st);

cudaError_t launch_checkpoint_restore(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb, int64_t rows,
                                      int F, void* a, void* b, void* h, cudaStream_t st);

cudaError_t launch_rmsnorm(const void* x, const void* residual, const float* weight, bool bf16, int64_t rows, int d,
                           int64_t ldx, int64_t ldr, float eps, void* residual_out, void* out, void* q, uint8_t* scales,
                           float* rstd, cudaStream_t st);
int rmsnorm_backward_parts(int64_t rows, int d);  // partial sums of dweight
cudaError_t launch_rmsnorm_backward(const void* dout, bool dout_bf16, const void* r, const float* weight,
                                    const float* rstd, const void* dresidual, bool bf16, int64_t rows, int d,
                                    int64_t ldr, void* dx, float* dweight, float* parts, cudaStream_t st);

// MOE_PATH_SIMT: segment counts (null: one segment of s.N rows) -> tile tables; clears the status
// word first.
cudaError_t launch_segments(const Shape& s, const Ws& ws, const int32_t* seg_counts, int n_seg, int n_experts,
                            cudaStream_t st);
// Dispatch of 8-bit rows x [T, d] with their factors xs into ws.xp and xs_out.
cudaError_t launch_permute(const Shape& s, const Ws& ws, const void* x, const uint8_t* xs, uint8_t* xs_out, int num_sms,
                           bool pdl, cudaStream_t st);
cudaError_t launch_gemm_simt(int kind, const GemmArgs& g, const Ws& ws, int num_sms, cudaStream_t st);
// The tensor-core products find their tiles from the segment counts themselves (null: one segment);
// `first`: the call's first launch, which sets the status word and waits for all earlier kernels before it
// reads anything.  The others read the counts before they wait, and the weights; a's rows and factors
// and the gates after it, whichever earlier kernel of the call writes them.
cudaError_t launch_gemm_tc(int kind, const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first,
                           int device, int num_sms, int64_t timeout_ns, cudaStream_t st);
// Which of the two sets of tensor-core kernels: see api_fp8.cu.
bool use_few(int64_t rows, int64_t n_seg, int64_t widest_out);
// ... for few rows an expert.
cudaError_t launch_gemm_few(int kind, const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first,
                            int device, int num_sms, int64_t timeout_ns, cudaStream_t st);

}  // namespace fp8
}  // namespace moe
