// quantize.cu -- 8-bit block quantisation (e4m3 with an e8m0 factor per block of 128), of rows
// (1 x 128) and of weights (128 x 128), and the 8-bit activation checkpoints of the SwiGLU.
//
// These kernels read and write each value once and compute a few operations on it: HBM bounds
// them.
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float load_any(const void* p, int bf16, int64_t i) {
  return bf16 ? __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// Rows: a warp takes one block of 128 columns of a row at a time, four columns a lane.
__global__ void __launch_bounds__(kThreads) quantize_rows_kernel(const void* x, int bf16, int64_t rows, int64_t cols,
                                                                 int64_t ldx, uint8_t* q, uint8_t* scales) {
  const int lane = threadIdx.x & 31;
  const int64_t sc = scale_cols(cols);
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < rows * sc; i += (int64_t)gridDim.x * kWarps) {
    const int64_t row = i / sc, blk = i % sc, c0 = blk * kBlock;
    float v[4];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + j * 32 + lane;
      v[j] = c < cols ? load_any(x, bf16, row * ldx + c) : 0.f;
      top = max(top, abs_bits(v[j]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    const uint32_t b = scale_byte(__uint_as_float(top));
    const float f = inv_scale_value(b);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = c0 + j * 32 + lane;
      if (c < cols) q[row * cols + c] = (uint8_t)pack_e4m3x2(v[j] * f, 0.f);
    }
    if (lane == 0) scales[i] = (uint8_t)b;  // a padding byte's block is empty: 0
  }
}

// Weights: one CTA per 128 x 128 block of an expert (x read twice, the second time from L2).
__global__ void __launch_bounds__(kThreads) quantize_blocks_kernel(const void* x, int bf16, int64_t cols, int64_t ldx,
                                                                   int64_t expert_rows, int64_t n_blocks, uint8_t* q,
                                                                   uint8_t* scales) {
  __shared__ uint32_t top_s;
  const int64_t sc = scale_cols(cols), nb = (expert_rows + kBlock - 1) / kBlock;
  for (int64_t i = blockIdx.x; i < n_blocks; i += gridDim.x) {
    const int64_t e = i / (nb * sc), r0 = i / sc % nb * kBlock, c0 = i % sc * kBlock;
    if (threadIdx.x == 0) top_s = 0;
    __syncthreads();
    const int64_t c = c0 + (threadIdx.x & 127);
    uint32_t top = 0;
    for (int64_t r = r0 + (threadIdx.x >> 7); r < r0 + kBlock && r < expert_rows; r += 2)
      if (c < cols) top = max(top, abs_bits(load_any(x, bf16, (e * expert_rows + r) * ldx + c)));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) atomicMax(&top_s, top);
    __syncthreads();
    const uint32_t b = scale_byte(__uint_as_float(top_s));
    const float f = inv_scale_value(b);
    for (int64_t r = r0 + (threadIdx.x >> 7); r < r0 + kBlock && r < expert_rows; r += 2)
      if (c < cols)
        q[(e * expert_rows + r) * cols + c] =
            (uint8_t)pack_e4m3x2(load_any(x, bf16, (e * expert_rows + r) * ldx + c) * f, 0.f);
    if (threadIdx.x == 0) scales[i] = (uint8_t)b;
    __syncthreads();
  }
}

// SwiGLU backward out of the checkpoint; a warp per block of 128 columns of a row.
__global__ void __launch_bounds__(kThreads)
    checkpoint_backward_kernel(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
                               const __nv_bfloat16* dh, int64_t rows, int F, __nv_bfloat16* da, __nv_bfloat16* db,
                               __nv_bfloat16* h) {
  const int lane = threadIdx.x & 31;
  const int64_t sc = scale_cols(F), nb = (F + kBlock - 1) / kBlock;
  for (int64_t i = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); i < rows * nb; i += (int64_t)gridDim.x * kWarps) {
    const int64_t row = i / nb, blk = i % nb;
    const float fa = scale_value(sa[row * sc + blk]), fb = scale_value(sb[row * sc + blk]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t c = blk * kBlock + j * 32 + lane;
      if (c >= F) continue;
      const int64_t o = row * F + c;
      const float a = unpack_e4m3x2(qa[o]).x * fa, b = unpack_e4m3x2(qb[o]).x * fb, g = __bfloat162float(dh[o]);
      const float s = __fdividef(1.f, 1.f + __expf(-a)), u = a * s;
      da[o] = __float2bfloat16_rn(g * b * (s + u * (1.f - s)));
      db[o] = __float2bfloat16_rn(g * u);
      if (h) h[o] = __float2bfloat16_rn(u * b);
    }
  }
}

unsigned grid_for(int64_t work, int64_t per_cta) {
  const int64_t g = (work + per_cta - 1) / per_cta;
  return (unsigned)(g < 1 ? 1 : g > 1 << 20 ? 1 << 20 : g);
}

}  // namespace

cudaError_t launch_quantize_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx, void* q,
                                 uint8_t* scales, cudaStream_t st) {
  return launch_kernel(quantize_rows_kernel, dim3(grid_for(rows * scale_cols(cols), kWarps)), dim3(kThreads), 0, st, false,
                       1, x, bf16 ? 1 : 0, rows, cols, ldx, (uint8_t*)q, scales);
}

cudaError_t launch_quantize_blocks(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                   int64_t expert_rows, void* q, uint8_t* scales, cudaStream_t st) {
  const int64_t n = rows / expert_rows * ((expert_rows + kBlock - 1) / kBlock) * scale_cols(cols);
  return launch_kernel(quantize_blocks_kernel, dim3(grid_for(n, 1)), dim3(kThreads), 0, st, false, 1, x, bf16 ? 1 : 0,
                       cols, ldx, expert_rows, n, (uint8_t*)q, scales);
}

cudaError_t launch_checkpoint_save(const void* a, const void* b, int64_t rows, int F, void* qa, uint8_t* sa, void* qb,
                                   uint8_t* sb, cudaStream_t st) {
  cudaError_t e = launch_quantize_rows(a, true, rows, F, F, qa, sa, st);
  return e != cudaSuccess ? e : launch_quantize_rows(b, true, rows, F, F, qb, sb, st);
}

cudaError_t launch_checkpoint_backward(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                       const void* dh, int64_t rows, int F, void* da, void* db, void* h,
                                       cudaStream_t st) {
  return launch_kernel(checkpoint_backward_kernel, dim3(grid_for(rows * ((F + kBlock - 1) / kBlock), kWarps)),
                       dim3(kThreads), 0, st, false, 1, (const uint8_t*)qa, sa, (const uint8_t*)qb, sb,
                       (const __nv_bfloat16*)dh, rows, F, (__nv_bfloat16*)da, (__nv_bfloat16*)db, (__nv_bfloat16*)h);
}

}  // namespace fp8
}  // namespace moe
