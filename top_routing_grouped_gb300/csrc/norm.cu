// norm.cu -- RMS norm with the residual's addition and an 8-bit output, and its backward.
//
//   r = x + residual (rounded to the stream's type),  n = r * rstd * weight,
//   rstd = 1 / sqrt(mean r^2 + eps);  n goes out in the stream's type and as e4m3 with a factor
//   for every 128 columns, both rounded from fp32
//   backward:  g = dn * weight, xhat = r * rstd,  dx = rstd (g - xhat mean(g xhat)) + dresidual,
//   dweight = sum_t dn xhat
//
// Both read and write each value once: HBM bounds them (one row: the launch does).
#include "device_common.cuh"
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <bool kBf16>
__device__ __forceinline__ float ld(const void* p, int64_t i) {
  if constexpr (kBf16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return reinterpret_cast<const float*>(p)[i];
}
template <bool kBf16>
__device__ __forceinline__ void st(void* p, int64_t i, float v) {
  if constexpr (kBf16)
    reinterpret_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  else
    reinterpret_cast<float*>(p)[i] = v;
}
template <bool kBf16>
__device__ __forceinline__ float rounded(float v) {
  if constexpr (kBf16) return __bfloat162float(__float2bfloat16_rn(v));
  return v;
}

// Sum over the CTA, the same value in every thread, in a fixed order.
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) s += red[w];
  __syncthreads();
  return s;
}

// One CTA per row, the row in shared memory between the sum and the scaling; any d, pitch and
// alignment.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads)
    rmsnorm_kernel(const void* x, const void* residual, const float* weight, int64_t rows, int d, int64_t ldx,
                   int64_t ldr, float eps, void* residual_out, void* out, uint8_t* q, uint8_t* scales, float* rstd) {
  extern __shared__ float row_s[];
  __shared__ float red[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t sc = scale_cols(d);
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    float ss = 0.f;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      float v = ld<kBf16>(x, t * ldx + c);
      if (residual) v = rounded<kBf16>(v + ld<kBf16>(residual, t * ldr + c));
      if (residual_out) st<kBf16>(residual_out, t * d + c, v);
      row_s[c] = v;
      ss += v * v;
    }
    const float inv = 1.f / sqrtf(cta_sum(ss, red) / (float)d + eps);
    if (rstd && threadIdx.x == 0) rstd[t] = inv;
    if (out || q) {
      for (int64_t b = warp; b < sc; b += kWarps) {
        float v[4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t c = b * kBlock + j * 32 + lane;
          v[j] = c < d ? row_s[c] * inv * (weight ? weight[c] : 1.f) : 0.f;
          if (out && c < d) st<kBf16>(out, t * d + c, v[j]);
          top = max(top, abs_bits(v[j]));
        }
        if (q) {
          const uint32_t sb = scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
          const float f = inv_scale_value(sb);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int64_t c = b * kBlock + j * 32 + lane;
            if (c < d) q[t * d + c] = (uint8_t)pack_e4m3x2(v[j] * f, 0.f);
          }
          if (lane == 0) scales[t * sc + b] = (uint8_t)sb;
        }
      }
    }
    __syncthreads();  // row_s is read before the next row overwrites it
  }
}

// CTA p takes rows p, p + P, ...; its sum of dweight stays in shared memory and leaves as one
// row of `parts`, which the second kernel adds in order.
template <bool kBf16, bool kDoutBf16>
__global__ void __launch_bounds__(kThreads)
    rmsnorm_backward_kernel(const void* dout, const void* r, const float* weight, const float* rstd,
                            const void* dresidual, int64_t rows, int d, int64_t ldr, void* dx, float* parts) {
  extern __shared__ float dw_s[];
  __shared__ float red[kWarps];
  if (parts)
    for (int c = threadIdx.x; c < d; c += kThreads) dw_s[c] = 0.f;
  for (int64_t t = blockIdx.x; t < rows; t += gridDim.x) {
    const float inv = rstd[t];
    float dot = 0.f;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      const float xh = ld<kBf16>(r, t * ldr + c) * inv, dn = ld<kDoutBf16>(dout, t * d + c);
      dot += dn * (weight ? weight[c] : 1.f) * xh;
      if (parts) dw_s[c] += dn * xh;
    }
    const float m = cta_sum(dot, red) / (float)d;
    for (int c = threadIdx.x; c < d; c += kThreads) {
      const float xh = ld<kBf16>(r, t * ldr + c) * inv, dn = ld<kDoutBf16>(dout, t * d + c);
      float v = inv * (dn * (weight ? weight[c] : 1.f) - xh * m);
      if (dresidual) v += ld<kBf16>(dresidual, t * d + c);
      st<kBf16>(dx, t * d + c, v);
    }
  }
  if (parts)
    for (int c = threadIdx.x; c < d; c += kThreads) parts[(int64_t)blockIdx.x * d + c] = dw_s[c];
}

__global__ void __launch_bounds__(kThreads) dweight_sum_kernel(const float* parts, int n, int d, float* dweight) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  pdl_wait();
  if (c >= d) return;
  float s = 0.f;
  for (int p = 0; p < n; ++p) s += parts[(int64_t)p * d + c];
  dweight[c] = s;
}

}  // namespace

cudaError_t launch_rmsnorm(const void* x, const void* residual, const float* weight, bool bf16, int64_t rows, int d,
                           int64_t ldx, int64_t ldr, float eps, void* residual_out, void* out, void* q, uint8_t* scales,
                           float* rstd, cudaStream_t st) {
  const size_t smem = (size_t)d * sizeof(float);
  auto kern = bf16 ? rmsnorm_kernel<true> : rmsnorm_kernel<false>;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024 &&  // what a launch may have without asking
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  const int64_t grid = rows < (1 << 20) ? rows : 1 << 20;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), smem, st, false, 1, x, residual, weight, rows, d, ldx,
                       ldr, eps, residual_out, out, (uint8_t*)q, scales, rstd);
}

int rmsnorm_backward_parts(int64_t rows) { return (int)(rows < 304 ? rows : 304); }

cudaError_t launch_rmsnorm_backward(const void* dout, bool dout_bf16, const void* r, const float* weight,
                                    const float* rstd, const void* dresidual, bool bf16, int64_t rows, int d,
                                    int64_t ldr, void* dx, float* dweight, float* parts, cudaStream_t st) {
  const int n = rmsnorm_backward_parts(rows);
  const size_t smem = (size_t)d * sizeof(float);
  auto kern = bf16 ? (dout_bf16 ? rmsnorm_backward_kernel<true, true> : rmsnorm_backward_kernel<true, false>)
                   : (dout_bf16 ? rmsnorm_backward_kernel<false, true> : rmsnorm_backward_kernel<false, false>);
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024 &&  // what a launch may have without asking
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) != cudaSuccess)
    return e;
  if (n > 0) {
    e = launch_kernel(kern, dim3((unsigned)n), dim3(kThreads), smem, st, false, 1, dout, r, weight, rstd, dresidual, rows,
                      d, ldr, dx, dweight ? parts : nullptr);
    if (e != cudaSuccess) return e;
  }
  if (!dweight) return cudaSuccess;
  return launch_kernel(dweight_sum_kernel, dim3((unsigned)((d + kThreads - 1) / kThreads)), dim3(kThreads), 0, st, n > 0, 1,
                       (const float*)parts, n, d, dweight);
}

}  // namespace fp8
}  // namespace moe
