// gemm_fp8_simt.cu -- the 8-bit grouped products in fp32 FMA (MOE_PATH_SIMT): any size, and the
// cross-check of the tensor-core kernels.  An e4m3 times its power of two is exact in fp32, as is
// the product of two; the sums are fp32 in ascending k.
//
// SiLU is silu_exact here, not the tensor-core kernels' shorter form.
//
// A CTA computes 32 rows x 128 columns (SwiGLU: of both products, so that a row's block of 128
// hidden values, which shares a factor, lies in one warp): lane l of warp w has rows 4w..4w+3 and
// columns l, l + 32, l + 64, l + 96.
#include "device_common.cuh"
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 32, kCols = 128, kBK = 32;

template <int kKind>
__global__ void __launch_bounds__(kThreads) gemm_fp8_simt_kernel(GemmArgs g, Ws ws) {
  __shared__ float a_s[kRows][kBK + 1];
  __shared__ float b_s[kKind == kSwiGLU ? 2 : 1][kCols][kBK + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_tiles = (g.n + kCols - 1) / kCols;
  const int64_t sck = scale_cols(g.K), scn = scale_cols(g.n), nb = (g.n + kBlock - 1) / kBlock;
  pdl_wait();
  pdl_launch_dependents();
  const int total = (int)ws.hdr[kHdrNumMTiles] * n_tiles;
  for (int64_t u = blockIdx.x; u < (int64_t)total * (kTileM / kRows); u += gridDim.x) {
    TileInfo ti = decode_tile(ws, n_tiles, (int)(u / (kTileM / kRows)));
    const int sub = (int)(u % (kTileM / kRows)) * kRows;
    const int valid = ti.rows - sub;
    if (valid <= 0) continue;  // the same for the whole CTA
    const int64_t row0 = (int64_t)ti.row0 + sub;
    const int n0 = ti.n_idx * kCols;
    float acc[kKind == kSwiGLU ? 2 : 1][4][4] = {};
    for (int k0 = 0; k0 < g.K; k0 += kBK) {
      const int kb = k0 / kBlock;
      for (int i = threadIdx.x; i < kRows * kBK; i += kThreads) {
        const int r = i / kBK, k = k0 + i % kBK;
        float v = 0.f;
        if (r < valid && k < g.K) v = unpack_e4m3x2(g.a[(row0 + r) * g.K + k]).x * scale_value(g.sa[(row0 + r) * sck + kb]);
        a_s[r][i % kBK] = v;
      }
      for (int i = threadIdx.x; i < kCols * kBK; i += kThreads) {
        const int c = n0 + i / kBK, k = k0 + i % kBK;
        const bool in = c < g.n && k < g.K;
        const int64_t o = ((int64_t)ti.e * g.n + c) * g.K + k, so = ((int64_t)ti.e * nb + c / kBlock) * sck + kb;
        b_s[0][i / kBK][i % kBK] = in ? unpack_e4m3x2(g.b[o]).x * scale_value(g.sb[so]) : 0.f;
        if constexpr (kKind == kSwiGLU)
          b_s[1][i / kBK][i % kBK] = in ? unpack_e4m3x2(g.b3[o]).x * scale_value(g.sb3[so]) : 0.f;
      }
      __syncthreads();
      for (int k = 0; k < kBK; ++k) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = a_s[4 * warp + i][k];
#pragma unroll
        for (int m = 0; m < (kKind == kSwiGLU ? 2 : 1); ++m)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float b = b_s[m][lane + 32 * j][k];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i][j] = fmaf(a[i], b, acc[m][i][j]);
          }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool row_ok = 4 * warp + i < valid;
      const int64_t p = row0 + 4 * warp + i;
      if constexpr (kKind == kSwiGLU) {
        float h[4];
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          h[j] = n0 + lane + 32 * j < g.n ? silu_exact(acc[0][i][j]) * acc[1][i][j] : 0.f;
          top = max(top, abs_bits(h[j]));
        }
        const uint32_t sb = scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
        const float f = inv_scale_value(sb);
        if (row_ok) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n0 + lane + 32 * j < g.n)
              reinterpret_cast<uint8_t*>(g.out)[p * g.n + n0 + lane + 32 * j] = (uint8_t)pack_e4m3x2(h[j] * f, 0.f);
          if (lane == 0) g.out_scales[p * scn + n0 / kBlock] = (uint8_t)sb;
        }
      } else if (row_ok) {
        const float gate = g.gate ? g.gate[p] : 1.f;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n0 + lane + 32 * j < g.n) store_act(g.out, kKind == kOutBf16, p * g.n + n0 + lane + 32 * j, gate * acc[0][i][j]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_gemm_simt(int kind, const GemmArgs& g, const Ws& ws, int num_sms, cudaStream_t st) {
  auto kern = kind == kSwiGLU ? gemm_fp8_simt_kernel<kSwiGLU>
              : kind == kOutBf16 ? gemm_fp8_simt_kernel<kOutBf16> : gemm_fp8_simt_kernel<kOutF32>;
  return launch_kernel(kern, dim3((unsigned)num_sms * 4), dim3(kThreads), 0, st, true, 1, g, ws);
}

}  // namespace fp8
}  // namespace moe
