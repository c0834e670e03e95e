// norm.cu -- RMS norm with the residual's addition and an 8-bit output, and its backward.
//
//   r = x + residual (rounded to the stream's type),  n = r * rstd * weight,
//   rstd = 1 / sqrt(mean r^2 + eps);  n goes out in the stream's type and as e4m3 with a factor
//   for every 128 columns, both rounded from fp32
//   backward:  g = dn * weight, xhat = r * rstd,  dx = rstd (g - xhat mean(g xhat)) + dresidual,
//   dweight = sum_t dn xhat
//
// Both read and write each value once: HBM bounds them (one row: the launch does).  32768 x 4096 bf16
// with residual, bf16 and e4m3 outputs: 192 us, 6.3 TB/s; backward from fp32 gradients: 201 us, 6.7
// TB/s; one row of 4096: 2.1 us.  By width (2^25 values, bf16, residual; forward / backward in TB/s): 1000 to 4096
// columns 5.0-6.2 / 5.8-6.0 (2500: 5.4 / 3.8), 4100 to 8192 3.9-5.6 / 4.6-5.2 (one CTA of 288 to 512 threads an
// SM), off whole pairs 2.1 / 1.8 at 257 and 3.3 / 2.7 at 2001, 64 and 128 columns 2.0-3.9 / 2.4-4.4, and past 8192,
// where a row goes through shared memory in single values, 1.5 / 0.8 at 12288 and 1.1 / 0.8 at 16384.
//
// A row is held in registers by W warps, eight values a thread and piece, V pieces a thread; the
// CTAs are persistent and a row's loads are issued before the row before it is reduced, so the
// loads of one row run under the reduction and the stores of another.  Rows of whole 16-byte
// vectors give a thread 8 consecutive columns (kVec); others give it four pairs of columns 64 apart,
// so that a warp's loads and stores of a pair (of single values, where the width is odd) still
// touch consecutive addresses.
#include "device_common.cuh"
#include "fp8_common.cuh"
#include "fp8_vec.cuh"

#include <string.h>

#include <atomic>

namespace moe {
namespace fp8 {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRegCols = 8192;  // 512 threads, two pieces each

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

// ---------------------------------------------------------------- rows in registers

// Columns of piece u of this thread: kVec: first(u) .. first(u) + 7; else four pairs, two in each of
// two blocks of 128.
template <bool kVec>
struct Cols {
  int W, warp, lane;  // warps of a row, this one among them
  bool even;          // not kVec: pairs lie on whole pairs in memory
  __device__ __forceinline__ int first(int u) const {
    return kVec ? ((u * W + warp) * 32 + lane) * 8 : (u * W + warp) * 256 + 2 * lane;
  }
  __device__ __forceinline__ int col(int u, int j) const { return first(u) + (kVec ? j : 64 * (j / 2) + (j & 1)); }
};

// Eight values of a row as they lie in memory.
template <bool kBf16, bool kVec>
struct Piece {
  uint32_t w[kBf16 ? 4 : 8];  // bf16: two to a word
  __device__ __forceinline__ void load(const void* row, const Cols<kVec>& cs, int u, int d) {
    if constexpr (kVec) {
      const int c = cs.first(u);
      Raw8<kBf16> r;
      if (c < d) r.load(row, c);
      else r.zero();
      memcpy(w, r.w, sizeof w);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = cs.col(u, 2 * j);
        if constexpr (kBf16) {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(row) + c;
          if (cs.even)
            w[j] = c < d ? *reinterpret_cast<const uint32_t*>(p) : 0u;
          else
            w[j] = (c < d ? p[0] : 0u) | (c + 1 < d ? (uint32_t)p[1] << 16 : 0u);
        } else {
          const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + c;
          if (cs.even) {
            const uint2 v = c < d ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
            w[2 * j] = v.x;
            w[2 * j + 1] = v.y;
          } else {
            w[2 * j] = c < d ? p[0] : 0u;
            w[2 * j + 1] = c + 1 < d ? p[1] : 0u;
          }
        }
      }
    }
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (kBf16) return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    return __uint_as_float(w[j]);
  }
};

template <bool kBf16, bool kVec>
__device__ __forceinline__ void store8(void* row, const Cols<kVec>& cs, int u, int d, const float (&v)[8]) {
  if constexpr (kVec) {
    const int c = cs.first(u);
    if (c >= d) return;
    if constexpr (kBf16) {
      *reinterpret_cast<uint4*>(reinterpret_cast<__nv_bfloat16*>(row) + c) = pack_bf16x8(v);
    } else {
      float4* o = reinterpret_cast<float4*>(reinterpret_cast<float*>(row) + c);
      o[0] = make_float4(v[0], v[1], v[2], v[3]);
      o[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const int c = cs.col(u, j);
      if (cs.even) {
        if (c >= d) continue;
        if constexpr (kBf16)
          *reinterpret_cast<__nv_bfloat162*>(reinterpret_cast<__nv_bfloat16*>(row) + c) = __floats2bfloat162_rn(v[j], v[j + 1]);
        else
          *reinterpret_cast<float2*>(reinterpret_cast<float*>(row) + c) = make_float2(v[j], v[j + 1]);
      } else {
        if (c < d) st<kBf16>(row, c, v[j]);
        if (c + 1 < d) st<kBf16>(row, c + 1, v[j + 1]);
      }
    }
  }
}

// The weight is on a 16-byte boundary whatever the rows are on.
template <bool kVec>
__device__ __forceinline__ void load_weight(const float* weight, const Cols<kVec>& cs, int u, int d, float (&v)[8]) {
  if (!weight) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 1.f;
    return;
  }
  Cols<kVec> c = cs;
  c.even = (d & 1) == 0;
  Piece<false, kVec> p;
  p.load(weight, c, u, d);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = p.get(j);
}

// Sum over the row's W <= 16 warps, the same bits in every thread.  `red` [2][16], zero where no warp
// writes: calls take turns (`turn`), so one barrier a call is enough.
__device__ __forceinline__ float row_sum(float v, float* red, int turn, int W, int warp, int lane) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (W > 1) {
    red += turn * 16;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    const float4* r4 = reinterpret_cast<const float4*>(red);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 x = r4[w];
      v += (x.x + x.y) + (x.z + x.w);
    }
  }
  return v;
}

// R = 1: a row a CTA; R > 1: a row a warp.
template <bool kBf16, bool kVec, int V, int R>
__global__ void __launch_bounds__(R > 1 ? 32 * R : 512)
    rmsnorm_reg_kernel(const void* x, const void* residual, const float* weight, int64_t rows, int d, int64_t ldx,
                       int64_t ldr, float eps, void* residual_out, void* out, uint8_t* q, uint8_t* scales, float* rstd, int even) {
  __shared__ __align__(16) float red[2 * 16];
  if (R == 1) {
    if (threadIdx.x < 32) red[threadIdx.x] = 0.f;
    __syncthreads();
  }
  constexpr int kEsz = kBf16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const Cols<kVec> cs{R > 1 ? 1 : (int)(blockDim.x >> 5), R > 1 ? 0 : (int)(threadIdx.x >> 5), lane, even != 0};
  const int64_t sc = scale_cols(d), step = (int64_t)gridDim.x * R;
  const int nb = (d + kBlock - 1) / kBlock;
  pdl_wait();  // an earlier kernel may write any of the inputs
  float wt[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u) load_weight(weight, cs, u, d, wt[u]);
  Piece<kBf16, kVec> px[V], pr[V];
  auto fetch = [&](int64_t t) {
    const char* xr = reinterpret_cast<const char*>(x) + t * ldx * kEsz;
    const char* rr = reinterpret_cast<const char*>(residual) + t * ldr * kEsz;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      px[u].load(xr, cs, u, d);
      if (residual) pr[u].load(rr, cs, u, d);
    }
  };
  int64_t t = (int64_t)blockIdx.x * R + (R > 1 ? threadIdx.x >> 5 : 0);
  if (t < rows) fetch(t);
  for (int turn = 0; t < rows; t += step, turn ^= 1) {
    float v[V][8];
    float ss = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[u][j] = px[u].get(j);
        if (residual) v[u][j] = rounded<kBf16>(v[u][j] + pr[u].get(j));
        ss += v[u][j] * v[u][j];  // zero past the row's end
      }
    }
    if (t + step < rows) fetch(t + step);
    if (residual_out) {
      char* ro = reinterpret_cast<char*>(residual_out) + t * d * kEsz;
#pragma unroll
      for (int u = 0; u < V; ++u) store8<kBf16>(ro, cs, u, d, v[u]);
    }
    const float inv = 1.f / sqrtf(row_sum(ss, red, turn, cs.W, cs.warp, lane) / (float)d + eps);
    if (rstd && cs.warp == 0 && lane == 0) rstd[t] = inv;
    if (!out && !q) continue;
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[u][j] = v[u][j] * inv * wt[u][j];
    if (out) {
      char* o = reinterpret_cast<char*>(out) + t * d * kEsz;
#pragma unroll
      for (int u = 0; u < V; ++u) store8<kBf16>(o, cs, u, d, v[u]);
    }
    if (!q) continue;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      if constexpr (kVec) {
        uint32_t top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, abs_bits(cs.first(u) < d ? v[u][j] : 0.f));
        const uint32_t b = scale_byte(__uint_as_float(half_warp_max(top)));
        const float f = inv_scale_value(b);
        const int c = cs.first(u);
        if (c < d) {
          *reinterpret_cast<uint2*>(q + t * d + c) = make_uint2(pack_e4m3x4(v[u][0] * f, v[u][1] * f, v[u][2] * f, v[u][3] * f),
                                                                pack_e4m3x4(v[u][4] * f, v[u][5] * f, v[u][6] * f, v[u][7] * f));
          if ((lane & 15) == 0) scales[t * sc + c / kBlock] = (uint8_t)b;
        }
      } else {
#pragma unroll
        for (int hb = 0; hb < 2; ++hb) {  // the piece's two blocks
          uint32_t top = 0;
#pragma unroll
          for (int j = 4 * hb; j < 4 * hb + 4; ++j) top = max(top, abs_bits(cs.col(u, j) < d ? v[u][j] : 0.f));
          const uint32_t b = scale_byte(__uint_as_float(__reduce_max_sync(0xffffffffu, top)));
          const float f = inv_scale_value(b);
#pragma unroll
          for (int j = 4 * hb; j < 4 * hb + 4; j += 2) {
            const int cc = cs.col(u, j);
            const uint32_t e2 = pack_e4m3x2(v[u][j] * f, v[u][j + 1] * f);
            uint8_t* o = q + t * d + cc;
            if (cs.even) {
              if (cc < d) *reinterpret_cast<uint16_t*>(o) = (uint16_t)e2;
            } else {
              if (cc < d) o[0] = (uint8_t)e2;
              if (cc + 1 < d) o[1] = (uint8_t)(e2 >> 8);
            }
          }
          const int blk = (u * cs.W + cs.warp) * 2 + hb;
          if (lane == 0 && blk < nb) scales[t * sc + blk] = (uint8_t)b;
        }
      }
    }
    if (cs.warp == 0 && lane < sc - nb) scales[t * sc + nb + lane] = 0;  // the row's padding bytes
  }
}

// dweight of 32 columns over all rows by one CTA: a warp takes every nth row, the warps' sums are
// added in order.
template <bool kBf16, bool kDoutBf16>
__device__ __forceinline__ void column_sums(const void* dout, const void* r, const float* rstd, int rows, int d, int64_t ldr,
                                            int c0, float* dweight, float (*all)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5, c = c0 + lane;
  float s = 0.f;
  if (c < d) {
#pragma unroll 8
    for (int t = warp; t < rows; t += n)
      s += ld<kDoutBf16>(dout, (int64_t)t * d + c) * (ld<kBf16>(r, t * ldr + c) * rstd[t]);
  }
  all[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    s = all[0][lane];
    for (int w = 1; w < n; ++w) s += all[w][lane];
    dweight[c] = s;
  }
}

// The CTA's sum of dweight stays in registers over its rows and leaves as one row of `parts`.  With
// few rows (`parts` null) the CTAs past the first `row_ctas` sum the columns instead, out of L2, and
// the call needs no second kernel.
template <bool kBf16, bool kDoutBf16, bool kVec, int V, int R>
__global__ void __launch_bounds__(R > 1 ? 32 * R : 512, kBf16 && kVec && V == 1 ? (R > 1 ? 4 : 2) : 1)
    rmsnorm_backward_reg_kernel(const void* dout, const void* r, const float* weight, const float* rstd,
                                const void* dresidual, int64_t rows, int d, int64_t ldr, void* dx, float* parts, int even,
                                int row_ctas, float* dweight) {
  __shared__ __align__(16) float red[2 * 16];
  if (R == 1) {
    if (threadIdx.x < 32) red[threadIdx.x] = 0.f;
    __syncthreads();
  }
  constexpr int kEsz = kBf16 ? 2 : 4, kDsz = kDoutBf16 ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const Cols<kVec> cs{R > 1 ? 1 : (int)(blockDim.x >> 5), R > 1 ? 0 : (int)(threadIdx.x >> 5), lane, even != 0};
  const int64_t step = (int64_t)row_ctas * R;
  pdl_wait();
  pdl_launch_dependents();
  if (blockIdx.x >= row_ctas) {
    __shared__ float all[16][32];
    column_sums<kBf16, kDoutBf16>(dout, r, rstd, (int)rows, d, ldr, ((int)blockIdx.x - row_ctas) * 32, dweight, all);
    return;
  }
  float wt[V][8], dw[V][8];
#pragma unroll
  for (int u = 0; u < V; ++u) {
    load_weight(weight, cs, u, d, wt[u]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[u][j] = 0.f;
  }
  Piece<kDoutBf16, kVec> pd[V];
  Piece<kBf16, kVec> pr[V], ps[V];
  float inv = 0.f;
  auto fetch = [&](int64_t t) {
#pragma unroll
    for (int u = 0; u < V; ++u) {
      pd[u].load(reinterpret_cast<const char*>(dout) + t * d * kDsz, cs, u, d);
      pr[u].load(reinterpret_cast<const char*>(r) + t * ldr * kEsz, cs, u, d);
      if (dresidual) ps[u].load(reinterpret_cast<const char*>(dresidual) + t * d * kEsz, cs, u, d);
    }
    inv = rstd[t];
  };
  int64_t t = (int64_t)blockIdx.x * R + (R > 1 ? threadIdx.x >> 5 : 0);
  if (t < rows) fetch(t);
  for (int turn = 0; t < rows; t += step, turn ^= 1) {
    // the row stays packed as it was loaded: unpacked twice it costs fewer registers than kept as
    // fp32, and two CTAs of 512 threads fit an SM
    Piece<kDoutBf16, kVec> cd[V];
    Piece<kBf16, kVec> cr[V], cres[V];
    const float iv = inv;
    float dot = 0.f;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      cd[u] = pd[u];
      cr[u] = pr[u];
      cres[u] = ps[u];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dx_hat = cd[u].get(j) * (cr[u].get(j) * iv);
        dw[u][j] += dx_hat;
        dot += dx_hat * wt[u][j];
      }
    }
    if (t + step < rows) fetch(t + step);
    const float m = row_sum(dot, red, turn, cs.W, cs.warp, lane) / (float)d;
    char* o = reinterpret_cast<char*>(dx) + t * d * kEsz;
#pragma unroll
    for (int u = 0; u < V; ++u) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[j] = iv * (cd[u].get(j) * wt[u][j] - cr[u].get(j) * iv * m);
        if (dresidual) v[j] += cres[u].get(j);
      }
      store8<kBf16>(o, cs, u, d, v);
    }
  }
  if (!parts) return;
  if constexpr (R > 1) {  // the CTA's R rows (one warp each, V = 1) in order
    __shared__ float all[R][256];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = cs.col(0, j);
      if (c < 256) all[threadIdx.x >> 5][c] = dw[0][j];
    }
    __syncthreads();
    for (int c = threadIdx.x; c < d; c += 32 * R) {
      float a = 0.f;
#pragma unroll
      for (int w = 0; w < R; ++w) a += all[w][c];
      parts[(int64_t)blockIdx.x * d + c] = a;
    }
  } else {
    float* o = parts + (int64_t)blockIdx.x * d;
#pragma unroll
    for (int u = 0; u < V; ++u)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (cs.col(u, j) < d) o[cs.col(u, j)] = dw[u][j];
  }
}

// ---------------------------------------------------------------- rows too long for registers

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

// dweight[c] = the n partial sums of column c: 32 columns a CTA, each of its 32 warps a
// thirty-second of the parts in order, then the 32 in order.
__global__ void __launch_bounds__(1024) dweight_sum_kernel(const float* parts, int n, int d, float* dweight) {
  __shared__ float all[32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
  pdl_wait();
  float s = 0.f;
  if (c < d) {
    const int end = (int)((int64_t)n * (warp + 1) / 32);
#pragma unroll 8
    for (int p = (int)((int64_t)n * warp / 32); p < end; ++p) s += parts[(int64_t)p * d + c];
  }
  all[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += all[w][lane];
    dweight[c] = s;
  }
}

}  // namespace

// Threads of a CTA for a row of d columns held in registers: a warp for every 256 columns, two pieces
// a thread above 4096.
static int pieces(int d) { return d <= 4096 ? 1 : 2; }
static int row_threads(int d) {
  if (d <= 256) return 256;  // eight rows of a warp each
  const int per_warp = 256 * pieces(d);
  return (d + per_warp - 1) / per_warp * 32;
}

// Persistent CTAs: what 152 SMs hold of them at 64 registers a thread, 128 with two pieces.  The forward's kernels
// and the backward's for bf16 on whole vectors have that (60 to 70; with two pieces 96 to 126); the other backward kernels
// take 87 to 113 with one piece, so that part of their grid waits for the rest.
static int resident(int d) {
  const int threads = row_threads(d), most = pieces(d) == 1 ? 1024 : 512;
  return 152 * (most / threads);
}

struct NormArgs {
  const void *x, *residual;
  const float* weight;
  int64_t rows;
  int d;
  int64_t ldx, ldr;
  float eps;
  void *residual_out, *out;
  uint8_t *q, *scales;
  float* rstd;
};

template <bool kBf16, bool kVec, int V, int R>
static cudaError_t norm_reg(const NormArgs& a, bool even, cudaStream_t st) {
  const int threads = row_threads(a.d);
  const int64_t want = (a.rows + R - 1) / R;
  const int64_t grid = want < resident(a.d) ? want : resident(a.d);
  return launch_kernel(rmsnorm_reg_kernel<kBf16, kVec, V, R>, dim3((unsigned)grid), dim3(threads), 0, st, true, 1, a.x,
                       a.residual, a.weight, a.rows, a.d, a.ldx, a.ldr, a.eps, a.residual_out, a.out, a.q, a.scales, a.rstd,
                       even ? 1 : 0);
}

template <bool kBf16, bool kVec>
static cudaError_t norm_width(const NormArgs& a, bool even, cudaStream_t st) {
  if (a.d <= 256) return norm_reg<kBf16, kVec, 1, 8>(a, even, st);
  return pieces(a.d) == 1 ? norm_reg<kBf16, kVec, 1, 1>(a, even, st) : norm_reg<kBf16, kVec, 2, 1>(a, even, st);
}

// Rows that lie on whole groups of `n` values (8: vectors, 2: pairs); a missing tensor does.
static bool on(int n, const void* p, bool bf16, int64_t ld) {
  const int per = n == 8 && !bf16 ? 4 : n;  // eight fp32 are two vectors
  return !p || (reinterpret_cast<uintptr_t>(p) % (per * (bf16 ? 2 : 4)) == 0 && ld % per == 0);
}

// Lets a kernel that keeps a row in shared memory have as much of it as the widest row takes.  Set to that
// once per kernel and device and never lowered: the attribute belongs to the process, and another thread may
// stand between a call that has set its own row's size and its launch.
template <typename Kern>
static cudaError_t allow_widest_row(Kern kern, std::atomic<uint64_t>& asked) {
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return e;
  const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
  if (bit && (asked.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxNormCols * (int)sizeof(float));
  if (e == cudaSuccess) asked.fetch_or(bit, std::memory_order_release);
  return e;
}

cudaError_t launch_rmsnorm(const void* x, const void* residual, const float* weight, bool bf16, int64_t rows, int d,
                           int64_t ldx, int64_t ldr, float eps, void* residual_out, void* out, void* q, uint8_t* scales,
                           float* rstd, cudaStream_t st) {
  if (d <= kMaxRegCols) {
    const NormArgs a{x, residual, weight, rows, d, ldx, ldr, eps, residual_out, out, (uint8_t*)q, scales, rstd};
    auto all = [&](int n) {
      return d % n == 0 && on(n, x, bf16, ldx) && on(n, residual, bf16, ldr) && on(n, residual_out, bf16, d) && on(n, out, bf16, d);
    };
    const bool vec = all(8), even = all(2);
    return bf16 ? (vec ? norm_width<true, true>(a, even, st) : norm_width<true, false>(a, even, st))
                : (vec ? norm_width<false, true>(a, even, st) : norm_width<false, false>(a, even, st));
  }
  const size_t smem = (size_t)d * sizeof(float);
  auto kern = bf16 ? rmsnorm_kernel<true> : rmsnorm_kernel<false>;
  static std::atomic<uint64_t> asked[2];
  const cudaError_t e = allow_widest_row(kern, asked[bf16]);
  if (e != cudaSuccess) return e;
  const int64_t grid = rows < (1 << 20) ? rows : 1 << 20;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), smem, st, false, 1, x, residual, weight, rows, d, ldx,
                       ldr, eps, residual_out, out, (uint8_t*)q, scales, rstd);
}

// Up to this many rows, a call is one kernel: the columns' sums read the rows again, from L2 (300 x 1000
// fp32: 4.6 us; with partial sums and a second kernel 5.5 us, and 2 us more of the host's).
constexpr int kOneKernelRows = 512;
static bool one_kernel(int64_t rows, int d) { return rows <= kOneKernelRows && d <= kMaxRegCols; }

// Rows a CTA sums dweight over before it writes a partial: enough CTAs to fill the GPU, but
// partials of a few rows each at least, which are written and read again.  The count depends on
// the shape alone, and so does the order of the sum.
static int row_ctas(int64_t rows, int d) {
  const int per_cta = d <= 256 ? 8 : 1;
  const int64_t most = d <= kMaxRegCols ? resident(d) : 152 * 2;
  const int64_t want = (rows + 2 * per_cta - 1) / (2 * per_cta);
  return (int)(want < most ? want : most);
}
int rmsnorm_backward_parts(int64_t rows, int d) { return one_kernel(rows, d) ? 0 : row_ctas(rows, d); }

struct NormBwdArgs {
  const void *dout, *r;
  const float *weight, *rstd;
  const void* dresidual;
  int64_t rows;
  int d;
  int64_t ldr;
  void* dx;
  int ctas;        // those that take rows
  float* parts;    // more rows: partial sums
  float* dweight;  // few rows: the sums
};

template <bool kBf16, bool kDoutBf16, bool kVec, int V, int R>
static cudaError_t norm_bwd_reg(const NormBwdArgs& a, bool even, cudaStream_t st) {
  const int cols = a.dweight ? (a.d + 31) / 32 : 0;
  return launch_kernel(rmsnorm_backward_reg_kernel<kBf16, kDoutBf16, kVec, V, R>, dim3((unsigned)(a.ctas + cols)),
                       dim3(row_threads(a.d)), 0, st, true, 1, a.dout, a.r, a.weight, a.rstd, a.dresidual, a.rows, a.d, a.ldr,
                       a.dx, a.parts, even ? 1 : 0, a.ctas, a.dweight);
}

template <bool kBf16, bool kDoutBf16, bool kVec>
static cudaError_t norm_bwd_width(const NormBwdArgs& a, bool even, cudaStream_t st) {
  if (a.d <= 256) return norm_bwd_reg<kBf16, kDoutBf16, kVec, 1, 8>(a, even, st);
  return pieces(a.d) == 1 ? norm_bwd_reg<kBf16, kDoutBf16, kVec, 1, 1>(a, even, st)
                          : norm_bwd_reg<kBf16, kDoutBf16, kVec, 2, 1>(a, even, st);
}

template <bool kVec>
static cudaError_t norm_bwd_types(const NormBwdArgs& a, bool bf16, bool dout_bf16, bool even, cudaStream_t st) {
  return bf16 ? (dout_bf16 ? norm_bwd_width<true, true, kVec>(a, even, st) : norm_bwd_width<true, false, kVec>(a, even, st))
              : (dout_bf16 ? norm_bwd_width<false, true, kVec>(a, even, st) : norm_bwd_width<false, false, kVec>(a, even, st));
}

cudaError_t launch_rmsnorm_backward(const void* dout, bool dout_bf16, const void* r, const float* weight,
                                    const float* rstd, const void* dresidual, bool bf16, int64_t rows, int d,
                                    int64_t ldr, void* dx, float* dweight, float* parts, cudaStream_t st) {
  const int n = row_ctas(rows, d);
  const bool one = one_kernel(rows, d);
  cudaError_t e = cudaSuccess;
  if (n > 0 && d <= kMaxRegCols) {
    NormBwdArgs a{dout, r, weight, rstd, dresidual, rows, d, ldr, dx, n, dweight && !one ? parts : nullptr,
                  one ? dweight : nullptr};
    auto all = [&](int k) {
      return d % k == 0 && on(k, dout, dout_bf16, d) && on(k, r, bf16, ldr) && on(k, dresidual, bf16, d) && on(k, dx, bf16, d);
    };
    const bool vec = all(8), even = all(2);
    auto launch = [&]() {
      return vec ? norm_bwd_types<true>(a, bf16, dout_bf16, even, st) : norm_bwd_types<false>(a, bf16, dout_bf16, even, st);
    };
    if (a.dweight && (dx == dout || dx == r)) {
      // in place: the columns' sums read what the rows' CTAs overwrite, so they go first, by themselves
      a.ctas = 0;
      if ((e = launch()) != cudaSuccess) return e;
      a.ctas = n;
      a.dweight = nullptr;
    }
    e = launch();
  } else if (n > 0) {
    const size_t smem = (size_t)d * sizeof(float);
    auto kern = bf16 ? (dout_bf16 ? rmsnorm_backward_kernel<true, true> : rmsnorm_backward_kernel<true, false>)
                     : (dout_bf16 ? rmsnorm_backward_kernel<false, true> : rmsnorm_backward_kernel<false, false>);
    static std::atomic<uint64_t> asked[2][2];
    if ((e = allow_widest_row(kern, asked[bf16][dout_bf16])) != cudaSuccess) return e;
    e = launch_kernel(kern, dim3((unsigned)n), dim3(kThreads), smem, st, false, 1, dout, r, weight, rstd, dresidual, rows, d,
                      ldr, dx, dweight ? parts : nullptr);
  }
  if (e != cudaSuccess || !dweight || (one && n > 0)) return e;
  return launch_kernel(dweight_sum_kernel, dim3((unsigned)((d + 31) / 32)), dim3(1024), 0, st, n > 0, 1,
                       (const float*)parts, n, d, dweight);
}

}  // namespace fp8
}  // namespace moe
