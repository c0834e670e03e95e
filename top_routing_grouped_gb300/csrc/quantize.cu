// quantize.cu -- 8-bit block quantisation (e4m3 with an e8m0 factor per block of 128), of rows
// (1 x 128) and of weights (128 x 128), and the 8-bit activation checkpoints of the SwiGLU.
//
// These kernels read and write each value once and compute a few operations on it: HBM bounds
// them.
#include "fp8_common.cuh"
#include "fp8_vec.cuh"

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

// ---- eight columns a thread -------------------------------------------------------------------
// With rows of whole 16-byte vectors a thread takes 8 consecutive columns and a half-warp a block
// of 128: loads of 16 bytes a lane, and the block's maximum in four shuffles.  A thread requests
// its kUnroll blocks before it uses the first, which keeps enough bytes in flight for HBM
// (blocks are dealt to half-warps in order, so a warp's loads stay contiguous).
constexpr int kUnroll = 4;

// Block `i` of a tensor of nb blocks a row.
struct BlockAt {
  int64_t row;
  int blk;
};
__device__ __forceinline__ BlockAt block_at(int64_t i, uint32_t nb) {
  // a 32-bit division where the index allows it
  if (i >> 32 == 0) return {(int64_t)((uint32_t)i / nb), (int)((uint32_t)i % nb)};
  return {i / nb, (int)(i % nb)};
}

// blockIdx.y picks one of two tensors of the same shape (the checkpoint's a and b).
struct QuantizeJob {
  const void* x[2];
  uint8_t* q[2];
  uint8_t* scales[2];
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_rows_vec_kernel(QuantizeJob job, int64_t rows, int cols, int64_t ldx) {
  const bool second = blockIdx.y != 0;
  const void* x = second ? job.x[1] : job.x[0];
  uint8_t* q = second ? job.q[1] : job.q[0];
  uint8_t* scales = second ? job.scales[1] : job.scales[0];
  const int l16 = threadIdx.x & 15;
  const uint32_t nb = (uint32_t)((cols + kBlock - 1) / kBlock);
  const int64_t sc = scale_cols(cols), n = rows * nb;
  // a CTA's share: kUnroll runs of kThreads / 16 consecutive blocks
  for (int64_t base = (int64_t)blockIdx.x * kUnroll * (kThreads / 16) + threadIdx.x / 16; base < (n + 1) / 2 * 2;  // the same for both halves of a warp
       base += (int64_t)gridDim.x * kUnroll * (kThreads / 16)) {
    Raw8<kBf16> raw[kUnroll];
    BlockAt at[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = base + u * (kThreads / 16);
      at[u] = block_at(i, nb);
      const int c = at[u].blk * kBlock + l16 * 8;
      if (i < n && c < cols) raw[u].load(x, at[u].row * ldx + c);
      else raw[u].zero();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t i = base + u * (kThreads / 16);
      const int c = at[u].blk * kBlock + l16 * 8;
      const Eight e = raw[u].get();
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = max(top, abs_bits(e.v[j]));
      const uint32_t b = scale_byte(__uint_as_float(half_warp_max(top)));
      const float f = inv_scale_value(b);
      if (i < n) {
        if (c < cols)
          *reinterpret_cast<uint2*>(q + at[u].row * cols + c) =
              make_uint2(pack_e4m3x4(e.v[0] * f, e.v[1] * f, e.v[2] * f, e.v[3] * f),
                         pack_e4m3x4(e.v[4] * f, e.v[5] * f, e.v[6] * f, e.v[7] * f));
        if (l16 == 0) scales[at[u].row * sc + at[u].blk] = (uint8_t)b;
        // the row's padding bytes, by the other lanes of its last block
        if (at[u].blk == (int)nb - 1 && l16 > 0 && nb - 1 + l16 < sc) scales[at[u].row * sc + nb - 1 + l16] = 0;
      }
    }
  }
}

// da = dh b silu'(a), db = dh silu(a), h = silu(a) b of one value.
__device__ __forceinline__ void swiglu_backward(float a, float b, float g, float& da, float& db, float& h) {
  const float s = __fdividef(1.f, 1.f + __expf(-a)), u = a * s;
  da = g * b * (s + u * (1.f - s));
  db = g * u;
  h = u * b;
}

constexpr int kBwdUnroll = 2;

__global__ void __launch_bounds__(kThreads)
    checkpoint_backward_vec_kernel(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
                                   const __nv_bfloat16* dh, int64_t rows, int F, __nv_bfloat16* da, __nv_bfloat16* db,
                                   __nv_bfloat16* h) {
  const int l16 = threadIdx.x & 15;
  const uint32_t nb = (uint32_t)((F + kBlock - 1) / kBlock);
  const int64_t sc = scale_cols(F), n = rows * nb;
  for (int64_t base = (int64_t)blockIdx.x * kBwdUnroll * (kThreads / 16) + threadIdx.x / 16; base < n;
       base += (int64_t)gridDim.x * kBwdUnroll * (kThreads / 16)) {
    uint2 va[kBwdUnroll], vb[kBwdUnroll];
    Raw8<true> g[kBwdUnroll];
    float fa[kBwdUnroll], fb[kBwdUnroll];
    int64_t o[kBwdUnroll];
    bool in[kBwdUnroll];
#pragma unroll
    for (int u = 0; u < kBwdUnroll; ++u) {
      const int64_t i = base + u * (kThreads / 16);
      const BlockAt at = block_at(i, nb);
      const int c = at.blk * kBlock + l16 * 8;
      in[u] = i < n && c < F;
      o[u] = at.row * F + c;
      if (in[u]) {
        va[u] = __ldcs(reinterpret_cast<const uint2*>(qa + o[u]));
        vb[u] = __ldcs(reinterpret_cast<const uint2*>(qb + o[u]));
        g[u].load(dh, o[u]);
        fa[u] = scale_value(__ldg(sa + at.row * sc + at.blk));
        fb[u] = scale_value(__ldg(sb + at.row * sc + at.blk));
      }
    }
#pragma unroll
    for (int u = 0; u < kBwdUnroll; ++u) {
      if (!in[u]) continue;
      const Eight e = g[u].get();
      float oa[8], ob[8], oh[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t wa = (j & 2 ? va[u].y : va[u].x) >> (16 * (j & 1)), wb = (j & 2 ? vb[u].y : vb[u].x) >> (16 * (j & 1));
        const float2 a = unpack_e4m3x2(wa), b = unpack_e4m3x2(wb);
        swiglu_backward(a.x * fa[u], b.x * fb[u], e.v[2 * j], oa[2 * j], ob[2 * j], oh[2 * j]);
        swiglu_backward(a.y * fa[u], b.y * fb[u], e.v[2 * j + 1], oa[2 * j + 1], ob[2 * j + 1], oh[2 * j + 1]);
      }
      *reinterpret_cast<uint4*>(da + o[u]) = pack_bf16x8(oa);
      *reinterpret_cast<uint4*>(db + o[u]) = pack_bf16x8(ob);
      if (h) *reinterpret_cast<uint4*>(h + o[u]) = pack_bf16x8(oh);
    }
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
      float oa, ob, oh;
      swiglu_backward(a, b, g, oa, ob, oh);
      da[o] = __float2bfloat16_rn(oa);
      db[o] = __float2bfloat16_rn(ob);
      if (h) h[o] = __float2bfloat16_rn(oh);
    }
  }
}

unsigned grid_for(int64_t work, int64_t per_cta) {
  const int64_t g = (work + per_cta - 1) / per_cta;
  return (unsigned)(g < 1 ? 1 : g > 1 << 20 ? 1 << 20 : g);
}

}  // namespace

// Rows that start and end on whole 16-byte vectors (bf16: 8 values, e4m3: 8 bytes).
static bool vectors(const void* x, bool bf16, int64_t cols, int64_t ldx) {
  return cols % 8 == 0 && ldx % (bf16 ? 8 : 4) == 0 && reinterpret_cast<uintptr_t>(x) % 16 == 0 && cols <= INT32_MAX - 512;
}

static cudaError_t quantize_vec(const QuantizeJob& job, int jobs, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                cudaStream_t st) {
  const dim3 grid(grid_for(rows * ((cols + kBlock - 1) / kBlock), kUnroll * (kThreads / 16)), (unsigned)jobs);
  return launch_kernel(bf16 ? quantize_rows_vec_kernel<true> : quantize_rows_vec_kernel<false>, grid, dim3(kThreads), 0, st,
                       false, 1, job, rows, (int)cols, ldx);
}

cudaError_t launch_quantize_rows(const void* x, bool bf16, int64_t rows, int64_t cols, int64_t ldx, void* q,
                                 uint8_t* scales, cudaStream_t st) {
  if (vectors(x, bf16, cols, ldx))
    return quantize_vec(QuantizeJob{{x, x}, {(uint8_t*)q, (uint8_t*)q}, {scales, scales}}, 1, bf16, rows, cols, ldx, st);
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
  if (vectors(a, true, F, F))
    return quantize_vec(QuantizeJob{{a, b}, {(uint8_t*)qa, (uint8_t*)qb}, {sa, sb}}, 2, true, rows, F, F, st);
  cudaError_t e = launch_quantize_rows(a, true, rows, F, F, qa, sa, st);
  return e != cudaSuccess ? e : launch_quantize_rows(b, true, rows, F, F, qb, sb, st);
}

cudaError_t launch_checkpoint_backward(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                       const void* dh, int64_t rows, int F, void* da, void* db, void* h,
                                       cudaStream_t st) {
  if (F % 8 == 0)
    return launch_kernel(checkpoint_backward_vec_kernel,
                         dim3(grid_for(rows * ((F + kBlock - 1) / kBlock), kBwdUnroll * (kThreads / 16))), dim3(kThreads), 0,
                         st, false, 1, (const uint8_t*)qa, sa, (const uint8_t*)qb, sb, (const __nv_bfloat16*)dh, rows, F,
                         (__nv_bfloat16*)da, (__nv_bfloat16*)db, (__nv_bfloat16*)h);
  return launch_kernel(checkpoint_backward_kernel, dim3(grid_for(rows * ((F + kBlock - 1) / kBlock), kWarps)),
                       dim3(kThreads), 0, st, false, 1, (const uint8_t*)qa, sa, (const uint8_t*)qb, sb,
                       (const __nv_bfloat16*)dh, rows, F, (__nv_bfloat16*)da, (__nv_bfloat16*)db, (__nv_bfloat16*)h);
}

}  // namespace fp8
}  // namespace moe
