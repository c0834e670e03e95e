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
// of 128: loads of 16 bytes a lane, and the block's maximum in four shuffles.  A thread keeps its
// columns and goes down the rows, so that its addresses advance by constants: with an index
// divided into row and block at every step these kernels were bound by integer instructions, not
// by HBM (saving 131072 x 2048 pre-activations: 337-400 us with the division, 255 us, 6.3 TB/s,
// without).  The next row's loads are issued before the present row is worked on.
constexpr int kResident = 152 * 16;  // CTAs, 8 of them resident on an SM (32 registers)

// The threads of a pass over `per_pass` rows, 16 * nb to a row (nb blocks).
struct Lanes {
  int64_t row;  // this thread's first row; at or past the end: none
  int col;      // its first column (the last block may end before it)
  int blk;
};
__device__ __forceinline__ Lanes lanes(int64_t rows, int per_pass, int nb) {
  const uint32_t s = blockIdx.x * kThreads + threadIdx.x, w = (uint32_t)nb * 16, r = s / w, c = s % w;
  return {(int)r < per_pass ? (int64_t)r : rows, (int)(c * 8), (int)(c / 16)};
}

// blockIdx.y picks one of two tensors of the same shape (the checkpoint's a and b).
struct QuantizeJob {
  const void* x[2];
  uint8_t* q[2];
  uint8_t* scales[2];
};

template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_rows_vec_kernel(QuantizeJob job, int64_t rows, int cols, int64_t ldx,
                                                                     int per_pass) {
  const bool second = blockIdx.y != 0;
  const int nb = (cols + kBlock - 1) / kBlock, sc = (int)scale_cols(cols);
  const Lanes at = lanes(rows, per_pass, nb);
  const bool in = at.col < cols;
  const int l16 = threadIdx.x & 15;
  const char* x = reinterpret_cast<const char*>(second ? job.x[1] : job.x[0]) + (at.row * ldx + at.col) * (kBf16 ? 2 : 4);
  uint8_t* q = (second ? job.q[1] : job.q[0]) + at.row * cols + at.col;
  uint8_t* s = (second ? job.scales[1] : job.scales[0]) + at.row * sc + at.blk;
  const int64_t dx = per_pass * ldx * (kBf16 ? 2 : 4), dq = (int64_t)per_pass * cols, ds = (int64_t)per_pass * sc;
  // the row's padding bytes are written by the other lanes of its last block
  const bool pad = at.blk == nb - 1 && l16 > 0 && nb - 1 + l16 < sc;
  Raw8<kBf16> raw;
  raw.zero();
  if (in && at.row < rows) raw.load(x, 0);
  for (int64_t row = at.row; row < rows; row += per_pass) {
    const Raw8<kBf16> now = raw;
    x += dx;
    if (in && row + per_pass < rows) raw.load(x, 0);
    const uint32_t b = scale_byte(__uint_as_float(half_warp_max(now.top())));
    const float f = inv_scale_value(b);
    const Eight e = now.get();
    if (in)
      *reinterpret_cast<uint2*>(q) = make_uint2(pack_e4m3x4(e.v[0] * f, e.v[1] * f, e.v[2] * f, e.v[3] * f),
                                                pack_e4m3x4(e.v[4] * f, e.v[5] * f, e.v[6] * f, e.v[7] * f));
    if (l16 == 0) *s = (uint8_t)b;
    if (pad) s[l16] = 0;
    q += dq;
    s += ds;
  }
}

// Weights on whole vectors: a CTA holds its 128 x 128 block in registers (a thread eight rows' eight
// columns) between the maximum and the rounding, and reads it once.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) quantize_blocks_vec_kernel(const void* x, int cols, int64_t ldx,
                                                                       int64_t expert_rows, int64_t n_blocks, uint8_t* q,
                                                                       uint8_t* scales) {
  __shared__ uint32_t top_s[kWarps];
  const int64_t sc = scale_cols(cols), nb = (expert_rows + kBlock - 1) / kBlock;
  const int l16 = threadIdx.x & 15, r16 = threadIdx.x >> 4;
  for (int64_t i = blockIdx.x; i < n_blocks; i += gridDim.x) {
    const int64_t e = i / (nb * sc), r0 = i / sc % nb * kBlock;
    const int c = (int)(i % sc) * kBlock + l16 * 8;
    Raw8<kBf16> raw[8];
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t r = r0 + 16 * j + r16;
      raw[j].zero();
      if (r < expert_rows && c < cols) raw[j].load(x, (e * expert_rows + r) * ldx + c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) top = max(top, raw[j].top());
    top = __reduce_max_sync(0xffffffffu, top);
    if ((threadIdx.x & 31) == 0) top_s[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = max(top, top_s[w]);
    const uint32_t b = scale_byte(__uint_as_float(top));
    const float f = inv_scale_value(b);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t r = r0 + 16 * j + r16;
      const Eight v = raw[j].get();
      if (r < expert_rows && c < cols)
        *reinterpret_cast<uint2*>(q + (e * expert_rows + r) * cols + c) =
            make_uint2(pack_e4m3x4(v.v[0] * f, v.v[1] * f, v.v[2] * f, v.v[3] * f),
                       pack_e4m3x4(v.v[4] * f, v.v[5] * f, v.v[6] * f, v.v[7] * f));
    }
    if (threadIdx.x == 0) scales[i] = (uint8_t)b;
    __syncthreads();  // top_s is read before the next block overwrites it
  }
}

// da = dh b silu'(a), db = dh silu(a), h = silu(a) b of one value.
__device__ __forceinline__ void swiglu_backward(float a, float b, float g, float& da, float& db, float& h) {
  float s, c;
  sigmoid_pair(a, s, c);
  const float u = a * s;
  da = g * b * (s + u * c);
  db = g * u;
  h = u * b;
}

template <bool kBackward>
__device__ __forceinline__ void one(float a, float b, float g, float& oa, float& ob, float& oh) {
  if constexpr (kBackward) {
    swiglu_backward(a, b, g, oa, ob, oh);
  } else {
    oa = a;  // e4m3 times a power of two: exact in bf16
    ob = b;
    oh = silu_exact(a) * b;
  }
}

constexpr int kBwdResident = 152 * 5;  // CTAs (48 registers); 20011 x 1072: 35.5 us, with 4 a SM 36.4, with 6 (two waves) 43

// kBackward: da, db and h from dh; else the values themselves, a and b, and h.  Every output but
// da and db may be null.
template <bool kBackward>
__global__ void __launch_bounds__(kThreads)
    checkpoint_vec_kernel(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
                                   const __nv_bfloat16* dh, int64_t rows, int F, __nv_bfloat16* da, __nv_bfloat16* db,
                                   __nv_bfloat16* h, int per_pass) {
  const int nb = (F + kBlock - 1) / kBlock, sc = (int)scale_cols(F);
  const Lanes at = lanes(rows, per_pass, nb);
  if (at.col >= F) return;
  int64_t o = at.row * F + at.col, os = at.row * sc + at.blk;
  const int64_t step = (int64_t)per_pass * F, sstep = (int64_t)per_pass * sc;
  uint2 va, vb;
  Raw8<true> g;
  g.zero();
  uint32_t fa, fb;
  auto fetch = [&](int64_t i, int64_t is) {
    va = __ldcs(reinterpret_cast<const uint2*>(qa + i));
    vb = __ldcs(reinterpret_cast<const uint2*>(qb + i));
    if (kBackward) g.load(dh, i);
    fa = __ldg(sa + is);
    fb = __ldg(sb + is);
  };
  if (at.row < rows) fetch(o, os);
  for (int64_t row = at.row; row < rows; row += per_pass) {
    const uint2 ca = va, cb = vb;
    const Eight e = g.get();
    const float sca = scale_value(fa), scb = scale_value(fb);
    os += sstep;
    if (row + per_pass < rows) fetch(o + step, os);
    float oa[8], ob[8], oh[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t wa = (j & 2 ? ca.y : ca.x) >> (16 * (j & 1)), wb = (j & 2 ? cb.y : cb.x) >> (16 * (j & 1));
      const float2 a = unpack_e4m3x2(wa), b = unpack_e4m3x2(wb);
      one<kBackward>(a.x * sca, b.x * scb, e.v[2 * j], oa[2 * j], ob[2 * j], oh[2 * j]);
      one<kBackward>(a.y * sca, b.y * scb, e.v[2 * j + 1], oa[2 * j + 1], ob[2 * j + 1], oh[2 * j + 1]);
    }
    if (kBackward || da) *reinterpret_cast<uint4*>(da + o) = pack_bf16x8(oa);
    if (kBackward || db) *reinterpret_cast<uint4*>(db + o) = pack_bf16x8(ob);
    if (h) *reinterpret_cast<uint4*>(h + o) = pack_bf16x8(oh);
    o += step;
  }
}

// The same for rows of any length; a warp per block of 128 columns of a row.
template <bool kBackward>
__global__ void __launch_bounds__(kThreads)
    checkpoint_kernel(const uint8_t* qa, const uint8_t* sa, const uint8_t* qb, const uint8_t* sb,
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
      const float a = unpack_e4m3x2(qa[o]).x * fa, b = unpack_e4m3x2(qb[o]).x * fb;
      const float g = kBackward ? __bfloat162float(dh[o]) : 0.f;
      float oa, ob, oh;
      one<kBackward>(a, b, g, oa, ob, oh);
      if (kBackward || da) da[o] = __float2bfloat16_rn(oa);
      if (kBackward || db) db[o] = __float2bfloat16_rn(ob);
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

// CTAs of at most `resident`, and the rows that their threads cover at a time.
struct Pass {
  unsigned ctas;
  int per_pass;
};
static Pass pass_of(int64_t rows, int64_t cols, int resident) {
  const int64_t w = (cols + kBlock - 1) / kBlock * 16, want = (rows * w + kThreads - 1) / kThreads;
  int64_t ctas = want < resident ? want : resident;
  if (ctas * kThreads < w) ctas = (w + kThreads - 1) / kThreads;  // a row longer than that
  return {(unsigned)ctas, (int)(ctas * kThreads / w)};
}

static cudaError_t quantize_vec(const QuantizeJob& job, int jobs, bool bf16, int64_t rows, int64_t cols, int64_t ldx,
                                cudaStream_t st) {
  const Pass p = pass_of(rows, cols, kResident / jobs);
  return launch_kernel(bf16 ? quantize_rows_vec_kernel<true> : quantize_rows_vec_kernel<false>, dim3(p.ctas, (unsigned)jobs),
                       dim3(kThreads), 0, st, false, 1, job, rows, (int)cols, ldx, p.per_pass);
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
  if (vectors(x, bf16, cols, ldx))
    return launch_kernel(bf16 ? quantize_blocks_vec_kernel<true> : quantize_blocks_vec_kernel<false>, dim3(grid_for(n, 1)),
                         dim3(kThreads), 0, st, false, 1, x, (int)cols, ldx, expert_rows, n, (uint8_t*)q, scales);
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

template <bool kBackward>
static cudaError_t checkpoint(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb, const void* dh,
                              int64_t rows, int F, void* da, void* db, void* h, cudaStream_t st) {
  if (F % 8 == 0) {
    const Pass p = pass_of(rows, F, kBwdResident);
    return launch_kernel(checkpoint_vec_kernel<kBackward>, dim3(p.ctas), dim3(kThreads), 0, st, false, 1, (const uint8_t*)qa, sa,
                         (const uint8_t*)qb, sb, (const __nv_bfloat16*)dh, rows, F, (__nv_bfloat16*)da, (__nv_bfloat16*)db,
                         (__nv_bfloat16*)h, p.per_pass);
  }
  return launch_kernel(checkpoint_kernel<kBackward>, dim3(grid_for(rows * ((F + kBlock - 1) / kBlock), kWarps)), dim3(kThreads),
                       0, st, false, 1, (const uint8_t*)qa, sa, (const uint8_t*)qb, sb, (const __nv_bfloat16*)dh, rows, F,
                       (__nv_bfloat16*)da, (__nv_bfloat16*)db, (__nv_bfloat16*)h);
}

cudaError_t launch_checkpoint_backward(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb,
                                       const void* dh, int64_t rows, int F, void* da, void* db, void* h,
                                       cudaStream_t st) {
  return checkpoint<true>(qa, sa, qb, sb, dh, rows, F, da, db, h, st);
}

cudaError_t launch_checkpoint_restore(const void* qa, const uint8_t* sa, const void* qb, const uint8_t* sb, int64_t rows,
                                      int F, void* a, void* b, void* h, cudaStream_t st) {
  return checkpoint<false>(qa, sa, qb, sb, nullptr, rows, F, a, b, h, st);
}

}  // namespace fp8
}  // namespace moe
