// optim.cu -- the gradients' norm and the step of AdamW over many tensors (include/moe_optim.h).
//
// Both go once over the data, so HBM bounds them: a step reads and writes, a value, 28 bytes (bf16 parameter
// with a master, fp32 gradient and moments) down to 12 (8-bit moments, no master).  The tensors' list is
// an argument of the kernel, so that a call needs no copy to the device.
#include <math.h>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "optim_internal.h"

namespace moe {
namespace optim {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;                    // consecutive values of a thread; 16 threads make a block of 128
constexpr int kTile = kThreads * kPer;     // values of a CTA at a time
constexpr int kChunk = 4 * kTile;          // values of a CTA
constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ the lists

struct Entry {  // 72 bytes
  void* param;
  float* master;
  const void* grad;
  void *m, *v;
  uint8_t *m_scales, *v_scales;
  int64_t n;
  float weight_decay;
  uint32_t index_flags;  // the index in the caller's list, above these flags
};
enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kVec = 4, kIndexShift = 3 };  // kVec: every array on 16 bytes (8-bit ones: 8)

// A launch's chunks are fewer than 2^31, whatever its tensors.
static_assert((int64_t)kMostTensors * (kMostValues / kChunk) < INT32_MAX, "too many chunks");

template <int kN>
struct Batch {
  Entry e[kN];
  int n;
  uint32_t first[kN + 1];  // the chunks before each tensor
};

struct GradEntry {
  const void* g;
  int64_t n;
  int bf16, vec;
};

template <int kN>
struct GradBatch {
  GradEntry e[kN];
  int n;
  uint32_t first[kN + 1];
};

// The tensor that a chunk belongs to: the last one with first <= chunk.
template <typename B>
__device__ __forceinline__ int owner(const B& b, uint32_t chunk) {
  int lo = 0, hi = b.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= chunk) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// ------------------------------------------------------------------ eight values

struct F8 {
  float v[kPer];
};

__device__ __forceinline__ F8 load_f32(const float* p, int left, bool vec) {
  F8 r;
  if (vec && left >= kPer) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    r.v[0] = a.x, r.v[1] = a.y, r.v[2] = a.z, r.v[3] = a.w, r.v[4] = b.x, r.v[5] = b.y, r.v[6] = b.z, r.v[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.v[i] = i < left ? p[i] : 0.f;
  }
  return r;
}

__device__ __forceinline__ F8 load_bf16(const uint16_t* p, int left, bool vec) {
  F8 r;
  if (vec && left >= kPer) {
    const uint4 a = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.v[i] = __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i) r.v[i] = i < left ? __uint_as_float((uint32_t)p[i] << 16) : 0.f;
  }
  return r;
}

__device__ __forceinline__ F8 load(const void* p, int64_t i, bool bf16, int left, bool vec) {
  return bf16 ? load_bf16(static_cast<const uint16_t*>(p) + i, left, vec) : load_f32(static_cast<const float*>(p) + i, left, vec);
}

__device__ __forceinline__ void store_f32(float* p, const F8& r, int left, bool vec) {
  if (vec && left >= kPer) {
    reinterpret_cast<float4*>(p)[0] = make_float4(r.v[0], r.v[1], r.v[2], r.v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(r.v[4], r.v[5], r.v[6], r.v[7]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = r.v[i];
  }
}

__device__ __forceinline__ void store_bf16(uint16_t* p, const uint32_t (&w)[4], int left, bool vec) {
  if (vec && left >= kPer) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = (uint16_t)(w[i / 2] >> 16 * (i & 1));
  }
}

__device__ __forceinline__ uint2 load_bytes(const uint8_t* p, int left, bool vec) {
  if (vec && left >= kPer) return __ldcs(reinterpret_cast<const uint2*>(p));
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (i < left) w[i / 4] |= (uint32_t)p[i] << 8 * (i % 4);
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_bytes(uint8_t* p, uint2 w, int left, bool vec) {
  if (vec && left >= kPer) {
    *reinterpret_cast<uint2*>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (i < left) p[i] = (uint8_t)((i < 4 ? w.x : w.y) >> 8 * (i % 4));
  }
}

__device__ __forceinline__ F8 from_e4m3(uint2 w, float by) {
  F8 r;
#pragma unroll
  for (int i = 0; i < kPer; i += 2) {
    const float2 f = fp8::unpack_e4m3x2((i < 4 ? w.x : w.y) >> 8 * (i % 4));
    r.v[i] = f.x * by;
    r.v[i + 1] = f.y * by;
  }
  return r;
}

__device__ __forceinline__ uint2 to_e4m3(const F8& r) {
  return make_uint2(fp8::pack_e4m3x4(r.v[0], r.v[1], r.v[2], r.v[3]), fp8::pack_e4m3x4(r.v[4], r.v[5], r.v[6], r.v[7]));
}

// The largest |.| of a block of 128, by its 16 threads, as fp32 bits (NaN above everything).
__device__ __forceinline__ uint32_t top_of_block(const F8& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = max(m, fp8::abs_bits(r.v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
  return m;
}

// ------------------------------------------------------------------ random words

__host__ __device__ __forceinline__ uint32_t mix(uint32_t x) {
  x *= 0x9E3779B1u;
  x ^= x >> 16;
  x *= 0x6A09E667u;
  x ^= x >> 15;
  x *= 0xBB67AE85u;
  return x ^ x >> 16;
}

// ------------------------------------------------------------------ stochastic rounding

// e4m3 has three bits below the leading one down to 2^-6, and below that steps of 2^-9, which is what
// [2^-6, 2^-5) has too: 2^-6 is added to such values, so that cutting fp32's last 20 bits off fits both.
constexpr uint32_t kCut = 0xfff00000u;
__device__ __forceinline__ float lift(float u) { return u < 0x1p-6f ? 0x1p-6f : 0.f; }

// u in [-448, 448] to an e4m3 value: up in magnitude where the bits that are cut, plus random ones, carry.
__device__ __forceinline__ float round_linear(float u, uint32_t rnd) {
  const float a = fabsf(u), c = lift(a);
  const float q = __uint_as_float((__float_as_uint(a + c) + (rnd >> 16 << 4)) & kCut) - c;
  return copysignf(q, u);
}

// r = sqrt(v), both times the block's factor (its square): to one of r's neighbours lo and hi so that the mean
// of the square is v; with v > 0 not to 0.
__device__ __forceinline__ float round_root(float u, float u2, uint32_t rnd) {
  const float c = lift(u);
  const uint32_t b = __float_as_uint(u + c) & kCut;
  const float lo = __uint_as_float(b) - c, hi = __uint_as_float(b + 0x100000u) - c, lo2 = lo * lo;
  const bool up = (u2 - lo2) * 65536.f > (float)(rnd >> 8 & 0xffffu) * (fmaf(hi, hi, -lo2)) || (lo == 0.f && u2 > 0.f);
  return up ? hi : lo;
}

// To bf16, the bits of two values in a word.
__device__ __forceinline__ uint32_t round_bf16(float v, uint32_t rnd) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x7f800000u) == 0x7f800000u ? u : u + (rnd & 0xffffu);
}

__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ------------------------------------------------------------------ the step

struct Step {
  float lr, c1, c2, eps, log1, log2;  // c: 1 - beta, log: ln of beta
  const float* lr_device;
  const float* factor;
  int64_t* steps;
  uint32_t* ticket;
  uint32_t seed_low, seed_high;
  bool last;  // launch of the call
};

template <int kN>
__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ Batch<kN> b, const __grid_constant__ Step s) {
  const int ti = owner(b, blockIdx.x);
  const Entry& t = b.e[ti];
  const int64_t begin = (int64_t)(blockIdx.x - b.first[ti]) * kChunk, end = min(begin + kChunk, t.n);
  const bool vec = t.index_flags & kVec, p_bf16 = t.index_flags & kParamBf16, g_bf16 = t.index_flags & kGradBf16;
  const bool small = t.m_scales != nullptr;
  pdl_wait();
  pdl_launch_dependents();

  const float f = s.factor ? *s.factor : 1.f;
  const bool skip = !isfinite(f);
  const int64_t taken = *s.steps + 1;
  if (!skip) {
    // 1 - beta^t, without the cancellation for small t
    const float bc1 = -expm1f((float)taken * s.log1), bc2 = -expm1f((float)taken * s.log2);
    const float lr = s.lr_device ? *s.lr_device : s.lr;
    const float rate = lr / bc1, root = rsqrtf(bc2), keep = 1.f - lr * t.weight_decay;
    const float c1 = s.c1, c2 = s.c2;
    const uint32_t key = mix(mix(mix(mix(s.seed_low) + s.seed_high) + (uint32_t)taken) + (t.index_flags >> kIndexShift));
    for (int64_t i0 = begin; i0 < end; i0 += kTile) {
      const int64_t i = i0 + threadIdx.x * kPer;
      const int left = (int)max((int64_t)0, min(end - i, (int64_t)kPer));
      F8 g = load(t.grad, i, g_bf16, left, vec);
      F8 w = t.master ? load_f32(t.master + i, left, vec) : load(t.param, i, p_bf16, left, vec);
      F8 m, v;
      if (small) {
        const int64_t blk = i >> 7;
        const bool in = left > 0;
        m = from_e4m3(load_bytes(static_cast<const uint8_t*>(t.m) + i, left, vec), fp8::scale_value(in ? t.m_scales[blk] : 0));
        v = from_e4m3(load_bytes(static_cast<const uint8_t*>(t.v) + i, left, vec), fp8::scale_value(in ? t.v_scales[blk] : 0));
#pragma unroll
        for (int j = 0; j < kPer; ++j) v.v[j] *= v.v[j];
      } else {
        m = load_f32(static_cast<const float*>(t.m) + i, left, vec);
        v = load_f32(static_cast<const float*>(t.v) + i, left, vec);
      }
      F8 r;  // sqrt(v)
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const float x = g.v[j] * f;
        m.v[j] = fmaf(c1, x - m.v[j], m.v[j]);  // b1 m + c1 x, with one rounding of m's size
        v.v[j] = fmaf(c2, fmaf(x, x, -v.v[j]), v.v[j]);
        r.v[j] = sqrt_fast(v.v[j]);
        w.v[j] = fmaf(keep, w.v[j], -rate * __fdividef(m.v[j], fmaf(r.v[j], root, s.eps)));
      }
      uint32_t rnd[kPer];
      if (small || (p_bf16 && !t.master)) {
        rnd[0] = mix((uint32_t)(i >> 3) + key);
#pragma unroll
        for (int j = 1; j < kPer; ++j) rnd[j] = rnd[j - 1] * 0x3C6EF375u + 0xA54FF53Bu;
      }
      if (t.master) store_f32(t.master + i, w, left, vec);
      if (!p_bf16) {
        store_f32(static_cast<float*>(t.param) + i, w, left, vec);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (t.master) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(w.v[2 * j], w.v[2 * j + 1]);
            o[j] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            o[j] = round_bf16(w.v[2 * j], rnd[2 * j]) >> 16 | (round_bf16(w.v[2 * j + 1], rnd[2 * j + 1]) & 0xffff0000u);
          }
        }
        store_bf16(static_cast<uint16_t*>(t.param) + i, o, left, vec);
      }
      if (small) {
        const uint32_t bm = fp8::scale_byte(__uint_as_float(top_of_block(m))), bv = fp8::scale_byte(__uint_as_float(top_of_block(r)));
        const float im = fp8::inv_scale_value(bm), iv = fp8::inv_scale_value(bv);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          m.v[j] = round_linear(m.v[j] * im, rnd[j]);
          r.v[j] = round_root(r.v[j] * iv, v.v[j] * iv * iv, rnd[j]);
        }
        store_bytes(static_cast<uint8_t*>(t.m) + i, to_e4m3(m), left, vec);
        store_bytes(static_cast<uint8_t*>(t.v) + i, to_e4m3(r), left, vec);
        if ((threadIdx.x & 15) == 0 && left > 0) {
          t.m_scales[i >> 7] = (uint8_t)bm;
          t.v_scales[i >> 7] = (uint8_t)bv;
        }
      } else {
        store_f32(static_cast<float*>(t.m) + i, m, left, vec);
        store_f32(static_cast<float*>(t.v) + i, v, left, vec);
      }
    }
  }
  // the CTA that is done last raises the step's number, when all have read it
  if (s.last) {
    __syncthreads();
    if (threadIdx.x == 0) {
      __threadfence();
      if (atomicAdd(s.ticket, 1u) == gridDim.x - 1) {
        *s.ticket = 0;
        if (!skip) *s.steps = taken;
      }
    }
  }
}

// A step without values: only its number.
__global__ void empty_step_kernel(const float* factor, int64_t* steps) {
  pdl_wait();
  pdl_launch_dependents();
  if (!factor || isfinite(*factor)) ++*steps;
}

template <int kN>
cudaError_t launch_list(const Entry* e, int n, const Step& s, cudaStream_t st) {
  Batch<kN> b{};
  b.n = n;
  for (int i = 0; i < n; ++i) {
    b.e[i] = e[i];
    b.first[i + 1] = b.first[i] + (uint32_t)((e[i].n + kChunk - 1) / kChunk);
  }
  return launch_kernel(adamw_kernel<kN>, dim3(b.first[n]), dim3(kThreads), 0, st, true, 1, b, s);
}

// ------------------------------------------------------------------ the norm

constexpr int kNormChunk = 8 * kTile;  // 64 values a thread are summed in fp32

// parts[CTA]: the sum of squares of its chunks, one in gridDim.x of all.
template <int kN>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ GradBatch<kN> b, double* parts) {
  __shared__ double of_warp[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  double total = 0;
  for (uint32_t chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    const int ti = owner(b, chunk);
    const GradEntry& e = b.e[ti];
    const int64_t begin = (int64_t)(chunk - b.first[ti]) * kNormChunk, end = min(begin + kNormChunk, e.n);
    float sum[kPer] = {};
    for (int64_t i0 = begin; i0 < end; i0 += 4 * kTile) {
      F8 g[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int64_t i = i0 + u * kTile + threadIdx.x * kPer;
        g[u] = load(e.g, i, e.bf16, (int)max((int64_t)0, min(end - i, (int64_t)kPer)), e.vec);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum[j] = fmaf(g[u].v[j], g[u].v[j], sum[j]);
    }
    total += (double)(((sum[0] + sum[1]) + (sum[2] + sum[3])) + ((sum[4] + sum[5]) + (sum[6] + sum[7])));
  }
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kThreads / 32; ++w) total += of_warp[w];
    parts[blockIdx.x] = total;
  }
}

__global__ void __launch_bounds__(1024) norm_end_kernel(const double* parts, int n, float max_norm, float* norm, float* factor) {
  __shared__ double of_warp[32];
  pdl_wait();
  pdl_launch_dependents();
  double total = 0;
  for (int i = threadIdx.x; i < n; i += 1024) total += parts[i];
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = total;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  total = of_warp[threadIdx.x];
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  if (threadIdx.x == 0) {
    const float r = (float)sqrt(total);
    *norm = r;
    if (factor) *factor = isfinite(r) ? (r > max_norm ? max_norm / r : 1.f) : __uint_as_float(0x7fffffffu);
  }
}

template <int kN>
cudaError_t launch_norm_list(const GradEntry* e, int n, double* parts, int* used, cudaStream_t st) {
  GradBatch<kN> b{};
  b.n = n;
  for (int i = 0; i < n; ++i) {
    b.e[i] = e[i];
    b.first[i + 1] = b.first[i] + (uint32_t)((e[i].n + kNormChunk - 1) / kNormChunk);
  }
  const unsigned grid = b.first[n] < (unsigned)kNormCtas ? b.first[n] : (unsigned)kNormCtas;
  *used = (int)grid;
  return launch_kernel(norm_kernel<kN>, dim3(grid), dim3(kThreads), 0, st, true, 1, b, parts);
}

bool on(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int n, const moe_adamw_config& cfg, const float* factor, int64_t* steps,
                         uint32_t* ticket, cudaStream_t st) {
  Step s{};
  s.lr = (float)cfg.lr;
  s.lr_device = cfg.lr_device;
  s.c1 = (float)(1 - cfg.beta1);
  s.c2 = (float)(1 - cfg.beta2);
  s.eps = (float)cfg.eps;
  s.log1 = (float)log(cfg.beta1);
  s.log2 = (float)log(cfg.beta2);
  s.factor = factor;
  s.steps = steps;
  s.ticket = ticket;
  s.seed_low = (uint32_t)cfg.seed;
  s.seed_high = (uint32_t)(cfg.seed >> 32);
  int last = -1;
  for (int i = 0; i < n; ++i)
    if (tensors[i].n > 0) last = i;
  if (last < 0) return launch_kernel(empty_step_kernel, dim3(1), dim3(1), 0, st, true, 1, factor, steps);
  Entry e[kMostTensors];
  for (int i = 0; i <= last;) {
    int m = 0;
    for (; i <= last && m < kMostTensors; ++i) {
      const moe_adamw_tensor& t = tensors[i];
      if (t.n == 0) continue;
      const uintptr_t moments = t.m_scales ? 8 : 16;
      const bool vec = on(t.param, 16) && on(t.master, 16) && on(t.grad, 16) && on(t.m, moments) && on(t.v, moments);
      e[m++] = {t.param, t.master, t.grad, t.m, t.v, t.m_scales, t.v_scales, t.n, t.weight_decay,
                (uint32_t)i << kIndexShift | (t.param_dtype == MOE_BF16 ? kParamBf16 : 0) | (t.grad_dtype == MOE_BF16 ? kGradBf16 : 0) | (vec ? kVec : 0)};
    }
    s.last = i > last;
    const cudaError_t err = m <= 24 ? launch_list<24>(e, m, s, st) : m <= 100 ? launch_list<100>(e, m, s, st) : launch_list<kMostTensors>(e, m, s, st);
    if (err != cudaSuccess) return err;
  }
  return cudaSuccess;
}

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int n, float max_norm, float* norm, float* factor, double* parts,
                             cudaStream_t st) {
  GradEntry e[kMostTensors];
  int used = 0;
  for (int i = 0; i < n;) {
    int m = 0;
    for (; i < n && m < kMostTensors; ++i) {
      const moe_grad_tensor& t = tensors[i];
      if (t.n == 0) continue;
      e[m++] = {t.grad, t.n, t.dtype == MOE_BF16, on(t.grad, 16)};
    }
    if (m == 0) continue;
    int grid = 0;
    const cudaError_t err = m <= 100 ? launch_norm_list<100>(e, m, parts + used, &grid, st) : launch_norm_list<kMostTensors>(e, m, parts + used, &grid, st);
    if (err != cudaSuccess) return err;
    used += grid;
  }
  return launch_kernel(norm_end_kernel, dim3(1), dim3(1024), 0, st, true, 1, (const double*)parts, used, max_norm, norm, factor);
}

}  // namespace optim
}  // namespace moe
