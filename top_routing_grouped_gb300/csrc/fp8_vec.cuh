// fp8_vec.cuh -- eight consecutive columns a thread: 16-byte loads and stores of rows that start
// and end on whole vectors.  A block of 128 columns is then a half-warp.
#pragma once
#include "fp8_common.cuh"

namespace moe {
namespace fp8 {

struct Eight {
  float v[8];
};

template <bool kBf16>
struct Raw8 {
  uint4 w[kBf16 ? 1 : 2];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* s = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(p) + i * (kBf16 ? 2 : 4));
    w[0] = __ldcs(s);
    if constexpr (!kBf16) w[1] = __ldcs(s + 1);
  }
  __device__ __forceinline__ void zero() {
    w[0] = make_uint4(0, 0, 0, 0);
    if constexpr (!kBf16) w[1] = w[0];
  }
  // the largest |value|, as fp32 bits (NaN above infinity above every number): bf16 two at a time
  __device__ __forceinline__ uint32_t top() const {
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
    if constexpr (kBf16) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) m = __vmaxu2(m, u[j] & 0x7fff7fffu);
      return max(m & 0xffff0000u, m << 16);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = max(m, u[j] & 0x7fffffffu);
      return m;
    }
  }
  __device__ __forceinline__ Eight get() const {
    Eight r;
    const uint32_t* u = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      r.v[j] = kBf16 ? __uint_as_float(j & 1 ? u[j / 2] & 0xffff0000u : u[j / 2] << 16) : __uint_as_float(u[j % (kBf16 ? 4 : 8)]);
    return r;
  }
};

// Largest |.| over the half-warp (each half on its own: the halves may have diverged).
__device__ __forceinline__ uint32_t half_warp_max(uint32_t v) {
  const uint32_t mask = 0xffffu << (threadIdx.x & 16);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(mask, v, o));
  return v;
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  uint4 r;
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(&r);
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
  return r;
}

}  // namespace fp8
}  // namespace moe
