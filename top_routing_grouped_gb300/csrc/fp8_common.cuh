// fp8_common.cuh -- device helpers of the 8-bit block format: e4m3 values with one e8m0
// (power-of-two) factor for each block of 128 along a row.
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

#include "fp8_internal.h"

namespace moe {
namespace fp8 {

// The block's scale byte b: b - 127 is the least e with amax <= 448 * 2^e.  448 = 1.75 * 2^8,
// so with amax = m * 2^x (1 <= m < 2) it is x - 8, or x - 7 when m > 1.75: read off amax's bits,
// exactly, without a logarithm.  A subnormal amax has exponent field 0 and falls under the clamp
// at 0 like everything below 448 * 2^-127; an infinite or NaN amax gives 255.
__device__ __forceinline__ uint32_t scale_byte(float amax) {
  const uint32_t u = __float_as_uint(amax) & 0x7fffffffu;
  const uint32_t x = u >> 23;
  if (x == 255u) return 255u;
  const int b = (int)x - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return b < 0 ? 0u : (uint32_t)b;
}

// 2^(b - 127), exact for every byte (b = 0: the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fffffffu : b == 0u ? 0x00400000u : b << 23);
}

// 2^(127 - b): what a value is multiplied with before it is rounded to e4m3 (b <= 254 gives at
// least the subnormal 2^-127; 255: NaN).
__device__ __forceinline__ float inv_scale_value(uint32_t b) {
  return __uint_as_float(b == 255u ? 0x7fffffffu : b == 254u ? 0x00400000u : (254u - b) << 23);
}

// Two fp32 -> two e4m3 (lo in the low byte), nearest, ties to even; |v| <= 448 here by the
// choice of the scale, NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  return pack_e4m3x2(a, b) | (pack_e4m3x2(c, d) << 16);
}

// Two e4m3 (the low half of v) -> two fp32, exact (by way of f16, which holds every e4m3).
__device__ __forceinline__ float2 unpack_e4m3x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)v));
  float lo, hi;
  asm("{.reg .f16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;}" : "=f"(lo), "=f"(hi) : "r"(h));
  return make_float2(lo, hi);
}

// max |.| that keeps a NaN (fmaxf drops it): compared as the bits of |v|, where infinities and
// NaNs are the largest.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// sigma(a) = 1 / (1 + e^-a) and 1 - sigma(a), from z = e^-|a|: the quotients' denominator 1 + z lies
// in [1, 2], so nothing overflows for any a.  The larger of the two is good to a few fp32 steps; the smaller
// one, z r, has z's relative error, which grows with |a| (__expf: 2 + 1.17 |a| steps, 1e-5 at |a| = 80; the
// results are rounded to bf16, 2^-8), and is 0 where e^-|a| is, past |a| = 104.
__device__ __forceinline__ void sigmoid_pair(float a, float& s, float& one_minus_s) {
  const float z = __expf(-fabsf(a)), r = __fdividef(1.f, 1.f + z), zr = z * r;
  s = a >= 0.f ? r : zr;
  one_minus_s = a >= 0.f ? zr : r;
}

// SiLU(a) = a sigma(a), as good as sigma(a).
__device__ __forceinline__ float silu_exact(float a) {
  float s, c;
  sigmoid_pair(a, s, c);
  return a * s;
}

// The same for the tensor-core kernels' hidden rows, in five instructions: a / (1 + 2^(-a log2 e)).  Down to
// a = -87 it is as good as silu_exact; below it is 0, since the reciprocal of what is past 2^126 leaves
// fp32's normal range, while SiLU is there at most 87.4 * 2^-126 = 1.03e-36 in magnitude.  (The quotient in
// plain fp32 is 0 from -88.8 on, where e^-a overflows.)  That can be seen in a hidden row whose 128 values of a block are
// all so small, nowhere else: beside any larger value they round to 0.  With K of one or two blocks the
// epilogue is what bounds the product, and with silu_exact, twice as many instructions, the experts of 128 x
// 3024 took 235 us, not 166.  The rows are rounded to e4m3 right after this: an error of the hardware tanh
// (2^-11) would move about one value in 128 to its neighbour.
__device__ __forceinline__ float silu_hidden(float a) {
  float z, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(z) : "f"(a * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + z));
  return a * r;
}

}  // namespace fp8
}  // namespace moe
