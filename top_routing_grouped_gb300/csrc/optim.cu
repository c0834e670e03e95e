// optim.cu -- the gradients' norm and the step of AdamW over many tensors (include/moe_optim.h).
//
// Both go once over the data, so HBM bounds them: a step reads and writes, a value, 30 bytes (bf16 parameter
// with a master, fp32 gradient and moments) down to 10 (bf16 gradient, 8-bit moments, no master).  403 M values at 30
// bytes take 1.75 ms, the norm of as many fp32 gradients 0.22 ms: both at the copy bandwidth.  The tensors' list is
// an argument of the kernel, so that a call needs no copy to the device.
#include <math.h>

#include <initializer_list>
#include <type_traits>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "optim_internal.h"

namespace moe {
namespace optim {
namespace {

constexpr int kPer = 8;  // consecutive values of a thread; 16 threads make a block of 128

// The step's CTAs, for moments in 32 or in 8 bits: threads, CTAs an SM, values at a time (a tile).  A chunk, what a CTA
// takes of a tensor, has 1 to kTiles tiles (a power of two), so many that there are kFew chunks and more.
// With moments in 32 bits HBM bounds the step whatever these are (403 M values with masters: 1775 us with 256 threads,
// 3 CTAs and 4 tiles; 1771 with 2 CTAs, 1781 with 8 tiles).  With moments in 8 bits the warps that an SM holds count (805 M
// values, no masters: 128 threads, 9 CTAs of 56 registers 1545 us, although 172 bytes spill; 8 of 64 1567, 7 of 72 1615, 10 of
// 48 1591; 256 threads 4 CTAs 1594, 3 1749), and how evenly it ends (kFew of 152 * 12, 24, 48: 131 M values 269, 269, 263 us,
// 35 M 80, 78, 80; 64, 32 and 16 tiles within 1 %).
template <bool kSmall>
struct Ctas {
  static constexpr int kThreads = kSmall ? 128 : 256, kOfSm = kSmall ? 9 : 3, kTile = kThreads * kPer, kTiles = kSmall ? 32 : 4,
                       kFew = 152 * (kSmall ? 48 : 12);
};
constexpr int kMostChunk = Ctas<true>::kTiles * Ctas<true>::kTile, kLeastChunk = Ctas<false>::kTiles * Ctas<false>::kTile;
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
static_assert((int64_t)kMostTensors * (kMostValues / kLeastChunk) < INT32_MAX, "too many chunks");

template <int kN>
struct Batch {
  Entry e[kN];
  int n;
  int chunk;               // values
  uint32_t first[kN + 1];  // the chunks before each tensor
};

struct GradEntry {
  const void* g;
  int64_t n;
  bool bf16, vec;
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

// The first `left` of eight values from i on, the others 0.
__device__ __forceinline__ F8 load(const void* p, int64_t i, bool bf16, int left) {
  F8 r;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    r.v[j] = j >= left ? 0.f : bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i + j] << 16) : static_cast<const float*>(p)[i + j];
  return r;
}

__device__ __forceinline__ F8 load_e4m3(const uint8_t* p, int left, float by) {
  F8 r;
#pragma unroll
  for (int j = 0; j < kPer; ++j) r.v[j] = j < left ? fp8::unpack_e4m3x2(p[j]).x * by : 0.f;
  return r;
}

__device__ __forceinline__ void store(float* p, int64_t i, const F8& r, int left) {
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < left) p[i + j] = r.v[j];
}

// The largest |.| of a block of 128, by its 16 threads (NaN above everything).
__device__ __forceinline__ float top_of_block(const F8& r) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) m = max(m, fp8::abs_bits(r.v[i]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kAll, m, o));
  return __uint_as_float(m);
}

// The scale byte of a block from its largest |m|, as fp8::scale_byte gives it; or, `root`, that of r = sqrt(v) from the
// largest v: b - 127 is the least e with v <= 448^2 * 4^e, read off v's bits (448^2 = 1.53125 * 2^17), so that it does not
// depend on how a root is rounded.  What counts as 0 gives 0, an infinity or NaN 255.
__device__ __forceinline__ uint32_t block_byte(float top, bool root) {
  const uint32_t u = __float_as_uint(top);
  const int x = (int)(u >> 23), y = x + ((u & 0x7fffffu) > (root ? 0x440000u : 0x600000u) ? 1 : 0);
  const int b = root ? (y + 111) >> 1 : max(y - 8, 0);
  return x >= 255 ? 255u : x == 0 ? 0u : (uint32_t)b;
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
constexpr uint32_t kTop = 0x07e00000u;  // 448 * 2^-120
__device__ __forceinline__ float lift(float u) { return u < 0x1p-6f ? 0x1p-6f : 0.f; }

// u in [-448, 448] to an e4m3 value: up in magnitude where the bits that are cut, plus random ones, carry.
__device__ __forceinline__ float round_linear(float u, uint32_t rnd) {
  const float a = fabsf(u), c = lift(a);
  const float q = __uint_as_float((__float_as_uint(a + c) + (rnd >> 16 << 4)) & kCut) - c;
  return copysignf(q, u);
}

// r = sqrt(v), both times the block's factor (its square): to one of r's neighbours lo and hi so that the mean
// of the square is v; with v > 0 not to 0, and not past 448.
__device__ __forceinline__ float round_root(float u, float u2, uint32_t rnd) {
  const float c = lift(u);
  const uint32_t b = __float_as_uint(u + c) & kCut;
  const float lo = __uint_as_float(b) - c, hi = __uint_as_float(b + 0x100000u) - c, lo2 = lo * lo;
  const float border = fmaf((float)(rnd >> 8 & 0xffffu) * 0x1p-16f, fmaf(hi, hi, -lo2), lo2);
  return u2 > (lo == 0.f ? 0.f : border) && lo < 448.f ? hi : lo;
}

// To bf16, in the upper half.
__device__ __forceinline__ uint32_t round_bf16(float v, uint32_t rnd) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x7f800000u) == 0x7f800000u ? u : u + (rnd & 0xffffu);
}

// sqrt and reciprocal to two steps of fp32; what is below 2^-126 counts as 0.
__device__ __forceinline__ float sqrt_fast(float x) {
  float r;
  asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ------------------------------------------------------------------ two values an instruction

// The step with 8-bit moments is bound by the instructions it issues as much as by HBM (62 a value, 3.1 a cycle and SM;
// 805 M values 1.54 ms, 93 % of the copy bandwidth with fp32 gradients, 78 % with bf16 ones): its fp32 products and sums
// are taken two at a time (the packed forms round as the plain ones do).  With 104 a value it took 2.83 ms.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 neg2(float2 v) { return make_float2(-v.x, -v.y); }

// the larger of two, NaN where one is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Four pairs of consecutive values.
struct P4 {
  float2 v[kPer / 2];
};

// The same as they lie in memory.
template <int kBytes>
struct Raw {
  using Part = typename std::conditional<kBytes == 1, uint2, uint4>::type;
  static constexpr int kParts = kBytes == 4 ? 2 : 1;
  Part part[kParts];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const Part* q = reinterpret_cast<const Part*>(static_cast<const char*>(p) + i * kBytes);
#pragma unroll
    for (int j = 0; j < kParts; ++j) part[j] = __ldcs(q + j);
  }
  __device__ __forceinline__ P4 get() const {
    const uint32_t* w = reinterpret_cast<const uint32_t*>(part);
    P4 r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kBytes == 4) r.v[j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
      else if constexpr (kBytes == 2) r.v[j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
      else r.v[j] = fp8::unpack_e4m3x2(w[j / 2] >> 16 * (j & 1));
    }
    return r;
  }
};

__device__ __forceinline__ void store4_f32(float* p, const P4& r) {
  __stcs(reinterpret_cast<float4*>(p), make_float4(r.v[0].x, r.v[0].y, r.v[1].x, r.v[1].y));
  __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(r.v[2].x, r.v[2].y, r.v[3].x, r.v[3].y));
}

// ------------------------------------------------------------------ the step

struct Step {
  float lr, b1, b2, c1, c2, a, neg_a2, eps, log1, log2;  // b: beta, neg_a2: -a^2, log: ln of beta; the others: see Common
  bool slow;
  const float* lr_device;
  const float* factor;
  int64_t* steps;
  uint32_t* ticket;
  uint32_t seed_low, seed_high;
  bool last;  // launch of the call
};

// What all values of a tensor have in common.
struct Common {
  float fa, c1, c2, rate, root, eps;  // fa = f a, rate = lr / (1 - beta1^t), root = 1 / sqrt(1 - beta2^t)
  // 1 - lr wd = keep + rest.  One float alone is off by up to 2^-25, the same for all values and steps: 1.4 % of a decay of
  // 1e-6, 19 % of 1e-7.  keep is cut towards 0 and rest is not 0, so that an infinite parameter stays what it is.
  float keep, rest;
  uint32_t key;
  // Both betas are 0.5 or more, as they mostly are: m + (1 - b1) (x - m) then has one rounding of m's size.  Where a beta is
  // small and m is large beside x, it would lose x; b1 m + (1 - b1) x does not.  In the first form x = f g is taken times
  // a, the largest power of two with a^2 <= 1 - b2, and c1 and c2 are (1 - b1) / a and (1 - b2) / a^2: exact, and x^2
  // overflows where (1 - b2) x^2 does, no sooner.  Else a = 1.
  bool slow;
};

enum : int { kF32 = 0, kBf16 = 1, kMaster = 2 };  // a parameter: fp32, bf16, bf16 with a master

// The factors of a chunk's 8-bit moments are in shared memory meanwhile, m's and then v's, read and written with
// whole sectors: stored and loaded a byte a block, in the loop, they took a third of the step's time.
constexpr int kMostBlocks = kMostChunk / 128;

// What a thread reads for eight values, all of them there and on whole vectors.  Nothing is read ahead: more warps an SM
// gain more than the registers that would take.
template <int kParam, bool kGradBf16, bool kSmall>
struct Read {
  Raw<kGradBf16 ? 2 : 4> g;
  Raw<kParam == kBf16 ? 2 : 4> w;
  Raw<kSmall ? 1 : 4> m, v;
  __device__ __forceinline__ void load(const Entry& t, int64_t i) {
    g.load(t.grad, i);
    w.load(kParam == kMaster ? t.master : t.param, i);
    m.load(t.m, i);
    v.load(t.v, i);
  }
};

template <int kParam, bool kGradBf16, bool kSmall>
__device__ __forceinline__ void step_whole(const Entry& t, int64_t i, const Step& s, const Common& k,
                                           const Read<kParam, kGradBf16, kSmall>& in, uint8_t* factors) {
  const P4 g = in.g.get();
  P4 w = in.w.get(), m = in.m.get(), v = in.v.get(), r;
  if constexpr (kSmall) {
    const float2 fm = both(fp8::scale_value(factors[0])), fv = both(fp8::scale_value(factors[kMostBlocks]));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m.v[j] = mul2(m.v[j], fm);
      v.v[j] = mul2(v.v[j], fv);
      v.v[j] = mul2(v.v[j], v.v[j]);
    }
  }
  if (k.slow) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = mul2(g.v[j], both(k.fa));
      m.v[j] = fma2(both(k.c1), fma2(m.v[j], both(-s.a), x), m.v[j]);
      v.v[j] = fma2(both(k.c2), fma2(x, x, mul2(v.v[j], both(s.neg_a2))), v.v[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = mul2(g.v[j], both(k.fa));
      m.v[j] = fma2(both(k.c1), x, mul2(both(s.b1), m.v[j]));
      v.v[j] = fma2(mul2(both(k.c2), x), x, mul2(both(s.b2), v.v[j]));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r.v[j] = make_float2(sqrt_fast(v.v[j].x), sqrt_fast(v.v[j].y));
    const float2 den = fma2(r.v[j], both(k.root), both(k.eps));
    const float2 u = mul2(m.v[j], make_float2(rcp_fast(den.x), rcp_fast(den.y)));
    w.v[j] = fma2(both(k.keep), w.v[j], fma2(both(k.rest), w.v[j], mul2(both(-k.rate), u)));
  }
  uint32_t rnd[kPer];
  if constexpr (kSmall || kParam == kBf16) {
    rnd[0] = mix((uint32_t)(i >> 3) + k.key);
#pragma unroll
    for (int j = 1; j < kPer; ++j) rnd[j] = rnd[j - 1] * 0x3C6EF375u + 0xA54FF53Bu;
  }
  if constexpr (kParam == kMaster) store4_f32(t.master + i, w);
  if constexpr (kParam == kF32) {
    store4_f32(static_cast<float*>(t.param) + i, w);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (kParam == kMaster) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(w.v[j].x, w.v[j].y);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      } else {  // adds the words' low halves to the bits that are cut; infinities and NaN stay
        asm("cvt.rs.bf16x2.f32 %0, %1, %2, %3;" : "=r"(o[j])
            : "f"(w.v[j].y), "f"(w.v[j].x), "r"(__byte_perm(rnd[2 * j], rnd[2 * j + 1], 0x5410)));
      }
    }
    __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.param) + i), make_uint4(o[0], o[1], o[2], o[3]));
  }
  if constexpr (!kSmall) {
    store4_f32(static_cast<float*>(t.m) + i, m);
    store4_f32(static_cast<float*>(t.v) + i, v);
  } else {
    // The largest |m| and v of the block.  From the first exchange on even lanes have m's, odd ones v's, and find
    // the factor of theirs.
    float tm = 0.f, tv = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      tm = max_nan(max_nan(tm, fabsf(m.v[j].x)), fabsf(m.v[j].y));
      tv = max_nan(max_nan(tv, v.v[j].x), v.v[j].y);
    }
    const bool odd = threadIdx.x & 1;
    float top = max_nan(odd ? tv : tm, __shfl_xor_sync(kAll, odd ? tm : tv, 1));
#pragma unroll
    for (int o = 2; o < 16; o *= 2) top = max_nan(top, __shfl_xor_sync(kAll, top, o));
    const uint32_t b = block_byte(top, odd);  // 247 at most, or 255
    if ((threadIdx.x & 14) == 0) factors[odd ? kMostBlocks : 0] = (uint8_t)b;
    const float inv = __uint_as_float(b == 255u ? 0x7fffffffu : (254u - b) << 23), other = __shfl_xor_sync(kAll, inv, 1);
    const float2 im = both(odd ? other : inv), iv = both(odd ? inv : other);
    // Times 2^-120 an e4m3 value has fp32's bits 27-20 for its own 7-0 but the sign's: its subnormals, below 2^-6,
    // are fp32's.  So cutting fp32's last 20 bits off, after the random ones are added, rounds both alike.  Four
    // bits up, the value is the top byte.  (Below 2^-6 the product is rounded to 2^-29, a step's 2^-20: four bits more than
    // the random ones.)
    constexpr float kDown = 0x1p-120f, kUp = 0x1p120f;
    uint32_t ym[kPer], yr[kPer];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 um = mul2(mul2(m.v[j], im), both(kDown)), ur = mul2(mul2(r.v[j], iv), both(kDown));
      const float2 u2 = mul2(mul2(v.v[j], iv), iv);
      const uint32_t bm[2] = {__float_as_uint(um.x), __float_as_uint(um.y)}, br[2] = {__float_as_uint(ur.x), __float_as_uint(ur.y)};
      // m: (bits + (word >> 16 << 4)) << 4 and the sign
#pragma unroll
      for (int h = 0; h < 2; ++h) ym[2 * j + h] = ((bm[h] << 4) + __byte_perm(rnd[2 * j + h], 0, 0x4324)) & 0x7fffffffu | bm[h] & 0x80000000u;
      // r: between lo and hi, up where v lies above lo^2 + word (hi^2 - lo^2)
      const uint32_t l0 = br[0] & kCut, l1 = br[1] & kCut;
      const float2 lo = mul2(make_float2(__uint_as_float(l0), __uint_as_float(l1)), both(kUp));
      const float2 hi = mul2(make_float2(__uint_as_float(l0 + 0x100000u), __uint_as_float(l1 + 0x100000u)), both(kUp));
      const float2 lo2 = mul2(lo, lo), gap = fma2(hi, hi, neg2(lo2));
      const float2 word = add2(make_float2(__uint_as_float(rnd[2 * j] >> 1 & 0x7fff80u | 0x3f800000u),
                                           __uint_as_float(rnd[2 * j + 1] >> 1 & 0x7fff80u | 0x3f800000u)), both(-1.f));
      const float2 border = fma2(word, gap, lo2);
      // not to 0 with v > 0, not past 448
      const bool up0 = u2.x > (l0 == 0 ? 0.f : border.x) && l0 < kTop, up1 = u2.y > (l1 == 0 ? 0.f : border.y) && l1 < kTop;
      yr[2 * j] = (br[0] << 4) + (up0 ? 1u << 24 : 0u);
      yr[2 * j + 1] = (br[1] << 4) + (up1 ? 1u << 24 : 0u);
    }
    const auto pack = [](const uint32_t* y) { return __byte_perm(__byte_perm(y[0], y[1], 0x0073), __byte_perm(y[2], y[3], 0x0073), 0x5410); };
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i), make_uint2(pack(ym), pack(ym + 4)));
    __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i), make_uint2(pack(yr), pack(yr + 4)));
  }
}

__device__ __forceinline__ void prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// The same for values at a tensor's end, or off whole vectors: one by one, 2 to 3.5 times as long a value (100 M values with
// masters and moments in 32 bits, each array one value off a 16-byte boundary: 935 us, on it 447; 134 M with moments in
// 8 bits 943 and 270).
template <bool kSmall>
__device__ __noinline__ void step_rest(const Entry& t, int64_t i, int64_t end, const Step& s, const Common& k, uint8_t* factors) {
  const int left = (int)max((int64_t)0, min(end - i, (int64_t)kPer));
  const bool p_bf16 = t.index_flags & kParamBf16;
  const F8 g = load(t.grad, i, t.index_flags & kGradBf16, left);
  F8 w = t.master ? load(t.master, i, false, left) : load(t.param, i, p_bf16, left);
  F8 m, v, r;
  if constexpr (kSmall) {
    m = load_e4m3(static_cast<const uint8_t*>(t.m) + i, left, fp8::scale_value(factors[0]));
    v = load_e4m3(static_cast<const uint8_t*>(t.v) + i, left, fp8::scale_value(factors[kMostBlocks]));
#pragma unroll
    for (int j = 0; j < kPer; ++j) v.v[j] *= v.v[j];
  } else {
    m = load(t.m, i, false, left);
    v = load(t.v, i, false, left);
  }
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const float x = g.v[j] * k.fa;
    if (k.slow) {
      m.v[j] = fmaf(k.c1, fmaf(m.v[j], -s.a, x), m.v[j]);
      v.v[j] = fmaf(k.c2, fmaf(x, x, v.v[j] * s.neg_a2), v.v[j]);
    } else {
      m.v[j] = fmaf(k.c1, x, s.b1 * m.v[j]);
      v.v[j] = fmaf(k.c2 * x, x, s.b2 * v.v[j]);
    }
    r.v[j] = sqrt_fast(v.v[j]);
    w.v[j] = fmaf(k.keep, w.v[j], fmaf(k.rest, w.v[j], -k.rate * (m.v[j] * rcp_fast(fmaf(r.v[j], k.root, k.eps)))));
  }
  uint32_t rnd[kPer];
  rnd[0] = mix((uint32_t)(i >> 3) + k.key);
#pragma unroll
  for (int j = 1; j < kPer; ++j) rnd[j] = rnd[j - 1] * 0x3C6EF375u + 0xA54FF53Bu;
  if (t.master) store(t.master, i, w, left);
  if (p_bf16) {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < left) {
        const __nv_bfloat16 h = __float2bfloat16_rn(w.v[j]);
        static_cast<uint16_t*>(t.param)[i + j] = t.master ? *reinterpret_cast<const uint16_t*>(&h) : (uint16_t)(round_bf16(w.v[j], rnd[j]) >> 16);
      }
  } else {
    store(static_cast<float*>(t.param), i, w, left);
  }
  if constexpr (!kSmall) {
    store(static_cast<float*>(t.m), i, m, left);
    store(static_cast<float*>(t.v), i, v, left);
    return;
  }
  const uint32_t bm = block_byte(top_of_block(m), false), bv = block_byte(top_of_block(v), true);
  const float im = fp8::inv_scale_value(bm), iv = fp8::inv_scale_value(bv);
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < left) {
      static_cast<uint8_t*>(t.m)[i + j] = (uint8_t)fp8::pack_e4m3x2(round_linear(m.v[j] * im, rnd[j]), 0.f);
      static_cast<uint8_t*>(t.v)[i + j] = (uint8_t)fp8::pack_e4m3x2(round_root(r.v[j] * iv, v.v[j] * iv * iv, rnd[j]), 0.f);
    }
  if ((threadIdx.x & 15) == 0) {
    factors[0] = (uint8_t)bm;
    factors[kMostBlocks] = (uint8_t)bv;
  }
}

template <int kParam, bool kGradBf16, bool kSmall>
__device__ __forceinline__ void step_tiles(const Entry& t, int64_t from, int64_t to, const Step& s, const Common& k, uint8_t* factors) {
  for (int64_t i = from + threadIdx.x * kPer; i < to; i += Ctas<kSmall>::kTile) {
    Read<kParam, kGradBf16, kSmall> in;
    in.load(t, i);
    step_whole(t, i, s, k, in, factors + (int)(i - from) / 128);
  }
}

// In blocks of r's largest factor, 2^56, 240 is the last value whose square is below 2^128: what was rounded up to 256 is
// taken back, once the block is done (in the loop, where hardly any block needs it, that made the step with bf16
// gradients 7 % slower).
constexpr uint8_t kLargestFactor = 127 + 56, kLargestOfIt = 0x77;
__device__ __noinline__ void keep_squares_finite(uint8_t* r, int n) {
  for (int i = 0; i < n; ++i) r[i] = min(r[i], kLargestOfIt);
}

// The steps' number is read by every CTA of a call and raised by one of the last launch, after all have read it.  Each
// draws a ticket once it has read the number, with release semantics (nothing else holds a read before an atomic on
// another word); the CTA that draws the last one, and so knows that all have read, fences before it writes.  The draw
// takes as long as what it waits for: the last warp does it behind the barrier (60 small tensors, clipped: 28.8 us;
// before the barrier, or at the end, 1.4 us more).
__device__ __forceinline__ uint32_t draw(uint32_t* ticket) {
  uint32_t n;
  asm volatile("atom.release.gpu.global.add.u32 %0, [%1], 1;" : "=r"(n) : "l"(ticket) : "memory");
  return n;
}

// One kernel for tensors with moments in 8 bits and one for those with 32, which takes more registers.
template <int kN, bool kSmall>
__global__ void __launch_bounds__(Ctas<kSmall>::kThreads, Ctas<kSmall>::kOfSm) adamw_kernel(const __grid_constant__ Batch<kN> b,
                                                                                              const __grid_constant__ Step s) {
  constexpr int kThreads = Ctas<kSmall>::kThreads, kTile = Ctas<kSmall>::kTile;
  __shared__ Common common;
  __shared__ bool skip;
  __shared__ int64_t taken;
  __shared__ uint8_t factors[kSmall ? 2 * kMostBlocks : 1];
  const int ti = owner(b, blockIdx.x);
  const Entry& t = b.e[ti];
  const int64_t begin = (int64_t)(blockIdx.x - b.first[ti]) * b.chunk, end = min(begin + b.chunk, t.n);
  const int64_t whole = t.index_flags & kVec ? begin + (end - begin) / kTile * kTile : begin;
  // the first tile is on its way to L2 while the kernel before ends and the first thread works (twelve small blocks, 60
  // tensors: 1.1 us of 29 less)
  if (const int64_t i = begin + threadIdx.x * kPer; i < whole) {
    prefetch(static_cast<const char*>(t.grad) + i * (t.index_flags & kGradBf16 ? 2 : 4));
    if (t.master) prefetch(t.master + i);
    else prefetch(static_cast<const char*>(t.param) + i * (t.index_flags & kParamBf16 ? 2 : 4));
    prefetch(static_cast<const char*>(t.m) + i * (kSmall ? 1 : 4));
    prefetch(static_cast<const char*>(t.v) + i * (kSmall ? 1 : 4));
  }
  bool raise = false;
  pdl_wait();
  pdl_launch_dependents();

  if (threadIdx.x == 0) {
    const float f = s.factor ? *s.factor : 1.f;
    taken = *static_cast<const volatile int64_t*>(s.steps) + 1;
    const float lr = s.lr_device ? *s.lr_device : s.lr;
    // 1 - beta^t, without the cancellation for small t
    const float bc1 = -expm1f((float)taken * s.log1), bc2 = -expm1f((float)taken * s.log2);
    const uint32_t key = mix(mix(mix(mix(s.seed_low) + s.seed_high) + (uint32_t)taken) + (t.index_flags >> kIndexShift));
    const float keep = __fmaf_rz(-lr, t.weight_decay, 1.f), rest = fmaf(-lr, t.weight_decay, 1.f - keep);
    common = Common{f * s.a, s.c1, s.c2, lr / bc1, rsqrtf(bc2), s.eps, keep, copysignf(fmaxf(fabsf(rest), 0x1p-126f), keep), key, s.slow};
    skip = !isfinite(f);
  }
  const int blocks = (int)((end - begin + 127) / 128);
  const int64_t block0 = begin / 128;
  if constexpr (kSmall)
    for (int j = threadIdx.x; j < blocks; j += kThreads) {
      factors[j] = t.m_scales[block0 + j];
      factors[kMostBlocks + j] = t.v_scales[block0 + j];
    }
  __syncthreads();
  if (s.last && threadIdx.x == kThreads - 32) raise = draw(s.ticket) == gridDim.x - 1;
  const Common k = common;
  if (!skip) {
    const bool g = t.index_flags & kGradBf16;
    if (t.master) g ? step_tiles<kMaster, true, kSmall>(t, begin, whole, s, k, factors) : step_tiles<kMaster, false, kSmall>(t, begin, whole, s, k, factors);
    else if (t.index_flags & kParamBf16) g ? step_tiles<kBf16, true, kSmall>(t, begin, whole, s, k, factors) : step_tiles<kBf16, false, kSmall>(t, begin, whole, s, k, factors);
    else g ? step_tiles<kF32, true, kSmall>(t, begin, whole, s, k, factors) : step_tiles<kF32, false, kSmall>(t, begin, whole, s, k, factors);
    for (int64_t i0 = whole; i0 < end; i0 += kTile) {
      const int64_t i = i0 + threadIdx.x * kPer;
      step_rest<kSmall>(t, i, end, s, k, factors + (int)(i - begin) / 128);
    }
    if constexpr (kSmall) {
      __syncthreads();
      for (int j = threadIdx.x; j < blocks; j += kThreads) {
        t.m_scales[block0 + j] = factors[j];
        t.v_scales[block0 + j] = factors[kMostBlocks + j];
        if (factors[kMostBlocks + j] == kLargestFactor)
          keep_squares_finite(static_cast<uint8_t*>(t.v) + begin + 128 * j, (int)min((int64_t)128, end - begin - 128 * j));
      }
    }
  }
  if (raise) {
    __threadfence();  // every CTA's read of the steps lies before what follows
    *s.ticket = 0;
    if (!skip) *s.steps = taken;
  }
}

// A step without values: only its number.
__global__ void empty_step_kernel(const float* factor, int64_t* steps) {
  pdl_wait();
  pdl_launch_dependents();
  if (!factor || isfinite(*factor)) ++*steps;
}

template <int kN, bool kSmall>
cudaError_t launch_list(const Entry* e, int n, const Step& s, cudaStream_t st) {
  constexpr int kTile = Ctas<kSmall>::kTile;
  Batch<kN> b;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) tiles += (e[i].n + kTile - 1) / kTile;
  b.n = n;
  b.chunk = kTile;
  while (b.chunk < Ctas<kSmall>::kTiles * kTile && tiles * kTile >= 2 * (int64_t)Ctas<kSmall>::kFew * b.chunk) b.chunk *= 2;
  b.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    b.e[i] = e[i];
    b.first[i + 1] = b.first[i] + (uint32_t)((e[i].n + b.chunk - 1) / b.chunk);
  }
  return launch_kernel(adamw_kernel<kN, kSmall>, dim3(b.first[n]), dim3(Ctas<kSmall>::kThreads), 0, st, true, 1, b, s);
}

template <bool kSmall>
cudaError_t launch_lists(const Entry* e, int n, const Step& s, cudaStream_t st) {
  return n <= 24    ? launch_list<24, kSmall>(e, n, s, st)
         : n <= 100 ? launch_list<100, kSmall>(e, n, s, st)
                    : launch_list<kMostTensors, kSmall>(e, n, s, st);
}

// ------------------------------------------------------------------ the norm

constexpr int kThreads = 256, kTile = kThreads * kPer;
constexpr int kNormTiles = 4, kNormChunk = kNormTiles * kTile;  // 32 values a thread, all under way at once

// The sum of a warp's squares of a chunk, in fp32.
template <bool kBf16>
__device__ __forceinline__ float sum_of_squares(const GradEntry& e, int64_t begin, int64_t end) {
  P4 g[kNormTiles];
  if (e.vec && end - begin == kNormChunk) {
    Raw<kBf16 ? 2 : 4> r[kNormTiles];
#pragma unroll
    for (int u = 0; u < kNormTiles; ++u) r[u].load(e.g, begin + u * kTile + threadIdx.x * kPer);
#pragma unroll
    for (int u = 0; u < kNormTiles; ++u) g[u] = r[u].get();
  } else {
#pragma unroll
    for (int u = 0; u < kNormTiles; ++u) {
      const int64_t i = begin + u * kTile + threadIdx.x * kPer;
      const F8 r = load(e.g, i, kBf16, (int)max((int64_t)0, min(end - i, (int64_t)kPer)));
#pragma unroll
      for (int j = 0; j < 4; ++j) g[u].v[j] = make_float2(r.v[2 * j], r.v[2 * j + 1]);
    }
  }
  float2 sum[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sum[j] = mul2(g[0].v[j], g[0].v[j]);
#pragma unroll
  for (int u = 1; u < kNormTiles; ++u)
#pragma unroll
    for (int j = 0; j < 4; ++j) sum[j] = fma2(g[u].v[j], g[u].v[j], sum[j]);
  const float2 s = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
  float all = s.x + s.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
  return all;
}

// The sum of a warp's squares of all its chunks in 64 bits, for what fp32 does not hold.
template <int kN>
__device__ __noinline__ double wide_sum_of_squares(const GradBatch<kN>& b) {
  double all = 0;
  for (uint32_t chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    const int ti = owner(b, chunk);
    const GradEntry& e = b.e[ti];
    const int64_t begin = (int64_t)(chunk - b.first[ti]) * kNormChunk, end = min(begin + kNormChunk, e.n);
    for (int64_t i = begin + threadIdx.x * kPer; i < end; i += kTile) {
      const F8 r = load(e.g, i, e.bf16, (int)min(end - i, (int64_t)kPer));
      for (int j = 0; j < kPer; ++j) all += (double)(r.v[j] * r.v[j]);
    }
  }
  for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(kAll, all, o);
  return all;
}

// The sum of the warps' first lanes' values, in the block's first thread.  A sum in 64 bits takes a warp several times
// as long as one in fp32, and they follow one another here: as few of them as can be.
__device__ __forceinline__ double sum_of_warps(double v) {
  constexpr int kWarps = kThreads / 32;
  __shared__ double of_warp[kWarps];
  __syncthreads();  // of_warp may still be read
  if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x < 32) {
    v = threadIdx.x < kWarps ? of_warp[threadIdx.x] : 0;
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  }
  return v;
}

struct NormOut {
  double* parts;     // of all launches; this one's are behind `before` others
  uint32_t* ticket;  // null: not the last launch
  int before;
  float max_norm;
  float *norm, *factor;
};

// parts[CTA]: the sum of squares of its chunks, one in gridDim.x of all.  Of the last launch the CTA that is done last
// adds all parts up, in their order.
template <int kN>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ GradBatch<kN> b, const NormOut out) {
  __shared__ bool ends;
  pdl_wait();
  pdl_launch_dependents();
  float sum = 0.f, lost = 0.f;
  for (uint32_t chunk = blockIdx.x; chunk < b.first[b.n]; chunk += gridDim.x) {
    const int ti = owner(b, chunk);
    const GradEntry& e = b.e[ti];
    const int64_t begin = (int64_t)(chunk - b.first[ti]) * kNormChunk, end = min(begin + kNormChunk, e.n);
    const float v = e.bf16 ? sum_of_squares<true>(e, begin, end) : sum_of_squares<false>(e, begin, end);
    // what the sum loses is kept beside it: as good as 64 bits, whose additions an SM has few units for
    const float t = sum + v, part = t - sum;
    lost += (sum - (t - part)) + (v - part);
    sum = t;
  }
  double total = (double)sum + (double)lost;
  if (!isfinite(sum)) total = wide_sum_of_squares(b);  // a warp's lanes have the same sum
  total = sum_of_warps(total);
  if (threadIdx.x == 0) {
    out.parts[out.before + blockIdx.x] = total;
    ends = false;
    if (out.ticket) {
      __threadfence();  // the part is there before the ticket is
      ends = atomicAdd(out.ticket, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!ends) return;
  __threadfence();
  total = 0;
  for (int i = threadIdx.x; i < out.before + (int)gridDim.x; i += kThreads) total += __ldcg(out.parts + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
  total = sum_of_warps(total);
  if (threadIdx.x == 0) {
    const float r = (float)sqrt(total);
    *out.ticket = 0;
    *out.norm = r;
    if (out.factor) *out.factor = isfinite(r) ? (r > out.max_norm ? out.max_norm / r : 1.f) : __uint_as_float(0x7fffffffu);
  }
}

template <int kN>
cudaError_t launch_norm_list(const GradEntry* e, int n, NormOut& out, uint32_t* ticket, cudaStream_t st) {
  GradBatch<kN> b;
  b.n = n;
  b.first[0] = 0;
  for (int i = 0; i < n; ++i) {
    b.e[i] = e[i];
    b.first[i + 1] = b.first[i] + (uint32_t)((e[i].n + kNormChunk - 1) / kNormChunk);
  }
  const unsigned grid = b.first[n] > (unsigned)kNormCtas ? (unsigned)kNormCtas : b.first[n] > 0 ? b.first[n] : 1;
  out.ticket = ticket;
  const cudaError_t err = launch_kernel(norm_kernel<kN>, dim3(grid), dim3(kThreads), 0, st, true, 1, b, out);
  out.before += (int)grid;
  return err;
}

bool on(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

}  // namespace

cudaError_t launch_adamw(const moe_adamw_tensor* tensors, int n, const moe_adamw_config& cfg, const float* factor, int64_t* steps,
                         uint32_t* ticket, cudaStream_t st) {
  Step s{};
  s.lr = (float)cfg.lr;
  s.lr_device = cfg.lr_device;
  s.b1 = (float)cfg.beta1;
  s.b2 = (float)cfg.beta2;
  s.c1 = (float)(1 - cfg.beta1);
  s.c2 = (float)(1 - cfg.beta2);
  s.slow = s.c1 <= 0.5f && s.c2 <= 0.5f;
  s.a = s.slow ? ldexpf(1.f, (ilogbf(s.c2) - (ilogbf(s.c2) & 1)) / 2) : 1.f;
  s.neg_a2 = -s.a * s.a;
  s.c1 /= s.a;
  s.c2 /= s.a * s.a;
  s.eps = (float)cfg.eps;
  s.log1 = (float)log(cfg.beta1);
  s.log2 = (float)log(cfg.beta2);
  s.factor = factor;
  s.steps = steps;
  s.ticket = ticket;
  s.seed_low = (uint32_t)cfg.seed;
  s.seed_high = (uint32_t)(cfg.seed >> 32);
  int left[2] = {0, 0};  // tensors with moments in 32 bits, in 8
  for (int i = 0; i < n; ++i) left[tensors[i].m_scales != nullptr] += tensors[i].n > 0;
  if (left[0] + left[1] == 0) return launch_kernel(empty_step_kernel, dim3(1), dim3(1), 0, st, true, 1, factor, steps);
  Entry e[kMostTensors];
  for (const bool small : {true, false})
    for (int i = 0; left[small] > 0;) {
      int m = 0;
      for (; i < n && m < kMostTensors; ++i) {
        const moe_adamw_tensor& t = tensors[i];
        if (t.n == 0 || (t.m_scales != nullptr) != small) continue;
        const uintptr_t moments = small ? 8 : 16;
        const bool vec = on(t.param, 16) && on(t.master, 16) && on(t.grad, 16) && on(t.m, moments) && on(t.v, moments);
        e[m++] = {t.param, t.master, t.grad, t.m, t.v, t.m_scales, t.v_scales, t.n, t.weight_decay,
                  (uint32_t)i << kIndexShift | (t.param_dtype == MOE_BF16 ? kParamBf16 : 0) | (t.grad_dtype == MOE_BF16 ? kGradBf16 : 0) | (vec ? kVec : 0)};
      }
      left[small] -= m;
      s.last = left[0] + left[1] == 0;
      const cudaError_t err = small ? launch_lists<true>(e, m, s, st) : launch_lists<false>(e, m, s, st);
      if (err != cudaSuccess) return err;
    }
  return cudaSuccess;
}

cudaError_t launch_grad_norm(const moe_grad_tensor* tensors, int n, float max_norm, float* norm, float* factor, void* workspace,
                             cudaStream_t st) {
  NormOut out{static_cast<double*>(workspace) + 1, nullptr, 0, max_norm, norm, factor};
  GradEntry e[kMostTensors];
  int left = 0;  // tensors with values
  for (int i = 0; i < n; ++i) left += tensors[i].n > 0;
  int i = 0;
  do {  // without values: one CTA that finds a sum of 0
    int m = 0;
    for (; i < n && m < kMostTensors; ++i) {
      const moe_grad_tensor& t = tensors[i];
      if (t.n > 0) e[m++] = {t.grad, t.n, t.dtype == MOE_BF16, on(t.grad, 16)};
    }
    left -= m;
    uint32_t* ticket = left == 0 ? static_cast<uint32_t*>(workspace) : nullptr;
    const cudaError_t err = m <= 100 ? launch_norm_list<100>(e, m, out, ticket, st) : launch_norm_list<kMostTensors>(e, m, out, ticket, st);
    if (err != cudaSuccess) return err;
  } while (left > 0);
  return cudaSuccess;
}

}  // namespace optim
}  // namespace moe
