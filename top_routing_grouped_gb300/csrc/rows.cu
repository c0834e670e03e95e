// rows.cu -- tokens sorted by expert and back with gates applied, and the gradients (include/moe_rows.h).
//
// All of it moves rows: a few operations a byte, so HBM bounds the large calls and the launch the small ones.
#include <cuda_bf16.h>

#include "device_common.cuh"
#include "rows_internal.h"

namespace moe {
namespace rows {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ sort and gather

template <bool kIdx64>
__device__ __forceinline__ int expert_of(const Args& a, int64_t slot) {
  if constexpr (kIdx64) {
    const long long v = static_cast<const long long*>(a.idx)[slot];
    return (unsigned long long)v < (unsigned long long)a.E ? (int)v : -1;
  } else {
    const int v = static_cast<const int*>(a.idx)[slot];
    return (unsigned)v < (unsigned)a.E ? v : -1;
  }
}

// table[e] += the slots of expert e among [from, to), by all threads of the block; `also`: a second table
// for those below `below`.  Lanes of one expert add once, together.
template <bool kIdx64>
__device__ __forceinline__ void count(const Args& a, int64_t from, int64_t to, int* table, int64_t below, int* also) {
  constexpr int kU = 8;  // loads in flight
  for (int64_t i0 = from; i0 < to; i0 += kU * kThreads) {
    int e[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = i0 + u * kThreads + threadIdx.x;
      e[u] = i < to ? expert_of<kIdx64>(a, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = i0 + u * kThreads + threadIdx.x;
      if (i0 + u * kThreads >= to) break;  // the same for the whole block
      const unsigned same = __match_any_sync(kAll, e[u]);
      const unsigned early = __ballot_sync(kAll, i < below) & same;
      if (e[u] >= 0 && (int)(threadIdx.x & 31) == __ffs(same) - 1) {
        atomicAdd(&table[e[u]], __popc(same));
        if (also && early) atomicAdd(&also[e[u]], __popc(early));
      }
    }
  }
}

int64_t count_slots(int64_t N) { return (N + kCountBlocks - 1) / kCountBlocks; }

// counted[b][e]: the slots of expert e in the b-th block of per_block slots.
template <bool kIdx64>
__global__ void __launch_bounds__(kThreads) count_kernel(Args a, int64_t per_block, int32_t* counted) {
  extern __shared__ int table[];
  for (int e = threadIdx.x; e < a.E; e += kThreads) table[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t N = a.T * a.k, from = blockIdx.x * per_block;
  count<kIdx64>(a, from, min(from + per_block, N), table, 0, nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += kThreads) counted[(int64_t)blockIdx.x * a.E + e] = table[e];
}

// A counting sort in one pass, and the rows' way with it.  Each CTA takes `tokens` tokens (grid.y: a share
// of their columns).  Where its slots' rows begin follows from the experts' totals and from the slots
// before its own: of up to 16384 slots it counts them all by itself (64 KB out of L2, 1 us, where another launch
// takes 2); of more it adds up what count_kernel counted in 64 blocks and counts the rest of its own
// block.  Inside the CTA each warp ranks a run of slots, 32 at a time, behind the warps before it, so that
// the order is that of the slots whatever the timing.
template <typename V, bool kSort, bool kIdx64>
__global__ void __launch_bounds__(kThreads) rows_kernel(Args a, int tokens, int64_t vecs_y, const int32_t* counted, int64_t per_block) {
  extern __shared__ int shared[];
  __shared__ int warp_sum[kWarps];
  int* pos = shared;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
  const int64_t t0 = (int64_t)blockIdx.x * tokens, s0 = t0 * a.k, N = a.T * a.k;
  const int nt = (int)min((int64_t)tokens, a.T - t0), own = nt * a.k;
  const bool first = blockIdx.y == 0;  // writes what does not depend on the columns

  if constexpr (!kSort) {
    pdl_wait();
    pdl_launch_dependents();
    for (int i = threadIdx.x; i < own; i += kThreads) {
      const int p = a.slot_pos[s0 + i];
      pos[i] = p;
      if (first && a.gates && p >= 0 && p < a.R) a.row_gates[p] = a.gates[s0 + i];
    }
  } else {
    int *total = shared + tokens * a.k, *before = total + E, *of_warp = before + E;  // [E], [E], [kWarps][E]
    for (int e = threadIdx.x; e < (2 + kWarps) * E; e += kThreads) total[e] = 0;
    pdl_wait();
    pdl_launch_dependents();
    __syncthreads();
    if (counted) {
      const int blocks = (int)((N + per_block - 1) / per_block), mine = (int)(s0 / per_block);
      const int groups = E < kThreads ? kThreads / E : 1;
      for (int i = threadIdx.x; i < groups * E; i += kThreads) {
        const int e = i % E, g = i / E;
        int all = 0, less = 0;
#pragma unroll 8
        for (int b = g; b < blocks; b += groups) {
          const int c = counted[(int64_t)b * E + e];
          all += c;
          less += b < mine ? c : 0;
        }
        if (all) atomicAdd(&total[e], all);
        if (less) atomicAdd(&before[e], less);
      }
      count<kIdx64>(a, mine * per_block, s0, before, 0, nullptr);
    } else {
      count<kIdx64>(a, 0, N, total, s0, before);
    }
    // its own slots, by warp
    const int run = (own + kThreads - 1) / kThreads * 32, w0 = warp * run, w1 = min(w0 + run, own);
    int* mine = of_warp + warp * E;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int e = i0 + lane < w1 ? expert_of<kIdx64>(a, s0 + i0 + lane) : -1;
      const unsigned same = __match_any_sync(kAll, e);
      if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
      __syncwarp();
    }
    __syncthreads();
    if (first && blockIdx.x == 0)
      for (int e = threadIdx.x; e < E; e += kThreads) a.counts[e] = total[e];
    // exclusive scan of the totals: four experts a thread at most
    const int each = (E + kThreads - 1) / kThreads;
    int v[kMaxSortExperts / kThreads], sum = 0;
#pragma unroll
    for (int i = 0; i < kMaxSortExperts / kThreads; ++i) {
      const int e = threadIdx.x * each + i;
      v[i] = i < each && e < E ? total[e] : 0;
      sum += v[i];
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += n;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int at = incl - sum, kept = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) at += warp_sum[w];
      kept += warp_sum[w];
    }
#pragma unroll
    for (int i = 0; i < kMaxSortExperts / kThreads; ++i) {
      const int e = threadIdx.x * each + i;
      if (i < each && e < E) {
        int next = at + before[e];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const int n = of_warp[w * E + e];
          of_warp[w * E + e] = next;
          next += n;
        }
        at += v[i];
      }
    }
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const int e = i < w1 ? expert_of<kIdx64>(a, s0 + i) : -1;
      const unsigned same = __match_any_sync(kAll, e);
      int p = -1;
      if (e >= 0) p = mine[e] + __popc(same & ((1u << lane) - 1));
      __syncwarp();
      if (e >= 0 && lane == __ffs(same) - 1) mine[e] += __popc(same);
      __syncwarp();
      if (i < w1) {
        pos[i] = p;
        if (first) {
          a.slot_pos[s0 + i] = p;
          if (p >= 0) {
            if (a.row_slot) a.row_slot[p] = (int)(s0 + i);
            if (a.gates && p < a.R) a.row_gates[p] = a.gates[s0 + i];
          }
          if (a.row_slot && s0 + i >= kept) a.row_slot[s0 + i] = -1;
        }
      }
    }
  }
  __syncthreads();
  if (a.row_bytes == 0) return;

  // the rows: a warp takes 32 kU vectors of one token, reads them once and writes them to each of its rows
  constexpr int kU = 4;
  const int64_t vecs = a.row_bytes / (int64_t)sizeof(V), v_first = blockIdx.y * vecs_y, v_end = min(v_first + vecs_y, vecs);
  const int segs = (int)((v_end - v_first + 32 * kU - 1) / (32 * kU));
  for (int unit = warp; unit < nt * segs; unit += kWarps) {
    const int t = unit / segs;
    const int64_t v0 = v_first + (int64_t)(unit - t * segs) * 32 * kU + lane;
    const V* src = reinterpret_cast<const V*>(a.x + (t0 + t) * a.ld_bytes);
    V buf[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + u * 32 < v_end) buf[u] = __ldcs(src + v0 + u * 32);
    for (int j = 0; j < a.k; ++j) {
      const int p = pos[t * a.k + j];
      if (p < 0 || p >= a.R) continue;
      V* dst = reinterpret_cast<V*>(a.x_rows + p * a.row_bytes);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (v0 + u * 32 < v_end) dst[v0 + u * 32] = buf[u];
    }
  }
  if (a.words && first) {
    const int64_t n = nt * a.words;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
      const int64_t t = i / a.words, w = i - t * a.words;
      const uint32_t f = a.x_words[(t0 + t) * a.words + w];
      for (int j = 0; j < a.k; ++j) {
        const int p = pos[t * a.k + j];
        if (p >= 0 && p < a.R) a.row_words[p * a.words + w] = f;
      }
    }
  }
}

template <typename V, bool kSort, bool kIdx64>
cudaError_t launch_as(const Args& a, int32_t* counted, cudaStream_t st) {
  constexpr int64_t kCtas = 152 * 8;
  const int64_t vecs = a.row_bytes / (int64_t)sizeof(V), segs = (vecs + 127) / 128;  // as the kernel's kU = 4 has them
  // tokens a CTA: enough CTAs to fill the GPU several times, of eight warps' work each; a sort's shared
  // memory holds 4096 positions.  Without rows to move: a slot for each thread.
  int64_t tokens = (a.T + kCtas - 1) / kCtas;
  const int64_t least = segs ? (8 + segs - 1) / segs : (kThreads + a.k - 1) / a.k;
  if (tokens < least) tokens = least;
  if (tokens > 4096 / a.k) tokens = 4096 / a.k;
  if (tokens > a.T) tokens = a.T;
  const int64_t gx = (a.T + tokens - 1) / tokens;
  // columns of a few tokens' long rows are shared out
  int64_t gy = 1, vecs_y = vecs;
  if (segs > 0 && gx < kCtas / 2) {
    gy = (tokens * segs + 7) / 8;
    if (gy > kCtas / 2 / gx) gy = kCtas / 2 / gx;
    if (gy > segs) gy = segs;
    vecs_y = (segs + gy - 1) / gy * 128;
    gy = (vecs + vecs_y - 1) / vecs_y;
  }
  size_t smem = (size_t)tokens * a.k * sizeof(int);
  int64_t per_block = 0;
  if constexpr (kSort) {
    smem += (size_t)(2 + kWarps) * a.E * sizeof(int);
    if (counted) {
      per_block = count_slots(a.T * a.k);
      const int64_t blocks = (a.T * a.k + per_block - 1) / per_block;
      const cudaError_t e = launch_kernel(count_kernel<kIdx64>, dim3((unsigned)blocks), dim3(kThreads), (size_t)a.E * sizeof(int), st,
                                          true, 1, a, per_block, counted);
      if (e != cudaSuccess) return e;
    }
  }
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(rows_kernel<V, kSort, kIdx64>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(rows_kernel<V, kSort, kIdx64>, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), smem, st, true, 1, a,
                       (int)tokens, vecs_y, (const int32_t*)counted, per_block);
}

template <typename V>
cudaError_t launch_vec(const Args& a, int32_t* counted, cudaStream_t st) {
  if (!a.idx) return launch_as<V, false, false>(a, nullptr, st);
  return a.idx64 ? launch_as<V, true, true>(a, counted, st) : launch_as<V, true, false>(a, counted, st);
}

// ------------------------------------------------------------------ combine

// n values of type T on a boundary of n * sizeof(T) bytes (16 at most at a time), to and from fp32
template <typename T, int n>
struct Values {
  static constexpr int kBytes = n * (int)sizeof(T) < 16 ? n * (int)sizeof(T) : 16, kParts = n * (int)sizeof(T) / kBytes;
  using Part = typename std::conditional<kBytes == 16, uint4,
               typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
  Part part[kParts];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) part[i] = __ldcs(reinterpret_cast<const Part*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) reinterpret_cast<Part*>(p)[i] = part[i];
  }
  __device__ __forceinline__ float get(int i) const {
    const T v = reinterpret_cast<const T*>(part)[i];
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
  }
  __device__ __forceinline__ void set(int i, float v) {
    if constexpr (sizeof(T) == 2) reinterpret_cast<T*>(part)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<T*>(part)[i] = v;
  }
};

// One warp for 32 V columns of one token: up to four rows in flight, summed in the slots' order.
template <typename Ty, typename To, int V>
__global__ void __launch_bounds__(kThreads) combine_kernel(const Ty* y, int64_t R, const int32_t* slot_pos, const float* gates,
                                                           int64_t T, int k, int64_t d, unsigned segs, const To* residual, To* out) {
  const int lane = threadIdx.x & 31;
  const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t t = unit <= 0xffffffffll ? (int64_t)((unsigned)unit / segs) : unit / segs;
  pdl_wait();
  pdl_launch_dependents();
  if (t >= T) return;
  const int64_t c = ((unit - t * segs) * 32 + lane) * V;
  const bool ok = c < d;
  Values<To, V> res;
  if (residual && ok) res.load(residual + t * d + c);
  float acc[V];
#pragma unroll
  for (int i = 0; i < V; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < k; j0 += 32) {
    const int n = min(32, k - j0);
    int p = -1;
    float g = 1.f;
    if (lane < n) {
      p = slot_pos[t * k + j0 + lane];
      if (gates) g = gates[t * k + j0 + lane];
    }
    if (p >= R) p = -1;
    for (int j = 0; j < n; j += 4) {
      Values<Ty, V> row[4];
      int at[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        at[q] = __shfl_sync(kAll, p, j + q);  // lanes past n hold -1
        if (at[q] >= 0 && ok) row[q].load(y + at[q] * d + c);
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float gq = __shfl_sync(kAll, g, j + q);
        if (at[q] >= 0) {
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = fmaf(gq, row[q].get(i), acc[i]);
        }
      }
    }
  }
  if (!ok) return;
  Values<To, V> o;
#pragma unroll
  for (int i = 0; i < V; ++i) o.set(i, residual ? res.get(i) + acc[i] : acc[i]);
  o.store(out + t * d + c);
}

template <typename Ty, typename To, int V>
cudaError_t combine_as(const void* y, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T, int k, int64_t d,
                       const void* residual, void* out, cudaStream_t st) {
  const int64_t segs = (d + 32 * V - 1) / (32 * V), blocks = (T * segs + kWarps - 1) / kWarps;
  return launch_kernel(combine_kernel<Ty, To, V>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, 1, static_cast<const Ty*>(y), R,
                       slot_pos, gates, T, k, d, (unsigned)segs, static_cast<const To*>(residual), static_cast<To*>(out));
}

// The gradients: kPer warps a token, each lane V columns at a time of up to eight rows; the products with dout
// are summed over the lanes, and over the warps in order.
template <typename Td, typename Ty, int V>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const Td* dout, const int32_t* slot_pos, const float* gates,
                                                                    int64_t T, int k, int64_t d, int64_t R, const Ty* y, Ty* dy,
                                                                    float* dgates, int per) {
  constexpr int kRows = 8;
  __shared__ float part[kWarps][kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % per;
  const int64_t t = (int64_t)blockIdx.x * (kWarps / per) + warp / per;
  pdl_wait();
  pdl_launch_dependents();
  const bool has = t < T;
  for (int j0 = 0; j0 < k; j0 += kRows) {
    const int n = min(kRows, k - j0);
    int p = -1;
    float g = 1.f;
    if (has && lane < n) {
      p = slot_pos[t * k + j0 + lane];
      if (gates) g = gates[t * k + j0 + lane];
    }
    if (p >= R) p = -1;
    int at[kRows];
    float gate[kRows], dot[kRows];
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      at[q] = __shfl_sync(kAll, p, q);
      gate[q] = __shfl_sync(kAll, g, q);
      dot[q] = 0.f;
    }
    if (has) {
      for (int64_t c = (mine * 32 + lane) * V; c < d; c += per * 32 * V) {
        Values<Td, V> go;
        go.load(dout + t * d + c);
        Values<Ty, V> row[kRows];
        if (dgates) {
#pragma unroll
          for (int q = 0; q < kRows; ++q)
            if (at[q] >= 0) row[q].load(y + at[q] * d + c);
        }
#pragma unroll
        for (int q = 0; q < kRows; ++q) {
          if (at[q] < 0) continue;
          if (dgates) {
#pragma unroll
            for (int i = 0; i < V; ++i) dot[q] = fmaf(go.get(i), row[q].get(i), dot[q]);
          }
          if (dy) {
            Values<Ty, V> o;
#pragma unroll
            for (int i = 0; i < V; ++i) o.set(i, gate[q] * go.get(i));
            o.store(dy + at[q] * d + c);
          }
        }
      }
    }
    if (dgates) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kRows; ++q) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot[q] += __shfl_xor_sync(kAll, dot[q], o);
        if (lane == q) sum = dot[q];
      }
      if (per > 1) {
        if (lane < kRows) part[warp][lane] = sum;
        __syncthreads();
        if (mine == 0 && lane < n) {
          sum = 0.f;
          for (int w = 0; w < per; ++w) sum += part[warp + w][lane];
        }
        __syncthreads();
      }
      if (has && mine == 0 && lane < n) dgates[t * k + j0 + lane] = sum;
    }
  }
}

template <typename Td, typename Ty, int V>
cudaError_t backward_as(const void* dout, const int32_t* slot_pos, const float* gates, int64_t T, int k, int64_t d, int64_t R,
                        const void* y, void* dy, float* dgates, cudaStream_t st) {
  // warps a token: as many as have columns, until the GPU's warps have a token each
  int per = 1;
  while (per < kWarps && (int64_t)per * 32 * V < d && T * per < 152 * 32) per *= 2;
  const int64_t blocks = (T + kWarps / per - 1) / (kWarps / per);
  return launch_kernel(combine_backward_kernel<Td, Ty, V>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, 1,
                       static_cast<const Td*>(dout), slot_pos, gates, T, k, d, R, static_cast<const Ty*>(y), static_cast<Ty*>(dy),
                       dgates, per);
}

// The most values, of `most`, that divide a row and that all these addresses are on boundaries of (16 bytes do
// for more than 16).
int values_at_once(int most, int64_t d, std::initializer_list<std::pair<const void*, int>> arrays) {
  for (; most > 1; most /= 2) {
    bool fits = d % most == 0;
    for (const auto& [p, size] : arrays) fits = fits && reinterpret_cast<uintptr_t>(p) % (most * size < 16 ? most * size : 16) == 0;
    if (fits) break;
  }
  return most;
}

}  // namespace

// One launch for all is the faster up to here (see rows_kernel).
bool counts_first(int64_t N) { return N > 16384; }

cudaError_t launch_rows(const Args& a, int32_t* counted, cudaStream_t st) {
  const uintptr_t b = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.x_rows) | (uintptr_t)a.row_bytes | (uintptr_t)a.ld_bytes;
  if (b % 16 == 0) return launch_vec<uint4>(a, counted, st);
  if (b % 8 == 0) return launch_vec<uint2>(a, counted, st);
  if (b % 4 == 0) return launch_vec<uint32_t>(a, counted, st);
  if (b % 2 == 0) return launch_vec<uint16_t>(a, counted, st);
  return launch_vec<uint8_t>(a, counted, st);
}

using bf16 = __nv_bfloat16;

cudaError_t launch_combine(const void* y, bool y_bf16, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T, int k,
                           int64_t d, const void* residual, void* out, bool out_bf16, cudaStream_t st) {
  const int v = values_at_once(y_bf16 ? 8 : 4, d, {{y, y_bf16 ? 2 : 4}, {residual, out_bf16 ? 2 : 4}, {out, out_bf16 ? 2 : 4}});
  const auto with = [&](auto ty, auto to) {
    using Ty = decltype(ty);
    using To = decltype(to);
    if constexpr (sizeof(Ty) == 2)
      if (v == 8) return combine_as<Ty, To, 8>(y, R, slot_pos, gates, T, k, d, residual, out, st);
    return v == 4   ? combine_as<Ty, To, 4>(y, R, slot_pos, gates, T, k, d, residual, out, st)
           : v == 2 ? combine_as<Ty, To, 2>(y, R, slot_pos, gates, T, k, d, residual, out, st)
                    : combine_as<Ty, To, 1>(y, R, slot_pos, gates, T, k, d, residual, out, st);
  };
  if (y_bf16) return out_bf16 ? with(bf16(), bf16()) : with(bf16(), float());
  return out_bf16 ? with(float(), bf16()) : with(float(), float());
}

cudaError_t launch_combine_backward(const void* dout, bool dout_bf16, const int32_t* slot_pos, const float* gates, int64_t T, int k,
                                    int64_t d, int64_t R, const void* y, void* dy, bool y_bf16, float* dgates, cudaStream_t st) {
  const int v = values_at_once(y_bf16 ? 8 : 4, d, {{dout, dout_bf16 ? 2 : 4}, {y, y_bf16 ? 2 : 4}, {dy, y_bf16 ? 2 : 4}});
  const auto with = [&](auto td, auto ty) {
    using Td = decltype(td);
    using Ty = decltype(ty);
    if constexpr (sizeof(Ty) == 2)
      if (v == 8) return backward_as<Td, Ty, 8>(dout, slot_pos, gates, T, k, d, R, y, dy, dgates, st);
    return v == 4   ? backward_as<Td, Ty, 4>(dout, slot_pos, gates, T, k, d, R, y, dy, dgates, st)
           : v == 2 ? backward_as<Td, Ty, 2>(dout, slot_pos, gates, T, k, d, R, y, dy, dgates, st)
                    : backward_as<Td, Ty, 1>(dout, slot_pos, gates, T, k, d, R, y, dy, dgates, st);
  };
  if (dout_bf16) return y_bf16 ? with(bf16(), bf16()) : with(bf16(), float());
  return y_bf16 ? with(float(), bf16()) : with(float(), float());
}

}  // namespace rows
}  // namespace moe
