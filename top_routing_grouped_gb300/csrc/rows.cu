// rows.cu -- tokens sorted by expert and back with gates applied, and the gradients (include/moe_rows.h).
//
// All of it moves rows: a few operations a byte, so HBM bounds the large calls and the launch the small ones.
#include <cuda_bf16.h>

#include <initializer_list>
#include <type_traits>
#include <utility>

#include "device_common.cuh"
#include "rows_internal.h"

namespace moe {
namespace rows {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 128;             // vectors of a row that a warp moves at a time, four a lane
constexpr int kMaxPositions = 4096;    // that a CTA keeps
// Up to kSortFew slots each CTA that moves rows counts them all by itself, with kSortCtas such CTAs at most; more are sorted
// in launches of their own.  In CUDA graphs, one launch and two or three: 2000 tokens' two rows of 1000 bf16 5.1 and
// 6.5 us, 1100 tokens' four of 2048 6.9 and 8.1, 1500 tokens' four of 2048 8.1 and 9.2, 760 tokens' eight of 1024 6.8 and 8.4;
// 1029 tokens' eight of 2050 10.8 and 9.8, 4096 tokens' two of 512 6.7 and 6.4, 4000 tokens' four of 256 10.0 and 7.2.
// With 152 CTAs: within 3 % up to 8192 slots but for one 10 % slower.
constexpr int64_t kSortFew = 6144;
constexpr int kSortCtas = 152 * 2;
// Up to kWarpSlots (32 at most) a warp compares with one another, a turn for each.  In a CUDA graph, against counting: 4 slots
// 2.3 and 3.3 us, 16 slots 3.4 and 4.0, 24 slots 3.7 and 4.0, 32 slots 4.15 and 4.0.
constexpr int kWarpSlots = 24;
constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ rows off 16-byte boundaries

// Sixteen bytes from any address, out of the two 16-byte words of memory that they lie in; [lo, hi) is what may be
// read.  Two loads and a shift: that pays for moving rows off 4-byte boundaries, not for others and not where the rows are
// computed with (16384 tokens to 4 rows each; loads of the alignment's own size -> this: moving 4095 bytes 145 -> 74 us,
// 2047 bf16 82 -> 71, 1023 fp32 59 -> 72; combining 2047 bf16 121 -> 138 us; its backward 153 -> 189).
__device__ __forceinline__ uint4 load_any(const void* at, const void* lo, const void* hi) {
  const char* p = static_cast<const char*>(at);
  const int off = (int)(reinterpret_cast<uintptr_t>(p) & 15);
  const char* base = p - off;
  if (off == 0) return *reinterpret_cast<const uint4*>(base);
  if (base < lo || base + 32 > hi) {  // at an array's ends
    uint64_t w[2] = {0, 0};
#pragma unroll 1
    for (int i = 0; i < 16; ++i) {
      const uint64_t v = (uint64_t)(uint8_t)p[i] << 8 * (i & 7);
      w[0] |= i < 8 ? v : 0;
      w[1] |= i < 8 ? 0 : v;
    }
    return make_uint4((uint32_t)w[0], (uint32_t)(w[0] >> 32), (uint32_t)w[1], (uint32_t)(w[1] >> 32));
  }
  const uint4 a = reinterpret_cast<const uint4*>(base)[0], b = reinterpret_cast<const uint4*>(base)[1];
  const bool two = off & 8, one = off & 4;
  const uint32_t w0 = two ? a.z : a.x, w1 = two ? a.w : a.y, w2 = two ? b.x : a.z, w3 = two ? b.y : a.w, w4 = two ? b.z : b.x, w5 = two ? b.w : b.y;
  const uint32_t x0 = one ? w1 : w0, x1 = one ? w2 : w1, x2 = one ? w3 : w2, x3 = one ? w4 : w3, x4 = one ? w5 : w4;
  const int bits = off % 4 * 8;
  return make_uint4(__funnelshift_r(x0, x1, bits), __funnelshift_r(x1, x2, bits), __funnelshift_r(x2, x3, bits), __funnelshift_r(x3, x4, bits));
}

// Lanes that share a token: all 32, or as few as hold a short row's `pieces`.  The kernels know 32 beforehand (kLanes;
// 0: what they are given), which saves a third of the registers of some.
int lanes_for(int64_t pieces) {
  int n = 8;
  while (n < 32 && n < pieces) n *= 2;
  return n;
}

// ------------------------------------------------------------------ sort and gather

// Read out of L2, past L1: a kernel may do so before it has waited for the one before it (sort_kernel, rows_kernel).
template <bool kIdx64>
__device__ __forceinline__ int expert_of(const Args& a, int64_t slot) {
  if constexpr (kIdx64) {
    const long long v = __ldcg(static_cast<const long long*>(a.idx) + slot);
    return (unsigned long long)v < (unsigned long long)a.E ? (int)v : -1;
  } else {
    const int v = __ldcg(static_cast<const int*>(a.idx) + slot);
    return (unsigned)v < (unsigned)a.E ? v : -1;
  }
}

// Counts each expert's slots among [from, to), by all threads of the block: those below `split` in low[e], the others
// in high[e].
template <bool kIdx64, int kThreadsOf>
__device__ __forceinline__ void count(const Args& a, int64_t from, int64_t to, int64_t split, int* low, int* high) {
  constexpr int kU = 8;  // loads in flight
  for (int64_t i0 = from + threadIdx.x; i0 < to; i0 += kU * kThreadsOf) {
    int e[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t i = i0 + u * kThreadsOf;
      e[u] = i < to ? expert_of<kIdx64>(a, i) : -1;
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (e[u] >= 0) atomicAdd((i0 + u * kThreadsOf < split ? low : high) + e[u], 1);
  }
}

// A block's own slots s0 .. s0 + own: each warp ranks a run of them, 32 at a time, behind the warps before it,
// so that the order is that of the slots whatever the timing.
template <bool kIdx64, int kW>
struct Ranks {
  static constexpr int kThreadsOf = kW * 32, kEach = (kMaxSortExperts + kThreadsOf - 1) / kThreadsOf;
  int w0, w1;        // the warp's run
  int e;             // the expert of its first 32 slots, and the lanes of the same one
  unsigned same;

  // Asks for the first 32.
  __device__ __forceinline__ void begin(const Args& a, int64_t s0, int own) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, run = (own + kThreadsOf - 1) / kThreadsOf * 32;
    w0 = warp * run;
    w1 = min(w0 + run, own);
    e = w0 + lane < w1 ? expert_of<kIdx64>(a, s0 + w0 + lane) : -1;
  }

  // table [kW][E], zeros: the warps' own counts, each by its warp.
  __device__ __forceinline__ void count_own(const Args& a, int64_t s0, int* table) {
    const int lane = threadIdx.x & 31;
    int* mine = table + (threadIdx.x >> 5) * a.E;
    same = 0;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int x = i0 == w0 ? e : i0 + lane < w1 ? expert_of<kIdx64>(a, s0 + i0 + lane) : -1;
      const unsigned m = __match_any_sync(kAll, x);
      if (x >= 0 && lane == __ffs(m) - 1) mine[x] += __popc(m);
      if (i0 == w0) same = m;
      __syncwarp();
    }
  }

  // put(i, p) for each of the slots.  `before` and `rest` [E] hold each expert's slots before s0 and from there on;
  // all(e, n) is called with each expert's number.  Returns the number of all rows.  Syncs the block first.
  template <typename Put, typename All>
  __device__ __forceinline__ int rank(const Args& a, int64_t s0, const int* before, const int* rest, int* table, Put put, All all) {
    __shared__ int warp_sum[kW];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, E = a.E;
    __syncthreads();
    const int each = (E + kThreadsOf - 1) / kThreadsOf;
    int v[kEach], sum = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int x = threadIdx.x * each + i;
      v[i] = i < each && x < E ? before[x] + rest[x] : 0;
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
    for (int w = 0; w < kW; ++w) {
      const int n = warp_sum[w];
      at += w < warp ? n : 0;
      kept += n;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int x = threadIdx.x * each + i;
      if (i < each && x < E) {
        all(x, v[i]);
        int n[kW], next = at + before[x];
#pragma unroll
        for (int w = 0; w < kW; ++w) n[w] = table[w * E + x];
#pragma unroll
        for (int w = 0; w < kW; ++w) {
          table[w * E + x] = next;
          next += n[w];
        }
        at += v[i];
      }
    }
    __syncthreads();
    int* mine = table + warp * E;
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      int x = e;
      unsigned m = same;
      if (i0 > w0) {
        x = i < w1 ? expert_of<kIdx64>(a, s0 + i) : -1;
        m = __match_any_sync(kAll, x);
      }
      int p = -1;
      if (x >= 0) p = mine[x] + __popc(m & ((1u << lane) - 1));
      __syncwarp();
      if (x >= 0 && lane == __ffs(m) - 1) mine[x] += __popc(m);
      __syncwarp();
      if (i < w1) put(i, p);
    }
    return kept;
  }
};

// What a sort writes of slot s, whose row is p.
__device__ __forceinline__ void write_slot(const Args& a, int64_t s, int p, const float* gate) {
  a.slot_pos[s] = p;
  if (p < 0) return;
  if (a.row_slot) a.row_slot[p] = (int)s;
  if (a.gates && p < a.R) a.row_gates[p] = *gate;
}

// Many slots: blocks of them, one a CTA, are counted in one launch and ranked in a second one, whose CTAs each
// add up the counts of the blocks before theirs.  Latency bounds both: 131072 slots of 64 experts 7.2 us, a million 19.
constexpr int kSortWarps = 16, kSortThreads = kSortWarps * 32;

// Slots of a block: one for each thread, more where kCountBlocks blocks do not do.
int64_t count_slots(int64_t N) {
  const int64_t n = (N + kCountBlocks * 32 - 1) / (kCountBlocks * 32) * 32;
  return n < kSortThreads ? kSortThreads : n;
}

template <bool kIdx64>
__global__ void __launch_bounds__(kSortThreads) count_kernel(Args a, int64_t per_block, int32_t* counted) {
  extern __shared__ int shared[];
  const int pitch = count_pitch(a.E);
  for (int e = threadIdx.x; e < pitch; e += kSortThreads) shared[e] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  const int64_t from = blockIdx.x * per_block, to = min(from + per_block, a.T * a.k);
  count<kIdx64, kSortThreads>(a, from, to, to, shared, nullptr);
  __syncthreads();
  for (int e = threadIdx.x; e < pitch; e += kSortThreads) counted[(int64_t)blockIdx.x * pitch + e] = shared[e];
}

// Starts while count_kernel runs, which has waited for what was before it: the choice is there, only the counts
// are not.
template <bool kIdx64>
__global__ void __launch_bounds__(kSortThreads) sort_kernel(Args a, int64_t per_block, const int32_t* counted) {
  extern __shared__ int shared[];
  const int E = a.E, pitch = count_pitch(E), quads = pitch / 4;
  int *before = shared, *rest = before + pitch, *table = rest + pitch;
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < 2 * pitch + kSortWarps * E; i += kSortThreads) shared[i] = 0;
  __syncthreads();
  const int64_t N = a.T * a.k, s0 = blockIdx.x * per_block;
  const int own = (int)min(per_block, N - s0);
  Ranks<kIdx64, kSortWarps> ranks;
  ranks.begin(a, s0, own);
  ranks.count_own(a, s0, table);
  pdl_wait();
  const int groups = quads < kSortThreads ? kSortThreads / quads : 1;
  for (int i = threadIdx.x; i < groups * quads; i += kSortThreads) {
    const int q = i % quads;
    constexpr int kU = 10;  // loads under way: one after the other they cost 0.5 us each (16 us, not 7, for 256 experts)
    int all[4] = {0, 0, 0, 0}, less[4] = {0, 0, 0, 0};
    for (int b0 = i / quads; b0 < (int)gridDim.x; b0 += kU * groups) {
      int4 c[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int b = b0 + u * groups;
        c[u] = b < (int)gridDim.x ? *reinterpret_cast<const int4*>(counted + (int64_t)b * pitch + 4 * q) : make_int4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int v[4] = {c[u].x, c[u].y, c[u].z, c[u].w};
        const bool ahead = b0 + u * groups < (int)blockIdx.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          all[j] += v[j];
          less[j] += ahead ? v[j] : 0;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (less[j]) atomicAdd(&before[4 * q + j], less[j]);
      if (all[j] != less[j]) atomicAdd(&rest[4 * q + j], all[j] - less[j]);
    }
  }
  const int kept = ranks.rank(
      a, s0, before, rest, table, [&](int i, int p) { write_slot(a, s0 + i, p, a.gates + s0 + i); },
      [&](int e, int n) {
        if (blockIdx.x == 0) a.counts[e] = n;
      });
  if (a.row_slot)
    for (int64_t p = max(s0, (int64_t)kept) + threadIdx.x; p < s0 + own; p += kSortThreads) a.row_slot[p] = -1;
}

// The rows' way: bound by HBM (32768 rows of 4096 bf16 to four experts each, sorted: 203 us, 98 % of the copy
// bandwidth; the sort is 6 us of it; small CTAs of a segment a warp, 27 tokens a CTA 230 us).  Each CTA takes `tokens`
// tokens (grid.y: a share of their columns).  With kSort, for few slots, it first sorts them: each CTA counts all of
// them by itself, out of L2, and ranks its own; a warp compares the fewest with one another.  The sort's outputs
// are written behind the rows.  `lanes` lanes move up to 4 * lanes vectors of a token at a time: they read them once and
// write them to each of the token's rows.  The first ones are on their way while the positions are found; `early`: even
// while the previous kernel, a sort of the same call that has waited for what was before it, ends.
// kSize 0: all rows begin and end on boundaries of V.  Else they are values of kSize bytes, and each row is written
// in whole 16-byte vectors of its own alignment, which are read from wherever they lie in x.
template <typename V, int kSize, bool kSort, bool kIdx64, int kLanes>
__global__ void __launch_bounds__(kThreads) rows_kernel(Args a, int tokens, int64_t vecs_y, bool early, int given_lanes) {
  const int lanes = kLanes ? kLanes : given_lanes;
  extern __shared__ int shared[];
  int* pos = shared;  // [tokens * k]
  const int lane = threadIdx.x % lanes, warp = threadIdx.x >> 5, of_warp = 32 / lanes, mine = (threadIdx.x & 31) / lanes;
  const int64_t t0 = (int64_t)blockIdx.x * tokens, s0 = t0 * a.k;
  const int nt = (int)min((int64_t)tokens, a.T - t0), own = nt * a.k;
  const bool first = blockIdx.y == 0;  // writes what does not depend on the columns

  constexpr int kU = kVecs / 32;
  const int64_t vecs = a.row_bytes / (int64_t)sizeof(V), v_first = blockIdx.y * vecs_y, v_end = min(v_first + vecs_y, vecs);
  const int segs = v_end == 0 && a.row_bytes > 0 ? 1 : (int)((v_end - v_first + lanes * kU - 1) / (lanes * kU)), units = (nt + of_warp - 1) / of_warp * segs;
  int t, unit = warp;
  int64_t v0;
  V buf[kU];
  const auto place = [&] {
    t = unit / segs;
    v0 = v_first + (int64_t)(unit - t * segs) * lanes * kU + lane;
    t = t * of_warp + mine;
  };
  const auto fetch = [&] {
    place();
    if (kSize != 0 || t >= nt) return;
    const V* src = reinterpret_cast<const V*>(a.x + (t0 + t) * a.ld_bytes);
#pragma unroll
    for (int u = 0; u < kU; ++u)
      if (v0 + u * lanes < v_end) buf[u] = __ldcg(src + v0 + u * lanes);
  };

  int kept = 0;
  float gate = 0.f;
  if constexpr (!kSort) {
    if (early && unit < units) fetch();
    pdl_wait();
    pdl_launch_dependents();
    if (!early && unit < units) fetch();
    for (int i = threadIdx.x; i < own; i += kThreads) {
      const int p = a.slot_pos[s0 + i];
      pos[i] = p;
      if (first && a.gates && p >= 0 && p < a.R) a.row_gates[p] = a.gates[s0 + i];
    }
  } else {
    int *before = shared + tokens * a.k, *rest = before + a.E, *table = rest + a.E;
    pdl_wait();
    pdl_launch_dependents();
    Ranks<kIdx64, kWarps> ranks;
    const int N = (int)(a.T * a.k);
    const bool counts = first && blockIdx.x == 0;
    if (N <= kWarpSlots) {  // a slot a lane: no shared memory but for the positions
      const int at = threadIdx.x & 31, e = at < N ? expert_of<kIdx64>(a, at) : -1;
      if (unit < units) fetch();
      kept = __popc(__ballot_sync(kAll, e >= 0));
      if (warp == 0) {
        int p = 0;
        for (int j = 0; j < N; ++j) {
          const int f = __shfl_sync(kAll, e, j);
          p += f >= 0 && (f < e || (f == e && j < at)) ? 1 : 0;
        }
        if (at >= s0 && at < s0 + own) pos[at - s0] = e >= 0 ? p : -1;
      } else if (counts) {
        for (int x0 = (warp - 1) * 32; x0 < a.E; x0 += (kWarps - 1) * 32) {
          int n = 0;
          for (int j = 0; j < N; ++j) n += __shfl_sync(kAll, e, j) == x0 + at ? 1 : 0;
          if (x0 + at < a.E) a.counts[x0 + at] = n;
        }
      }
    } else {
      ranks.begin(a, s0, own);
      for (int i = threadIdx.x; i < (2 + kWarps) * a.E; i += kThreads) before[i] = 0;
      __syncthreads();
      count<kIdx64, kThreads>(a, 0, N, s0, before, rest);
      if (unit < units) fetch();
      ranks.count_own(a, s0, table);
      kept = ranks.rank(
          a, s0, before, rest, table, [&](int i, int p) { pos[i] = p; },
          [&](int e, int n) {
            if (counts) a.counts[e] = n;
          });
    }
    if (first && a.gates && threadIdx.x < own) gate = a.gates[s0 + threadIdx.x];
  }
  __syncthreads();
  const char* x_end = a.x + (a.T - 1) * a.ld_bytes + a.row_bytes;
  while (unit < units) {
    for (int j = 0; t < nt && j < a.k; ++j) {
      const int p = pos[t * a.k + j];
      if (p < 0 || p >= a.R) continue;
      char* row = a.x_rows + p * a.row_bytes;
      if constexpr (kSize == 0) {
        V* dst = reinterpret_cast<V*>(row);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (v0 + u * lanes < v_end) __stcs(dst + v0 + u * lanes, buf[u]);
      } else {
        const char* src = a.x + (t0 + t) * a.ld_bytes;
        const int head = (int)min(a.row_bytes, (int64_t)(-reinterpret_cast<uintptr_t>(row) & 15));  // bytes to its first boundary
        const int64_t whole = (a.row_bytes - head) / 16, v_last = min(v_end, whole);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (v0 + u * lanes < v_last) buf[u] = load_any(src + head + 16 * (v0 + u * lanes), a.x, x_end);
        if (v0 == lane) {  // and what lies before and behind the whole vectors, a value a lane
          using Value = typename std::conditional<kSize == 2, uint16_t, uint8_t>::type;
          const int64_t gap = 16 * whole;
          for (int64_t i = lane * kSize; i < a.row_bytes - gap; i += lanes * kSize) {
            const int64_t b = i < head ? i : i + gap;
            *reinterpret_cast<Value*>(row + b) = *reinterpret_cast<const Value*>(src + b);
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u)
          if (v0 + u * lanes < v_last) __stcs(reinterpret_cast<uint4*>(row + head + 16 * (v0 + u * lanes)), buf[u]);
      }
    }
    unit += kWarps;
    if (unit < units) fetch();
  }
  if (kSort && first)
    for (int i = threadIdx.x; i < own; i += kThreads) {
      write_slot(a, s0 + i, pos[i], i == threadIdx.x ? &gate : a.gates + s0 + i);
      if (a.row_slot && s0 + i >= kept) a.row_slot[s0 + i] = -1;
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

template <typename V, int kSize, bool kSort, bool kIdx64>
cudaError_t launch_as(const Args& a, bool early, cudaStream_t st) {
  const int64_t vecs = a.row_bytes / (int64_t)sizeof(V);
  const int lanes = lanes_for(vecs);
  const int64_t most_vecs = lanes * (kVecs / 32), segs = vecs == 0 && a.row_bytes > 0 ? 1 : (vecs + most_vecs - 1) / most_vecs;
  // Tokens a CTA: a segment for each group of lanes; where each CTA counts all slots, no more CTAs than kSortCtas.
  int64_t tokens = segs ? (kThreads / lanes + segs - 1) / segs : (kThreads + a.k - 1) / a.k;
  if (kSort && tokens < (a.T + kSortCtas - 1) / kSortCtas) tokens = (a.T + kSortCtas - 1) / kSortCtas;
  if (tokens > kMaxPositions / a.k) tokens = kMaxPositions / a.k;
  if (tokens > a.T) tokens = a.T;
  const int64_t gx = (a.T + tokens - 1) / tokens;
  // columns of a few tokens' long rows are shared out
  int64_t gy = 1, vecs_y = vecs;
  if (segs > 1 && gx < kSortCtas) {
    gy = (tokens * segs + kWarps - 1) / kWarps;
    if (gy > kSortCtas / gx) gy = kSortCtas / gx;
    if (gy > segs) gy = segs;
    vecs_y = (segs + gy - 1) / gy * kVecs;
    gy = (vecs + vecs_y - 1) / vecs_y;
  }
  const size_t smem = ((size_t)tokens * a.k + (kSort ? (size_t)(2 + kWarps) * a.E : 0)) * sizeof(int);
  const auto kernel = lanes == 32 ? rows_kernel<V, kSize, kSort, kIdx64, 32> : rows_kernel<V, kSize, kSort, kIdx64, 0>;
  if (smem > 48 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(kernel, dim3((unsigned)gx, (unsigned)gy), dim3(kThreads), smem, st, true, 1, a, (int)tokens,
                       vecs_y, early, lanes);
}

template <typename V, int kSize>
cudaError_t launch_vec(const Args& a, bool sort, cudaStream_t st) {
  if (!sort) return launch_as<V, kSize, false, false>(a, a.idx != nullptr, st);
  return a.idx64 ? launch_as<V, kSize, true, true>(a, false, st) : launch_as<V, kSize, true, false>(a, false, st);
}

template <bool kIdx64>
cudaError_t launch_sort(const Args& a, int32_t* counted, cudaStream_t st) {
  const int64_t N = a.T * a.k, per_block = count_slots(N);
  const dim3 grid((unsigned)((N + per_block - 1) / per_block)), block(kSortThreads);
  const size_t pitch = (size_t)count_pitch(a.E) * sizeof(int);
  cudaError_t e = launch_kernel(count_kernel<kIdx64>, grid, block, pitch, st, true, 1, a, per_block, counted);
  if (e != cudaSuccess) return e;
  const size_t smem = 2 * pitch + (size_t)kSortWarps * a.E * sizeof(int);
  if (smem > 48 * 1024) {
    e = cudaFuncSetAttribute(sort_kernel<kIdx64>, cudaFuncAttributeMaxDynamicSharedMemorySize, (2 + kSortWarps) * kMaxSortExperts * sizeof(int));
    if (e != cudaSuccess) return e;
  }
  return launch_kernel(sort_kernel<kIdx64>, grid, block, smem, st, true, 1, a, per_block, (const int32_t*)counted);
}

// ------------------------------------------------------------------ combine

// n values of type T, 16 bytes at most at a time, to and from fp32.
template <typename T, int n>
struct Values {
  static constexpr int kBytes = n * (int)sizeof(T) < 16 ? n * (int)sizeof(T) : 16, kParts = n * (int)sizeof(T) / kBytes;
  using Part = typename std::conditional<kBytes == 16, uint4,
               typename std::conditional<kBytes == 8, uint2, typename std::conditional<kBytes == 4, uint32_t, uint16_t>::type>::type>::type;
  Part part[kParts];
  __device__ __forceinline__ void load(const T* p) {  // on a boundary of kBytes
#pragma unroll
    for (int i = 0; i < kParts; ++i) part[i] = __ldcs(reinterpret_cast<const Part*>(p) + i);
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) __stcs(reinterpret_cast<Part*>(p) + i, part[i]);
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

// Bound by HBM: 32768 tokens' four rows of 4096 bf16 and the stream back into it in 251 us, 95 % of the copy bandwidth (with
// six CTAs an SM, for which 16 to 56 bytes spill; four 302, eight, for which more do, 356).  Of the others, one slot a token
// spills 64 bytes, 128 from bf16 to fp32, and single values to bf16 28.
// `lanes` lanes for lanes * V * C columns of one token, C pieces of V a lane: kJ rows in flight at a time, summed in the
// slots' order.  What counts is the bytes of rows that a lane has under way: for one slot a token, four pieces of its row,
// not one of up to four rows (16384 x 2048 bf16: 36.8 -> 23.4 us); where rows lie on 4-byte boundaries, four or eight
// pieces of four rows (4 slots of 2044 bf16: 124 -> 79 us, 1023 fp32 108 -> 65, 2047 bf16 206 -> 121).
template <typename Ty, typename To, int V, int C, int kJ, int kLanes>
__global__ void __launch_bounds__(kThreads, C == 1 && kLanes ? 6 : 4) combine_kernel(const Ty* y, int64_t R, const int32_t* slot_pos,
                                                                                    const float* gates, int64_t T, int k, int64_t d,
                                                                                    unsigned segs, int given_lanes, const To* residual,
                                                                                    To* out) {
  const int lanes = kLanes ? kLanes : given_lanes;
  const int lane = threadIdx.x % lanes;
  const int64_t unit = ((int64_t)blockIdx.x * kThreads + threadIdx.x) / lanes;
  const int64_t t = unit <= 0xffffffffll ? (int64_t)((unsigned)unit / segs) : unit / segs;
  pdl_wait();
  pdl_launch_dependents();
  const bool has = t < T;
  const int64_t piece = (unit - t * segs) * lanes * C + lane;
  const auto col = [&](int x) { return (piece + x * lanes) * V; };
  Values<To, V> res[C];
  if (residual && has) {
#pragma unroll
    for (int x = 0; x < C; ++x)
      if (col(x) < d) res[x].load(residual + t * d + col(x));
  }
  float acc[C][V];
#pragma unroll
  for (int x = 0; x < C; ++x)
#pragma unroll
    for (int i = 0; i < V; ++i) acc[x][i] = 0.f;
  for (int j0 = 0; j0 < k; j0 += lanes) {
    const int n = min(lanes, k - j0);
    int p = -1;
    float g = 1.f;
    if (has && lane < n) {
      p = slot_pos[t * k + j0 + lane];
      if (gates) g = gates[t * k + j0 + lane];
    }
    if (p >= R) p = -1;
    for (int j = 0; j < n; j += kJ) {
      Values<Ty, V> row[kJ][C];
      int at[kJ];
#pragma unroll
      for (int q = 0; q < kJ; ++q) {
        at[q] = __shfl_sync(kAll, p, j + q, lanes);  // lanes past n hold -1
        if (at[q] < 0) continue;
#pragma unroll
        for (int x = 0; x < C; ++x)
          if (col(x) < d) row[q][x].load(y + at[q] * d + col(x));
      }
#pragma unroll
      for (int q = 0; q < kJ; ++q) {
        const float gq = __shfl_sync(kAll, g, j + q, lanes);
        if (at[q] < 0) continue;
#pragma unroll
        for (int x = 0; x < C; ++x)
#pragma unroll
          for (int i = 0; i < V; ++i) acc[x][i] = fmaf(gq, row[q][x].get(i), acc[x][i]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < C; ++x) {
    if (!has || col(x) >= d) continue;
    Values<To, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.set(i, residual ? res[x].get(i) + acc[x][i] : acc[x][i]);
    o.store(out + t * d + col(x));
  }
}

template <typename Ty, typename To, int V, int C, int kJ, int kLanes>
cudaError_t combine_as(const void* y, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T, int k, int64_t d,
                       const void* residual, void* out, cudaStream_t st) {
  const int64_t pieces = d / V;
  const int lanes = kLanes ? kLanes : lanes_for((pieces + C - 1) / C);
  const int64_t segs = (pieces + lanes * C - 1) / (lanes * C), of_block = kThreads / lanes, blocks = (T * segs + of_block - 1) / of_block;
  return launch_kernel(combine_kernel<Ty, To, V, C, kJ, kLanes>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, 1,
                       static_cast<const Ty*>(y), R, slot_pos, gates, T, k, d, (unsigned)segs, lanes, static_cast<const To*>(residual),
                       static_cast<To*>(out));
}

// The gradients, bound by HBM: 8192 tokens' eight rows of 2048 bf16 in 90.5 us, 99 % of the copy bandwidth.  `per` warps a token, or `lanes` lanes of one; each lane C pieces of V columns at a time of up to kJ rows;
// the products with dout are summed over the lanes, and over the warps in order.
template <typename Td, typename Ty, int V, int C, int kJ, int kLanes>
__global__ void __launch_bounds__(kThreads) combine_backward_kernel(const Td* dout, const int32_t* slot_pos, const float* gates,
                                                                    int64_t T, int k, int64_t d, int64_t R, const Ty* y, Ty* dy,
                                                                    float* dgates, int per, int given_lanes) {
  __shared__ float part[kWarps][kJ];
  const int lanes = kLanes ? kLanes : given_lanes;
  const int lane = threadIdx.x % lanes, warp = threadIdx.x >> 5, mine = warp % per;
  const int64_t t = ((int64_t)blockIdx.x * (kWarps / per) + warp / per) * (32 / lanes) + (threadIdx.x & 31) / lanes;
  pdl_wait();
  pdl_launch_dependents();
  const bool has = t < T;
  for (int j0 = 0; j0 < k; j0 += kJ) {
    const int n = min(kJ, k - j0);
    int p = -1;
    float g = 1.f;
    if (has && lane < n) {
      p = slot_pos[t * k + j0 + lane];
      if (gates) g = gates[t * k + j0 + lane];
    }
    if (p >= R) p = -1;
    int at[kJ];
    float gate[kJ], dot[kJ];
#pragma unroll
    for (int q = 0; q < kJ; ++q) {
      at[q] = __shfl_sync(kAll, p, q, lanes);
      gate[q] = __shfl_sync(kAll, g, q, lanes);
      dot[q] = 0.f;
    }
    if (has) {
      for (int64_t c = (mine * lanes * C + lane) * V; c < d; c += per * lanes * V * C) {
        const auto col = [&](int x) { return c + x * lanes * V; };
        Values<Td, V> go[C];
#pragma unroll
        for (int x = 0; x < C; ++x)
          if (col(x) < d) go[x].load(dout + t * d + col(x));
        Values<Ty, V> row[kJ][C];
        if (dgates) {
#pragma unroll
          for (int q = 0; q < kJ; ++q)
#pragma unroll
            for (int x = 0; x < C; ++x)
              if (at[q] >= 0 && col(x) < d) row[q][x].load(y + at[q] * d + col(x));
        }
#pragma unroll
        for (int q = 0; q < kJ; ++q) {
          if (at[q] < 0) continue;
#pragma unroll
          for (int x = 0; x < C; ++x) {
            if (col(x) >= d) continue;
            if (dgates) {
#pragma unroll
              for (int i = 0; i < V; ++i) dot[q] = fmaf(go[x].get(i), row[q][x].get(i), dot[q]);
            }
            if (dy) {
              Values<Ty, V> o;
#pragma unroll
              for (int i = 0; i < V; ++i) o.set(i, gate[q] * go[x].get(i));
              o.store(dy + at[q] * d + col(x));
            }
          }
        }
      }
    }
    if (dgates) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < kJ; ++q) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          if (o < lanes) dot[q] += __shfl_xor_sync(kAll, dot[q], o);
        if (lane == q) sum = dot[q];
      }
      if (per > 1) {
        if (lane < kJ) part[warp][lane] = sum;
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

template <typename Td, typename Ty, int V, int C, int kJ, int kLanes>
cudaError_t backward_as(const void* dout, const int32_t* slot_pos, const float* gates, int64_t T, int k, int64_t d, int64_t R,
                        const void* y, void* dy, float* dgates, cudaStream_t st) {
  const int lanes = kLanes ? kLanes : lanes_for((d / V + C - 1) / C);
  // warps a token: each has its columns in kTurns turns at most (8192 x 8 x 2048: 94 us with 8 turns, 90.6 with 4, 89.3 with
  // 2; 32768 x 4 x 4096: 352, 350, 358), in one turn while there are few tokens
  constexpr int kTurns = 4;
  int per = 1;
  while (lanes == 32 && per < kWarps && (int64_t)per * 32 * V * C * (T * per < 152 * 16 ? 1 : kTurns) < d) per *= 2;
  const int64_t of_block = kThreads / (per * lanes), blocks = (T + of_block - 1) / of_block;
  return launch_kernel(combine_backward_kernel<Td, Ty, V, C, kJ, kLanes>, dim3((unsigned)blocks), dim3(kThreads), 0, st, true, 1,
                       static_cast<const Td*>(dout), slot_pos, gates, T, k, d, R, static_cast<const Ty*>(y), static_cast<Ty*>(dy),
                       dgates, per, lanes);
}

// How many values a lane takes at once: `most`, 2 or 1, so many that they divide a row and that all these arrays (address,
// bytes a value) are on boundaries of them, 16 bytes doing for more than 16.
int values_at_once(int most, int64_t d, std::initializer_list<std::pair<const void*, int>> arrays) {
  for (const int v : {most, 2}) {
    bool fits = d % v == 0;
    for (const auto& [p, size] : arrays) fits = fits && reinterpret_cast<uintptr_t>(p) % (v * size < 16 ? v * size : 16) == 0;
    if (fits) return v;
  }
  return 1;
}

}  // namespace

bool counts_first(int64_t N) { return N > kSortFew; }  // see there

cudaError_t launch_rows(const Args& args, int32_t* counted, cudaStream_t st) {
  Args a = args;
  bool sort = a.idx != nullptr;
  if (sort && counted) {
    const cudaError_t e = a.idx64 ? launch_sort<true>(a, counted, st) : launch_sort<false>(a, counted, st);
    if (e != cudaSuccess || a.row_bytes == 0) return e;
    a.gates = nullptr;  // they are on their rows
    sort = false;
  }
  const uintptr_t b = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.x_rows) | (uintptr_t)a.row_bytes | (uintptr_t)a.ld_bytes;
  if (b % 16 == 0) return launch_vec<uint4, 0>(a, sort, st);
  if (b % 8 == 0) return launch_vec<uint2, 0>(a, sort, st);
  if (b % 4 == 0) return launch_vec<uint32_t, 0>(a, sort, st);
  if (b % 2 == 0) return launch_vec<uint4, 2>(a, sort, st);
  return launch_vec<uint4, 1>(a, sort, st);
}

using bf16 = __nv_bfloat16;

cudaError_t launch_combine(const void* y, bool y_bf16, int64_t R, const int32_t* slot_pos, const float* gates, int64_t T, int k,
                           int64_t d, const void* residual, void* out, bool out_bf16, cudaStream_t st) {
  const int v = values_at_once(y_bf16 ? 8 : 4, d, {{y, y_bf16 ? 2 : 4}, {residual, out_bf16 ? 2 : 4}, {out, out_bf16 ? 2 : 4}});
  const auto with = [&](auto ty, auto to) {
    using Ty = decltype(ty);
    using To = decltype(to);
    constexpr int kV = 16 / sizeof(Ty);
    const bool wide = lanes_for(d / v) == 32;
    const auto as = [&](auto f) { return f(y, R, slot_pos, gates, T, k, d, residual, out, st); };
    if (v == kV)
      return !wide    ? as(combine_as<Ty, To, kV, 1, 4, 0>)
             : k == 1 ? as(combine_as<Ty, To, kV, 4, 1, 32>)
             : k == 2 ? as(combine_as<Ty, To, kV, 2, 2, 32>)
                      : as(combine_as<Ty, To, kV, 1, 4, 32>);
    if (v == 2) return wide ? as(combine_as<Ty, To, 2, 4, 4, 32>) : as(combine_as<Ty, To, 2, 1, 4, 0>);
    return wide ? as(combine_as<Ty, To, 1, 8, 4, 32>) : as(combine_as<Ty, To, 1, 1, 4, 0>);
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
    constexpr int kV = 16 / sizeof(Ty);
    const bool wide = lanes_for(d / v) == 32;
    const auto as = [&](auto f) { return f(dout, slot_pos, gates, T, k, d, R, y, dy, dgates, st); };
    if (v == kV)
      return !wide    ? as(backward_as<Td, Ty, kV, 1, 4, 0>)
             : k == 1 ? as(backward_as<Td, Ty, kV, 4, 1, 32>)
             : k == 2 ? as(backward_as<Td, Ty, kV, 2, 2, 32>)
             : k <= 4 ? as(backward_as<Td, Ty, kV, 1, 4, 32>)
                      : as(backward_as<Td, Ty, kV, 1, 8, 32>);
    if (v == 2) return !wide ? as(backward_as<Td, Ty, 2, 1, 4, 0>) : k <= 4 ? as(backward_as<Td, Ty, 2, 4, 4, 32>) : as(backward_as<Td, Ty, 2, 4, 8, 32>);
    return !wide ? as(backward_as<Td, Ty, 1, 1, 4, 0>) : k <= 4 ? as(backward_as<Td, Ty, 1, 4, 4, 32>) : as(backward_as<Td, Ty, 1, 4, 8, 32>);
  };
  if (dout_bf16) return y_bf16 ? with(bf16(), bf16()) : with(bf16(), float());
  return y_bf16 ? with(float(), bf16()) : with(float(), float());
}

}  // namespace rows
}  // namespace moe
