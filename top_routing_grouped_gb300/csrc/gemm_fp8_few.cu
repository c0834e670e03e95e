// gemm_fp8_few.cu -- the 8-bit grouped products where an expert has few rows (decoding, short
// batches): the same results as gemm_fp8_tc.cu, bound by reading the weights once.
//
//   out[p, n] = gate(p) * (A[p] . W_e[n])   and   h[p, n] = SiLU(A[p] . W1_e[n]) * (A[p] . W3_e[n])
//
// With a handful of rows a 256-row tile is padding, and an MMA of 256 rows takes as long for one of
// them as for all.  Here the weights are the MMA's 128 rows and the activations its N columns
// (16 to 96), so D[m][t] is output column m of row t; an MMA takes 39-56 clocks, a stage of
// 16 KB (SwiGLU: 32 KB) of weights a third of the time that HBM takes to deliver it.
//
// A unit of work is (segment, block of 128 weight rows, up to 96 of the segment's rows).  Every CTA
// finds its units from the segment counts itself (a scan over at most 256 numbers), so a call needs no
// kernel for tile tables.  When there are fewer units than SMs, a cluster of up to 8 CTAs shares a
// unit: each sums a part of K, and the unit's rows are dealt out to the CTAs, eight at a time; for its
// rows a CTA adds the others' sums, which arrive in its shared memory, in rank order.  (With all rows
// summed by the first CTA 96 x 8192 x 2048 took 13.4 us, not 9.7.)
//
// What bounds it: HBM while the weights stream (1500 rows over 128 experts of 2048 x 1024: 129 us,
// 6.1 TB/s of weights, rows and results); with one unit for each SM the fixed part counts, about 5 us of
// a launch (one token of 64 experts of 4096 x 2048: 25.1 us for 101 MB; 13 x 2064 x 8208: 7.4 us for
// 17 MB).  The CTA pairs take 141, 34 and 9.8 us for the three.  In the token's call HBM stands still for some
// 3.5 us between the two products (epilogue, launch, set-up); fetching the second one's first weights
// to L2 meanwhile gained nothing (24 MB: 25.4 -> 26.2 us, 12 MB: 25.2), nor did two CTAs an SM.
//
// Roles of a CTA: three TMA warps (ring of stages), an MMA warp (one elected lane issues), eight
// epilogue warps and four warps that store the block factors to TMEM, as in gemm_fp8_tc.cu.  Waits are
// bounded (MOE_ERR_TIMEOUT, no trap).
#include <cuda.h>
#include <cuda_bf16.h>
#include <stddef.h>

#include <atomic>

#include "device_common.cuh"
#include "fp8_common.cuh"
#include "fp8_mma.cuh"
#include "fp8_units.cuh"
#include "gemm_tc.h"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace moe {
namespace fp8 {
namespace {

constexpr int kBK = 128;              // k's (bytes) per stage: one block of factors
constexpr int kWRows = 128;           // weight rows per unit
constexpr int kMaxTok = 96;           // activation rows per unit: two buffers of two matrices, and factors, fill TMEM
constexpr int kTokBox = 16;           // rows of one TMA box of activations
constexpr int kWBytes = kWRows * kBK;
constexpr int kMaxStages = 12;
constexpr int kThreads = 512;
constexpr int kEpiWarp0 = 4, kEpiWarps = 8;  // two sets of four warps take turns with the rows, eight at a time
constexpr int kSfWarp0 = 12;

// TMEM columns: accumulator (buffer b, matrix m) at 192 b + 96 m; factor set i at 384 + 16 i
// (4 of W1 or W, 4 of W3, 4 of the activations)
constexpr int kTmemCols = 512;
constexpr int kSfCol = 4 * kMaxTok;
constexpr int kSfStep = 16;
constexpr int kSfSets = 8;

struct Ctl {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t tfull[2], tempty[2];
  uint64_t sf_full[kSfSets], sf_empty[kSfSets];
  uint64_t rfull;  // the others' sums for this CTA's rows have arrived
  uint64_t rfree;  // the others have read this CTA's sums of the unit before
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  uint32_t top[2][2][4][8];      // epilogue: [set][turn] largest hidden value of each warp and row
  Segments seg;
};

// The launch's sizes, chosen on the host.
struct FewShape {
  int n_seg;       // segments; segment s holds rows of expert s % E
  int tok;         // rows per unit: a multiple of 16, at most kMaxTok
  int stages;
  int stage_bytes;
  int split;       // CTAs of a cluster that share a unit
  int part;        // rows of a unit that fall to one of them at most, a multiple of 8
  int recv_bytes;  // shared memory for one other CTA's sums: [matrix][part][128 weight rows]
  int first;       // this launch starts the call: it sets the status word
};

__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity, int64_t timeout_ns, const volatile int* abort) {
  const uint64_t t0 = global_ns();
  for (uint32_t i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63u) == 0u && (*abort || (int64_t)(global_ns() - t0) > timeout_ns)) return false;
  }
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Barrier of the 128 threads of an epilogue set, with the AND of a flag over them.
__device__ __forceinline__ bool epi_bar_and(int set, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(1 + set), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&v)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
               : "r"(taddr)
               : "memory");
}

struct Unit {
  int e;       // weight expert
  int n0;      // first weight row of the block
  int row0;    // first activation row
  int rows;    // activation rows, 1..tok
};

// Unit u: segments in order, in a segment the blocks of weight rows, in a block the groups of rows
// (neighbouring CTAs then read the same weights, once from HBM).
__device__ __forceinline__ Unit decode(const Ctl* ctl, const FewShape& f, int E, int u) {
  const int sg = segment_of(&ctl->seg, f.n_seg, u);
  const int cnt = ctl->seg.row0[sg + 1] - ctl->seg.row0[sg], groups = (cnt + f.tok - 1) / f.tok, local = u - ctl->seg.unit0[sg];
  Unit r;
  r.e = sg % E;
  r.n0 = local / groups * kWRows;
  const int g0 = local % groups * f.tok;
  r.row0 = ctl->seg.row0[sg] + g0;
  r.rows = min(f.tok, cnt - g0);
  return r;
}

// kSplit: a unit is shared by a cluster (its code costs the others 0.2 us a launch where it is merely there).
template <int kKind, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_few_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmW3, GemmArgs g, Ws ws, const int32_t* seg_counts, FewShape f,
                        int64_t timeout_ns) {
  constexpr int kMats = kKind == kSwiGLU ? 2 : 1;
  const int split = kSplit ? f.split : 1;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* stages = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* recv = reinterpret_cast<float*>(stages + (size_t)f.stages * f.stage_bytes);
  Ctl* ctl = reinterpret_cast<Ctl*>(reinterpret_cast<uint8_t*>(recv) + (size_t)(split - 1) * f.recv_bytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = kSplit ? ptx::cluster_ctarank() : 0;
  const int cid = (int)blockIdx.x / split, ncl = (int)gridDim.x / split;
  const int nblk = (g.n + kWRows - 1) / kWRows;
  const int kblocks = (g.K + kBK - 1) / kBK;
  const int sck = (int)(scale_cols(g.K) / 4);
  const int gk0 = sck * (int)rank / split, gk1 = sck * ((int)rank + 1) / split;  // this CTA's groups of four K blocks
  const int kb0 = gk0 * 4, kb1 = min(gk1 * 4, kblocks);

  // Warp 8 makes the barriers and warp 12 takes TMEM while warps 0-7 wait for the counts and find the units.
  if (threadIdx.x == 8 * 32) {
    for (int i = 0; i < f.stages; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->tfull[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&ctl->tempty[i]), kEpiWarps);
    }
    for (int i = 0; i < kSfSets; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->sf_full[i]), 4);
      ptx::mbar_init(ptx::smem_u32(&ctl->sf_empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&ctl->rfull), kSplit ? kEpiWarps * (split - 1) : 1);
    ptx::mbar_init(ptx::smem_u32(&ctl->rfree), kSplit ? kEpiWarps * (split - 1) : 1);
    ptx::mbar_init(ptx::smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 9 * 32) {
    ptx::tma_prefetch_desc(&tmX);
    ptx::tma_prefetch_desc(&tmW);
    if (kMats == 2) ptx::tma_prefetch_desc(&tmW3);
  }
  if (kSplit) asm volatile("barrier.cluster.arrive;" ::: "memory");
  if (warp == kSfWarp0) {
    ptx::tmem_alloc(ptx::smem_u32(&ctl->tmem_base), kTmemCols);
    ptx::tmem_relinquish();
    ptx::tc_fence_before();
  }
  // The call's first launch waits here for the counts and the activations.  Another one starts as soon as
  // the launch before it has (as far as SMs are free), and that may be one which has waited for nothing
  // itself: in the layer the dispatch may still run then.  So only what the caller gives (weights and
  // their factors) and what was there before the dispatch started (the counts) is read before a wait;
  // rows, their factors and gates are read after one.
  if (f.first) pdl_wait();
  pdl_launch_dependents();

  int total = scan_segments(&ctl->seg, seg_counts, f.n_seg, g.rows, [&](int cnt) { return (cnt + f.tok - 1) / f.tok * nblk; });
  if (f.first) begin_status(ws, total < 0, 0x950u);
  total = max(total, 0);
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;  // made visible by the scan's barriers, as the barriers are
  if (kSplit) asm volatile("barrier.cluster.wait;" ::: "memory");  // every CTA's barriers exist before another arrives on them
  volatile int* abort_flag = &ctl->abort;

  if (warp == 0 || warp == 2 || warp == 3) {
    // ------------------------------------------------------------ TMA producers
    // Warp 0 loads W (W1), warp 2 W3, warp 3 the activations, each converged with one elected lane
    // issuing: a load costs its warp about 200 clocks, and one lane that issued all of a stage's took
    // as long to fill the ring for the first time as HBM.  In a call's second launch the weights that fill the
    // ring once are requested before the first launch has ended; the wait for it comes before the first
    // wait for an MMA, whose limit would else run while nothing can have happened yet.
    if (!f.first && warp == 3) pdl_wait();
    const CUtensorMap* map = warp == 0 ? &tmW : warp == 2 ? &tmW3 : &tmX;
    const uint32_t ctl0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ctl), 0);
    const uint32_t dst0 = __shfl_sync(0xffffffffu, ptx::smem_u32(stages), 0) + (uint32_t)(warp == 0 ? 0 : warp == 2 ? kWBytes : kMats * kWBytes);
    const bool elected = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = cid; u < total && ok && (kMats == 2 || warp != 2); u += ncl) {
      const Unit un = decode(ctl, f, g.E, u);
      const int boxes = __shfl_sync(0xffffffffu, (un.rows + kTokBox - 1) / kTokBox, 0);
      const uint32_t bytes = (uint32_t)(kMats * kWBytes + boxes * kTokBox * kBK);
      const int y = __shfl_sync(0xffffffffu, warp == 3 ? un.row0 : un.e * g.n + un.n0, 0), n = warp == 3 ? boxes : 1;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(ctl0 + (uint32_t)offsetof(Ctl, empty) + 8 * stage, phase ^ 1u, timeout_ns,
                                                    abort_flag)) != 0;
        if (!ok) break;
        if (elected) {
          const uint32_t bar = ctl0 + (uint32_t)offsetof(Ctl, full) + 8 * stage, dst = dst0 + (uint32_t)(stage * f.stage_bytes);
          if (warp == 0) ptx::mbar_arrive_expect_tx(bar, bytes);
          for (int b = 0; b < n; ++b) ptx::tma_load_2d(dst + b * kTokBox * kBK, map, kb * kBK, y + b * kTokBox, bar);
        }
        __syncwarp();
        if (++stage == f.stages) {
          stage = 0;
          phase ^= 1u;
          if (!f.first) pdl_wait();  // returns at once after the first time
        }
      }
    }
    if (!ok && elected) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x960u + kKind);
      ctl->abort = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (converged warp)
    if (!f.first) pdl_wait();  // its limits run from here
    const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
    const uint64_t desc0 = ptx::desc_kmajor_sw128(__shfl_sync(0xffffffffu, ptx::smem_u32(stages), 0));
    const uint32_t ctl0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ctl), 0);
    const bool elected = elect_one();
    auto wait = [&](uint32_t bar, uint32_t parity) {
      return __all_sync(0xffffffffu, ptx::mbar_wait(ctl0 + bar, parity, timeout_ns, abort_flag)) != 0;
    };
    int stage = 0, acc = 0, set = 0;
    uint32_t phase = 0, acc_phase = 0, sf_phase = 0;
    bool ok = true;
    for (int u = cid; u < total && ok; u += ncl) {
      const int cols = (__shfl_sync(0xffffffffu, decode(ctl, f, g.E, u).rows, 0) + 15) & ~15;
      if (!(ok = wait(offsetof(Ctl, tempty) + 8 * acc, acc_phase ^ 1u))) break;
      ptx::tc_fence_after();
      const uint32_t d = tm + (uint32_t)(acc * 2 * kMaxTok);
      uint32_t sf = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if ((kb & 3) == 0) {
          if (!(ok = wait(offsetof(Ctl, sf_full) + 8 * set, sf_phase))) break;
          sf = tm + (uint32_t)(kSfCol + set * kSfStep);
        }
        if (!(ok = wait(offsetof(Ctl, full) + 8 * stage, phase))) break;
        ptx::tc_fence_after();
        const bool last_of_group = (kb & 3) == 3 || kb + 1 == kb1;
        if (elected) {
          const uint64_t dw = desc0 + (uint64_t)(stage * (f.stage_bytes >> 4)), dx = dw + (kMats * kWBytes >> 4);
          const uint32_t idesc = idesc_mxf8(kWRows, 0, 0) + (uint32_t)(kb & 3) * idesc_byte() + ((uint32_t)(cols >> 3) << 17);
#pragma unroll
          for (int m = 0; m < kMats; ++m)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_mxf8(d + kMaxTok * m, dw + (m * kWBytes >> 4) + 2 * ks, dx + 2 * ks, idesc, sf + 4 * m, sf + 8,
                       (kb != kb0 || ks != 0) ? 1u : 0u);
          ptx::mma_commit(ctl0 + offsetof(Ctl, empty) + 8 * stage);
          if (last_of_group) ptx::mma_commit(ctl0 + offsetof(Ctl, sf_empty) + 8 * set);
          if (kb + 1 == kb1) ptx::mma_commit(ctl0 + offsetof(Ctl, tfull) + 8 * acc);
        }
        __syncwarp();
        if (last_of_group && ++set == kSfSets) {
          set = 0;
          sf_phase ^= 1u;
        }
        if (++stage == f.stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && elected) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x970u + kKind);
      ctl->abort = 1;
    }
    // every MMA has finished before TMEM is released
    if (elected) ptx::mma_commit(ctl0 + offsetof(Ctl, drain));
    __syncwarp();
    ptx::mbar_wait(ctl0 + offsetof(Ctl, drain), 0u, timeout_ns, nullptr);
  } else if (warp >= kSfWarp0) {
    // ------------------------------------------------------------ block factors
    if (!f.first) pdl_wait();  // those of the hidden rows
    const uint32_t* sx32 = reinterpret_cast<const uint32_t*>(g.sa);
    const uint32_t* sw32 = reinterpret_cast<const uint32_t*>(g.sb);
    const uint32_t* sw3_32 = reinterpret_cast<const uint32_t*>(kMats == 2 ? g.sb3 : g.sb);
    const uint32_t dst = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kSfCol;
    int set = 0, u = cid, gk = gk0;
    uint32_t phase = 0;
    bool ok = true;
    int64_t rx[3], rw = 0;
    auto locate = [&]() {
      const Unit un = decode(ctl, f, g.E, u);
#pragma unroll
      for (int c = 0; c < 3; ++c) rx[c] = min((int64_t)un.row0 + 32 * c + lane, g.rows - 1) * sck;  // clamped: unused rows
      rw = ((int64_t)un.e * nblk + un.n0 / kBlock) * sck;
    };
    uint32_t x[3], w0 = 0, w1 = 0;
    auto request = [&]() {
#pragma unroll
      for (int c = 0; c < 3; ++c) x[c] = sx32[rx[c] + gk];  // not __ldg: written while this kernel already runs
      w0 = __ldg(sw32 + rw + gk);
      w1 = __ldg(sw3_32 + rw + gk);
    };
    if (u < total && gk0 < gk1) {
      locate();
      request();
    }
    while (u < total && gk0 < gk1) {
      const uint32_t wx[4] = {x[0], x[1], x[2], x[2]}, v0 = w0, v1 = w1;
      if (++gk == gk1) {
        gk = gk0;
        u += ncl;
        if (u < total) locate();
      }
      if (u < total) request();
      ok = ptx::mbar_wait(ptx::smem_u32(&ctl->sf_empty[set]), phase ^ 1u, timeout_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      tmem_st_x4(dst + set * kSfStep, v0, v0, v0, v0);
      tmem_st_x4(dst + set * kSfStep + 4, v1, v1, v1, v1);
      tmem_st_x4(dst + set * kSfStep + 8, wx[0], wx[1], wx[2], wx[3]);
      tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&ctl->sf_full[set]));
      if (++set == kSfSets) {
        set = 0;
        phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x980u + kKind);
      ctl->abort = 1;
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    // A warp here runs alone on its scheduler for the most part, so what counts is the length of its
    // instruction chain: rows eight at a time (short code, fetched once), two sets of warps.
    if (!f.first) pdl_wait();  // the dispatch writes the layer's gates; and the limits of the waits run from here
    const int q = warp & 3, set = (warp - kEpiWarp0) >> 2, m = q * 32 + lane;  // m: weight row of the block
    // Rows 8 gi .. 8 gi + 7 fall to CTA gi % split, which counts them its group gi / split; a set takes
    // every other one of these counts.  Where the others' sums land: [other CTA, this one left out].
    const float* mine = recv + m;
    const int recv_floats = f.recv_bytes / 4, me = (int)rank;
    const int64_t scn = scale_cols(g.n);
    constexpr int kOsz = kKind == kSwiGLU ? 1 : kKind == kOutBf16 ? 2 : 4;
    const int64_t pitch = (int64_t)g.n * kOsz;
    int acc = 0, turn = 0;
    uint32_t acc_phase = 0, full_phase = 0, free_phase = 0;
    bool ok = true;
    for (int u = cid; u < total; u += ncl) {
      const Unit un = decode(ctl, f, g.E, u);
      const int col = un.n0 + m;
      const bool in = col < g.n;
      float gate0 = 1.f, gate1 = 1.f, gate2 = 1.f;  // of rows lane, lane + 32 and lane + 64
      if (kKind != kSwiGLU && g.gate) {
        if (lane < un.rows) gate0 = g.gate[un.row0 + lane];
        if (lane + 32 < un.rows) gate1 = g.gate[un.row0 + lane + 32];
        if (lane + 64 < un.rows) gate2 = g.gate[un.row0 + lane + 64];
      }
      ok = ptx::mbar_wait(ptx::smem_u32(&ctl->tfull[acc]), acc_phase, timeout_ns, abort_flag);
      if (kSplit && u != cid) {
        ok = ok && wait_cluster(ptx::smem_u32(&ctl->rfree), free_phase, timeout_ns, abort_flag);
        free_phase ^= 1u;
      }
      ok = epi_bar_and(set, ok);  // the set's four warps go on or stop together
      if (!ok) break;
      ptx::tc_fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * 2 * kMaxTok);
      const int owners = min(split, (un.rows + 7) / 8);  // CTAs that have rows of this unit
      if constexpr (kSplit) {
        const uint32_t base = ptx::smem_u32(recv) + (uint32_t)(m * 4);
#pragma unroll 1
        for (int li = set; 8 * li * split < un.rows; li += 2)
#pragma unroll 1
          for (int to = 0; to < split; ++to) {
            const int c = 8 * (li * split + to);
            if (to == me || c >= un.rows) continue;
            const uint32_t dst = ptx::mapa(base + (uint32_t)((me - (me > to)) * f.recv_bytes + li * 8 * 512), (uint32_t)to);
#pragma unroll 1
            for (int mt = 0; mt < kMats; ++mt) {
              uint32_t v[8];
              tmem_ld_x8(t_row + kMaxTok * mt + c, v);
              ptx::tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 8; ++i) st_cluster_f32(dst + (uint32_t)(mt * f.part * 512) + 512 * i, v[i]);
            }
          }
        __syncwarp();
        if (lane < owners && lane != me) ptx::mbar_arrive_cluster(ptx::mapa(ptx::smem_u32(&ctl->rfull), (uint32_t)lane));
        if (me < owners) {
          ok = wait_cluster(ptx::smem_u32(&ctl->rfull), full_phase, timeout_ns, abort_flag);
          full_phase ^= 1u;
          ok = epi_bar_and(set, ok);
          if (!ok) break;
        }
      }
      {
        auto load = [&](int mt, int c, float(&v)[8]) {
          uint32_t w[8];
          tmem_ld_x8(t_row + kMaxTok * mt + c, w);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = kSplit ? 0.f : __uint_as_float(w[i]);
          if constexpr (kSplit) {
            const float* o = mine + (mt * f.part + 8 * (c / 8 / split)) * 128;
#pragma unroll 1
            for (int r = 0; r < split; ++r) {  // in rank order, whichever CTA adds
              float x[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] = r == me ? __uint_as_float(w[i]) : o[128 * i];
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] += x[i];
              if (r != me) o += recv_floats;
            }
          }
        };
#pragma unroll 1
        for (int c = 8 * (set * split + me); c < un.rows; c += 16 * split) {
          const int nt = un.rows - c;
          const int64_t p0 = (int64_t)un.row0 + c;
          uint8_t* out = reinterpret_cast<uint8_t*>(g.out) + p0 * pitch + (int64_t)col * kOsz;
          if constexpr (kKind == kSwiGLU) {
            float a[8], b[8];
            load(0, c, a);
            load(1, c, b);
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) a[i] = silu_hidden(a[i]) * b[i];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // the row's largest value over this warp's 32 columns, kept by lane i
              const uint32_t t = __reduce_max_sync(0xffffffffu, in ? abs_bits(a[i]) : 0u);
              if (lane == i) top = t;
            }
            if (lane < 8) ctl->top[set][turn][q][lane] = top;
            epi_bar_and(set, true);
            const uint32_t* o = &ctl->top[set][turn][0][lane & 7];
            top = max(max(o[0], o[8]), max(o[16], o[24]));
            turn ^= 1;
            const uint32_t sb = scale_byte(__uint_as_float(top));
            const float fac = inv_scale_value(sb);
            if (q == 0 && lane < min(nt, 8)) g.out_scales[(p0 + lane) * scn + un.n0 / kBlock] = (uint8_t)sb;
#pragma unroll
            for (int i = 0; i < 8; ++i, out += pitch) {
              const float fi = __shfl_sync(0xffffffffu, fac, i);
              if (i < nt && in) *out = (uint8_t)pack_e4m3x2(a[i] * fi, 0.f);
            }
          } else {
            float v[8];
            load(0, c, v);
            const float gates = c < 32 ? gate0 : c < 64 ? gate1 : gate2;
#pragma unroll
            for (int i = 0; i < 8; ++i, out += pitch) {
              const float y = __shfl_sync(0xffffffffu, gates, (c + i) & 31) * v[i];
              if (i < nt && in) store_act(out, kKind == kOutBf16, 0, y);
            }
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&ctl->tempty[acc]));
        // Read: the others may send the next unit's sums (after the last unit no one waits for this).  One
        // that has no rows of the next unit may arrive for that too before all others' arrivals for this
        // one have landed here; it has seen them, so the sums were read by then.
        if (kSplit && lane < split && lane != me && u + ncl < total)
          ptx::mbar_arrive_cluster(ptx::mapa(ptx::smem_u32(&ctl->rfree), (uint32_t)lane));
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x990u + kKind);
      ctl->abort = 1;
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // copies already in flight land within microseconds; give them 200 us before the shared
    // memory they target goes away
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 200000ull) {
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  // No CTA's shared memory goes while another may still write to it.  After an undisturbed run none
  // does: a CTA has waited for all sums of its rows, and for every release but the last unit's, which
  // is not sent; so it leaves at once and makes room for the next launch.
  if (kSplit && *abort_flag) ptx::cluster_sync();
  if (warp == kSfWarp0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kTmemCols);
  }
}

constexpr int kSmemMax = 232448;
constexpr int kMaxSplit = 8;

// Clusters of `split` CTAs, each CTA alone on its SM, that run at the same time.  A cluster lies within
// a group of SMs that the hardware has, so this is less than SMs / split (152 SMs: 36 clusters of 4, 15 of 8).
template <int kKind>
int most_clusters(int device, int split) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices][kMaxSplit + 1];
  const bool keep = device >= 0 && device < kMaxDevices;
  if (keep)
    if (const int n = known[device][split].load(std::memory_order_acquire)) return n;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)split;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)split);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemMax;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, gemm_fp8_few_kernel<kKind, true>, &cfg) != cudaSuccess || n < 1) n = 1;
  if (keep) known[device][split].store(n, std::memory_order_release);
  return n;
}

template <int kKind>
cudaError_t launch_kind(const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first, int device,
                        int num_sms, int64_t timeout_ns, cudaStream_t st) {
  constexpr int kMats = kKind == kSwiGLU ? 2 : 1;
  cudaError_t e;
  static std::atomic<uint64_t> asked{0};  // devices on which the kernels may use all shared memory
  const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
  if (!(asked.load(std::memory_order_acquire) & bit) || !bit) {
    constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    if ((e = cudaFuncSetAttribute(gemm_fp8_few_kernel<kKind, false>, kAttr, kSmemMax)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(gemm_fp8_few_kernel<kKind, true>, kAttr, kSmemMax)) != cudaSuccess) return e;
    asked.fetch_or(bit, std::memory_order_release);
  }
  FewShape f{};
  f.n_seg = n_seg;
  f.first = first ? 1 : 0;
  f.tok = g.rows <= 16 ? 16 : g.rows <= 32 ? 32 : g.rows <= 64 ? 64 : kMaxTok;
  f.stage_bytes = kMats * kWBytes + f.tok * kBK;
  // rows of a CTA in a cluster of s, and the shared memory for the others' sums of them
  auto part = [&](int s) { return (f.tok / 8 + s - 1) / s * 8; };
  auto recv = [&](int s) { return s == 1 ? 0 : kMats * part(s) * kWRows * 4; };
  // Units, when the segments differ by no more than a quarter; clusters that run all of them at once (a second
  // unit of a cluster waits for the first one's epilogue).  K is split in whole groups of four blocks (of
  // the splits with the same longest part the smallest), and the others' sums need shared memory.
  const int64_t nblk = (g.n + kWRows - 1) / kWRows, owners = g.rows < n_seg ? g.rows : n_seg;
  const int64_t top_rows = owners == 1 ? g.rows : (5 * g.rows + 4 * owners - 1) / (4 * owners);
  const int64_t units = owners * nblk * ((top_rows + f.tok - 1) / f.tok);
  const int sck = (int)(scale_cols(g.K) / 4), fixed = 1024 + (int)sizeof(Ctl);
  f.split = 1;
  for (int s = 2; s <= kMaxSplit && s <= sck && s * units <= num_sms; ++s) {
    if (fixed + (s - 1) * recv(s) + 4 * f.stage_bytes > kSmemMax || units > most_clusters<kKind>(device, s)) break;
    if ((sck + s - 1) / s < (sck + f.split - 1) / f.split) f.split = s;
  }
  f.part = part(f.split);
  f.recv_bytes = recv(f.split);
  f.stages = (kSmemMax - fixed - (f.split - 1) * f.recv_bytes) / f.stage_bytes;
  if (f.stages > kMaxStages) f.stages = kMaxStages;
  const size_t smem = (size_t)fixed + (size_t)(f.split - 1) * f.recv_bytes + (size_t)f.stages * f.stage_bytes;
  CUtensorMap mX, mW, mW3;
  const uint64_t wrows = (uint64_t)g.E * (uint64_t)g.n;
  if ((e = make_tmap_rows128(&mX, g.a, 1, (uint64_t)g.rows, (uint64_t)g.K, kTokBox)) != cudaSuccess) return e;
  if ((e = make_tmap_rows128(&mW, g.b, 1, wrows, (uint64_t)g.K, kWRows)) != cudaSuccess) return e;
  mW3 = mW;
  if (kMats == 2 && (e = make_tmap_rows128(&mW3, g.b3, 1, wrows, (uint64_t)g.K, kWRows)) != cudaSuccess) return e;
  const int64_t clusters = num_sms / f.split, most = (g.rows / f.tok + owners) * nblk;  // no more units than that
  const int grid = (int)(clusters < most ? clusters : most) * f.split;
  auto kern = f.split > 1 ? gemm_fp8_few_kernel<kKind, true> : gemm_fp8_few_kernel<kKind, false>;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), smem, st, true, f.split, mX, mW, mW3, g, ws, seg_counts, f,
                       timeout_ns);
}

}  // namespace

cudaError_t launch_gemm_few(int kind, const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first,
                            int device, int num_sms, int64_t timeout_ns, cudaStream_t st) {
  switch (kind) {
    case kSwiGLU: return launch_kind<kSwiGLU>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
    case kOutBf16: return launch_kind<kOutBf16>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
    default: return launch_kind<kOutF32>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
  }
}

}  // namespace fp8
}  // namespace moe
