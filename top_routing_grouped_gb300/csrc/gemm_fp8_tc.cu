// gemm_fp8_tc.cu -- the 8-bit grouped products on CTA pairs (2-SM tcgen05.mma with block
// factors, kind::mxf8f6f4.block_scale).
//
//   out[p, n] = sum_j 2^(sA[p,j] + sW[n/128,j]) sum_{k in block j} A[p,k] W_e[n,k]   (j: 128 k's)
//
// A power-of-two factor for a block of 128 is the tensor core's own factor for a block of 32,
// given four times: the MMA multiplies by both factors while it accumulates, so nothing is
// rescaled between K blocks and the accumulator stays in TMEM over the whole sum.
//
// Tiles, ring and roles are those of gemm_tc2.cu: a cluster of two CTAs computes 256 x 256 with
// one MMA stream issued by the leader, each CTA loads its own 128 rows of A and its half of the
// 256 weight rows (SwiGLU: the leader W1's 128, the peer W3's), 128 k's (128 bytes) a stage, so a
// stage is 32 KB and takes 512 clocks of MMA, as in bf16 with half the k's.
//
// Factors.  A 32-bit word holds a row's bytes of four K blocks, in the order the rows' scale
// bytes lie in memory; the instruction descriptor picks the byte of the current block, so one
// load of words serves 512 k's.  Four warps of each CTA, one for each TMEM lane quarter, gather the
// words of the CTA's 128 rows and of the tile's two blocks of weight rows and store them to TMEM (the
// same words in every quarter; column c of a group of four belongs to rows 32c..32c+31) up to four
// groups ahead of the MMAs (two sets instead of four: 5-7 % slower).
//
// TMEM.  The sets take 64 columns, so the two accumulators of 256 columns overlap by 64: the
// epilogue warps that own those columns read them first and hand them over before they go on, and
// the next tile's MMAs start then.
//
// SwiGLU epilogue: the 128 columns of a tile are one block of each hidden row.  Two warps share a
// row's 128 values (64 each), agree on the largest one through shared memory, and write e4m3 and
// one factor byte, so the hidden rows cost N*F bytes instead of 2*N*F twice.
//
// What bounds it.  At the full MMA rate the ring alone moves 64 bytes a clock into shared memory and
// the MMAs read 64 out of it, all that it has; the output tiles pass through it too (staging, TMA store:
// 1000 clocks a tile).  Counted in clocks, the MMAs run 91 % of the time from a CTA's first to its last on
// 8192 x 8192 x 2048 (64 K blocks a tile) and 80 % on 8192 x 2048 x 8192 (16 K blocks), where handing over the
// shared columns costs about 700 of 10200 clocks a tile.  Before the first MMA go some 5000 clocks, half
// of them until the tiles are found, half for the first loads.  With one to four K blocks a tile the
// SwiGLU epilogue bounds it, some 4000 clocks a tile (51482 rows of 32 experts of 128 x 3024: 165 us).
// Times: 85 us for 8192 x 2048 x 8192 (3.2 PFLOP/s), 80 us for 8192 x 4096 x 4096 (3.4), 11 us for 2048 x
// 2048 x 2048, 2.24 ms for 131072 rows of 64 experts of 4096 x 2048 (2.95, at 1.55 GHz under the power cap).
//
// Tried and dropped: 224-wide tiles, whose accumulators share no columns (the ring's time per K block
// does not shrink with the tile: 98 -> 106 us); the output stored from registers, 32 bytes a lane, and
// five stages and two store blocks a warp, and L2 eviction priorities for A and the output (no
// difference beyond noise).
//
// Waits are bounded (MOE_ERR_TIMEOUT, no trap); an abort raises the flag in both CTAs; the pair
// meets at cluster barriers before TMEM is released.
#include <cuda.h>
#include <cuda_bf16.h>

#include <stddef.h>

#include <atomic>

#include "fp8_common.cuh"
#include "fp8_mma.cuh"
#include "fp8_units.cuh"
#include "gemm_tc.h"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace moe {
namespace fp8 {
namespace {

constexpr int kBK = 128;  // bytes = k's per stage: one block of factors
constexpr int kStages = 6;
constexpr int kRowsPerCta = 128;
constexpr int kMmaM = 256;
constexpr int kMmaN = 256;
constexpr int kMmaK = 32;
constexpr int kABytes = kRowsPerCta * kBK;
constexpr int kBHalfBytes = (kMmaN / 2) * kBK;
constexpr int kStageBytes = kABytes + kBHalfBytes;
constexpr int kThreads = 512;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;  // two per TMEM lane quarter, one per half of the tile's columns
constexpr int kSfWarp0 = 12;
constexpr int kSfWarps = 4;   // one per TMEM lane quarter
// Registers a thread: the launch gives every thread 128; the TMA / MMA warps and the factor warps
// hand some to the epilogue (256 * 72 + 256 * 184 <= 512 * 128).
constexpr int kRegsFew = 72, kRegsEpi = 184;

// TMEM columns: accumulator i at 192 i (256 wide), factor set i at 448 + 16 i (4 of A, 8 of B)
constexpr int kTmemCols = 512;
constexpr int kAccStep = 192;
constexpr int kSfCol = 448;
constexpr int kSfStep = 16;
constexpr int kSfSets = 4;

constexpr int kStgBlockBytes = 32 * 128;      // a store block: 32 rows of 128 bytes, swizzled
constexpr int kStgBytes = kEpiWarps * kStgBlockBytes;

struct Ctl {
  uint64_t full[kStages];   // leader's: both CTAs' bytes of a stage
  uint64_t empty[kStages];  // each CTA: stage free again (leader's multicast commit)
  uint64_t tfull[2];        // each CTA: accumulator ready (leader's multicast commit)
  uint64_t tempty[2];       // leader's: both CTAs' epilogue warps have read the accumulator
  uint64_t over;            // leader's: the columns the accumulators share have been read
  uint64_t sf_full[kSfSets];   // leader's: both CTAs' factor words of a group are in TMEM
  uint64_t sf_empty[kSfSets];  // each CTA: the group's MMAs have run (leader's multicast commit)
  uint64_t drain;
  uint32_t tmem_base;
  uint32_t peer_tmem_base;
  int abort;
  Segments seg;
};

constexpr size_t kSmemBytes = (size_t)kStages * kStageBytes + kStgBytes + sizeof(Ctl);
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

__device__ __forceinline__ uint32_t pack_bf16x2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

// 2-D tiled TMA store of a staged block (x = column, y = row), as a bulk group of its own
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int32_t x, int32_t y, uint32_t src) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
      "cp.async.bulk.commit_group;" ::"l"(reinterpret_cast<uint64_t>(map)),
      "r"(x), "r"(y), "r"(src)
      : "memory");
}
// this thread's bulk groups have read their shared-memory source / are complete
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Named barrier of the two warps of one lane quarter, with the AND of a flag over them.
__device__ __forceinline__ bool pair_bar_and(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %2, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"((uint32_t)v)
      : "memory");
  return r != 0;
}

template <int kRegs>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// Tile u of the segments: up to 16 m-tiles of a segment form a group whose tiles share a few weight
// tiles at a time (pairs of m-tiles fastest, then the weight tile, then the group), as in the bf16
// kernels' tables.  The m-tile of CTA `rank` of the pair; rows <= 0: there is none.
__device__ __forceinline__ int pairs_of(int cnt) { return ((cnt + kTileM - 1) / kTileM + 1) / 2; }
__device__ __forceinline__ TileInfo decode(const Segments* sg, int n_seg, int E, int n_tiles, int u, int rank) {
  constexpr int kPairs = kGroupM / 2;
  const int s = segment_of(sg, n_seg, u), row0 = sg->row0[s], cnt = sg->row0[s + 1] - row0;
  const int local = u - sg->unit0[s], grp = local / (kPairs * n_tiles), rem = local - grp * kPairs * n_tiles;
  const int gp = min(kPairs, pairs_of(cnt) - grp * kPairs);
  TileInfo ti;
  ti.e = s % E;
  ti.n_idx = rem / gp;
  const int m0 = grp * kGroupM * kTileM + (2 * (rem % gp) + rank) * kTileM;
  ti.row0 = row0 + m0;
  ti.rows = cnt - m0;  // to the end of its segment: may be above kTileM, or below 1 for a pair's second tile
  return ti;
}

// A warp's tiles in turn (first, first + stride, ...).  Decoding one takes some 700 clocks of search and
// division, a fifth of what an epilogue takes; the lanes decode the next 32 at once.
struct Tiles {
  TileInfo mine;
  int left = 0;  // decoded tiles not yet taken

  __device__ __forceinline__ TileInfo next(const Segments* sg, int n_seg, int E, int n_tiles, int tile, int stride, int total,
                                           int rank) {
    const int lane = threadIdx.x & 31;
    if (left == 0) {
      mine = decode(sg, n_seg, E, n_tiles, (int)min((uint32_t)tile + (uint32_t)(lane * stride), (uint32_t)total - 1u), rank);
      left = 32;
    }
    const int from = 32 - left--;
    TileInfo ti;
    ti.e = __shfl_sync(0xffffffffu, mine.e, from);
    ti.row0 = __shfl_sync(0xffffffffu, mine.row0, from);
    ti.rows = __shfl_sync(0xffffffffu, mine.rows, from);
    ti.n_idx = __shfl_sync(0xffffffffu, mine.n_idx, from);
    return ti;
  }
};

__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }

__device__ __forceinline__ void raise_abort(Ctl* ctl, uint32_t rank) {
  ctl->abort = 1;
  ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&ctl->abort), rank ^ 1u), 1u);
}

template <int kKind>
__global__ void __launch_bounds__(kThreads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmB3, const __grid_constant__ CUtensorMap tmY, GemmArgs g, Ws ws,
                    const int32_t* seg_counts, int n_seg, int first, int64_t timeout_ns) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* stages = smem_raw;  // the swizzled boxes need 1024-byte boundaries (checked below)
  uint8_t* stg_base = stages + kStages * kStageBytes;
  Ctl* ctl = reinterpret_cast<Ctl*>(stg_base + kStgBytes);
  // SwiGLU stages four blocks; the warps' maxima lie behind them: [half][128 rows]
  uint32_t* top_s = reinterpret_cast<uint32_t*>(stg_base + 4 * kStgBlockBytes);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  const bool leader = rank == 0;
  const int cid = (int)ptx::cluster_id_x();
  const int ncl = (int)ptx::cluster_count_x();

  constexpr int bn = kKind == kSwiGLU ? kMmaN / 2 : kMmaN;  // output columns per tile
  const int n_tiles = (g.n + bn - 1) / bn;
  const int kblocks = (g.K + kBK - 1) / kBK;
  const int sck = (int)(scale_cols(g.K) / 4);  // words of factors per row
  const int nb = (g.n + kBlock - 1) / kBlock;

  // Setting up takes microseconds where its steps wait for one another: warp 8 makes the barriers and warp 9,
  // once the peer has started, takes TMEM, while the others wait for the previous kernel or find the tiles.
  asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
  if (threadIdx.x == 8 * 32) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->full[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&ctl->empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->tfull[i]), 1);
      ptx::mbar_init(ptx::smem_u32(&ctl->tempty[i]), 2 * kEpiWarps);
    }
    ptx::mbar_init(ptx::smem_u32(&ctl->over), kEpiWarps);  // half of both CTAs' epilogue warps
    for (int i = 0; i < kSfSets; ++i) {
      ptx::mbar_init(ptx::smem_u32(&ctl->sf_full[i]), 2 * kSfWarps);
      ptx::mbar_init(ptx::smem_u32(&ctl->sf_empty[i]), 1);
    }
    ptx::mbar_init(ptx::smem_u32(&ctl->drain), 1);
    ctl->abort = 0;
    ptx::fence_mbar_init();
  }
  if (threadIdx.x == 10 * 32) {
    ptx::tma_prefetch_desc(&tmA);
    ptx::tma_prefetch_desc(&tmB);
    if (kKind == kSwiGLU) ptx::tma_prefetch_desc(&tmB3);
    ptx::tma_prefetch_desc(&tmY);
  }
  cluster_wait();
  if (warp == 9) {
    ptx::tmem_alloc_pair(ptx::smem_u32(&ctl->tmem_base), kTmemCols);
    ptx::tmem_relinquish_pair();
    if (lane == 0) ptx::st_cluster_u32(ptx::mapa(ptx::smem_u32(&ctl->peer_tmem_base), rank ^ 1u), ctl->tmem_base);
  }
  asm volatile("barrier.cluster.arrive;" ::: "memory");  // both CTAs' barriers exist before any load or cross-CTA arrive
  // The call's first launch waits here for the counts and the activations; its second one waits for
  // the hidden rows alone, once it has found its tiles, as does a call without counts.
  const bool counts_ready = !first || seg_counts == nullptr;
  if (!counts_ready) pdl_wait();
  int total = scan_segments(&ctl->seg, seg_counts, n_seg, g.rows, [&](int cnt) { return pairs_of(cnt) * n_tiles; });
  if (counts_ready) pdl_wait();
  if (first) begin_status(ws, total < 0, 0x900u);
  total = max(total, 0);
  pdl_launch_dependents();
  cluster_wait();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl->tmem_base;
  // a pair's accumulators must sit at the same TMEM address, the ring on its boundary
  if (ctl->peer_tmem_base != tmem || (ptx::smem_u32(stages) & 1023u) != 0) {
    if (threadIdx.x == 0) {
      const uint64_t t0 = global_ns();  // not before CTA 0 has set the status word
      while (global_ns() - t0 < kMinTimeoutNs) {
      }
      record_error(ws, MOE_ERR_INTERNAL, 0x908u + kKind);
    }
    total = 0;
  }
  volatile int* abort_flag = &ctl->abort;

  if (warp < kEpiWarp0) {
    regs_dec<kRegsFew>();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- TMA producers (both CTAs)
      // Warp 0 loads A, warp 2 the weights; the warps run converged and one elected lane issues (205
      // clocks for a wait, an arrive and a load; 337 for one lane in a branch of its own, close to
      // the 512 that a stage's MMAs take).
      const bool a_side = warp == 0;
      const CUtensorMap* map = a_side ? &tmA : (kKind == kSwiGLU && rank == 1) ? &tmB3 : &tmB;
      const uint32_t ctl0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ctl), 0);
      const uint32_t bar0 = __shfl_sync(0xffffffffu, ptx::mapa(ctl0 + (uint32_t)offsetof(Ctl, full), 0), 0);
      const uint32_t dst0 = __shfl_sync(0xffffffffu, ptx::smem_u32(stages), 0) + (a_side ? 0u : (uint32_t)kABytes);
      const int first_tile = __shfl_sync(0xffffffffu, cid, 0), stride = __shfl_sync(0xffffffffu, ncl, 0);
      const int tiles_end = __shfl_sync(0xffffffffu, total, 0);
      const bool elected = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      Tiles tiles;
      for (int tile = first_tile; tile < tiles_end && ok; tile += stride) {
        const TileInfo ti = tiles.next(&ctl->seg, n_seg, g.E, n_tiles, tile, stride, tiles_end, (int)rank);
        // a pair's second m-tile may not exist: its A rows are neither loaded nor waited for (the leader's
        // view; its peer expects nothing)
        const uint32_t bytes = ti.rows > kTileM ? 2 * kStageBytes : 2 * kStageBytes - kABytes;
        const int brow = ti.e * g.n + ti.n_idx * bn + (kKind == kSwiGLU ? 0 : (int)rank * (kMmaN / 2));
        const int y = __shfl_sync(0xffffffffu, a_side ? ti.row0 : brow, 0);
        const bool load = !a_side || ti.rows > 0;
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(ctl0 + (uint32_t)offsetof(Ctl, empty) + 8 * stage, phase ^ 1u,
                                                      timeout_ns, abort_flag)) != 0;
          if (!ok) break;
          if (elected) {
            if (a_side && leader) ptx::mbar_arrive_expect_tx(ctl0 + (uint32_t)offsetof(Ctl, full) + 8 * stage, bytes);
            if (load) ptx::tma_load_2d_pair(dst0 + stage * kStageBytes, map, kb * kBK, y, bar0 + 8 * stage);
          }
          __syncwarp();
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && elected) {
        record_error(ws, MOE_ERR_TIMEOUT, 0x910u + kKind);
        raise_abort(ctl, rank);
      }
    } else if (warp == 1 && leader) {
      // ---------------------------------------------------------- MMA issuer (leader only)
      // The whole warp runs the loop and one elected lane issues: with every operand the same in
      // all lanes for the compiler to see, an MMA costs 39 clocks to issue; from a branch of one
      // lane it cost 93, and issuing, at 680 clocks a stage, was what bound the kernel.
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int first_tile = __shfl_sync(0xffffffffu, cid, 0), stride = __shfl_sync(0xffffffffu, ncl, 0);
      const int tiles_end = __shfl_sync(0xffffffffu, total, 0);
      const uint64_t desc0 = ptx::desc_kmajor_sw128(__shfl_sync(0xffffffffu, ptx::smem_u32(stages), 0));
      const uint32_t ctl0 = __shfl_sync(0xffffffffu, ptx::smem_u32(ctl), 0);
      const bool elected = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, ptx::mbar_wait(ctl0 + bar, parity, timeout_ns, abort_flag)) != 0;
      };
      int stage = 0, acc = 0, set = 0;
      uint32_t phase = 0, acc_phase = 0, over_phase = 0, sf_phase = 0;
      bool ok = true, first = true;
      for (int tile = first_tile; tile < tiles_end && ok; tile += stride) {
        const uint32_t d_tmem = tm + (uint32_t)(acc * kAccStep);
        uint32_t sf = 0;
        for (int kb = 0; kb < kblocks; ++kb) {
          if ((kb & 3) == 0) {  // a new group: its factors
            if (!(ok = wait(offsetof(Ctl, sf_full) + 8 * set, sf_phase))) break;
            sf = tm + (uint32_t)(kSfCol + set * kSfStep);
          }
          if (!(ok = wait(offsetof(Ctl, full) + 8 * stage, phase))) break;
          if (kb == 0) {
            // The accumulator before the last has been read, and so have the columns shared with the
            // last one: waited for when all else is there, since the MMAs stand still until then.
            ok = wait(offsetof(Ctl, tempty) + 8 * acc, acc_phase ^ 1u) && (first || wait(offsetof(Ctl, over), over_phase));
            if (!ok) break;
            if (!first) over_phase ^= 1u;
            first = false;
          }
          ptx::tc_fence_after();
          const bool last_of_group = (kb & 3) == 3 || kb + 1 == kblocks;
          if (elected) {
            const uint64_t da = desc0 + (uint64_t)(stage * (kStageBytes >> 4)), db = da + (kABytes >> 4);
            const uint32_t idesc = idesc_mxf8(kMmaM, kMmaN, 0) | (uint32_t)(kb & 3) * idesc_byte();
#pragma unroll
            for (int ks = 0; ks < kBK / kMmaK; ++ks)
              mma_mxf8_pair(d_tmem, da + ks * (kMmaK >> 4), db + ks * (kMmaK >> 4), idesc, sf, sf + 4, (kb | ks) != 0 ? 1u : 0u);
            ptx::mma_commit_pair_multicast(ctl0 + offsetof(Ctl, empty) + 8 * stage, 0x3);
            if (last_of_group) ptx::mma_commit_pair_multicast(ctl0 + offsetof(Ctl, sf_empty) + 8 * set, 0x3);
          }
          __syncwarp();
          if (last_of_group && ++set == kSfSets) {
            set = 0;
            sf_phase ^= 1u;
          }
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elected) ptx::mma_commit_pair_multicast(ctl0 + offsetof(Ctl, tfull) + 8 * acc, 0x3);
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && elected) {
        record_error(ws, MOE_ERR_TIMEOUT, 0x920u + kKind);
        raise_abort(ctl, rank);
      }
      // every MMA of this pair has finished with both CTAs' TMEM
      if (elected) ptx::mma_commit_pair(ctl0 + offsetof(Ctl, drain));
      __syncwarp();
      ptx::mbar_wait(ctl0 + offsetof(Ctl, drain), 0u, timeout_ns, nullptr);
    }
    __syncwarp();
  } else if (warp >= kSfWarp0) {
    // ------------------------------------------------------------ factor words (both CTAs)
    regs_dec<kRegsFew>();
    const uint32_t* sa32 = reinterpret_cast<const uint32_t*>(g.sa);
    const uint32_t* sb32 = reinterpret_cast<const uint32_t*>(g.sb);
    const uint32_t* sb3_32 = reinterpret_cast<const uint32_t*>(kKind == kSwiGLU ? g.sb3 : g.sb);
    const uint32_t dst = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kSfCol;
    int set = 0;
    uint32_t phase = 0;
    bool ok = true;
    // The words of the next group are requested before the present group's wait, across tiles too:
    // a group of MMAs lasts about as long as one trip to L2.
    int tile = cid, gk = 0;
    int64_t ra[4], r0 = 0, r1 = 0;
    Tiles tiles;
    auto locate = [&]() {
      const TileInfo ti = tiles.next(&ctl->seg, n_seg, g.E, n_tiles, tile, ncl, total, (int)rank);
#pragma unroll
      for (int c = 0; c < 4; ++c)  // rows past the buffer belong to no output: any row's words do
        ra[c] = min((int64_t)ti.row0 + 32 * c + lane, g.rows - 1) * sck;
      const int blk = ti.n_idx * (bn / kBlock);
      r0 = ((int64_t)ti.e * nb + blk) * sck;
      r1 = kKind == kSwiGLU ? r0 : ((int64_t)ti.e * nb + min(blk + 1, nb - 1)) * sck;
    };
    uint32_t a[4], b0, b1;
    auto request = [&]() {
#pragma unroll
      for (int c = 0; c < 4; ++c) a[c] = sa32[ra[c] + gk];  // not __ldg: written while this kernel already runs
      b0 = __ldg(sb32 + r0 + gk);
      b1 = __ldg(sb3_32 + r1 + gk);
    };
    if (tile < total) {
      locate();
      request();
    }
    while (tile < total) {
      ok = ptx::mbar_wait(ptx::smem_u32(&ctl->sf_empty[set]), phase ^ 1u, timeout_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      ptx::tc_fence_after();
      tmem_st_x4(dst + set * kSfStep, a[0], a[1], a[2], a[3]);
      tmem_st_x4(dst + set * kSfStep + 4, b0, b0, b0, b0);
      tmem_st_x4(dst + set * kSfStep + 8, b1, b1, b1, b1);
      tmem_st_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_relaxed_cluster(ptx::mapa(ptx::smem_u32(&ctl->sf_full[set]), 0));
      if (++set == kSfSets) {
        set = 0;
        phase ^= 1u;
      }
      if (++gk == sck) {
        gk = 0;
        tile += ncl;
        if (tile < total) locate();
      }
      if (tile < total) request();
    }
    if (!ok && lane == 0) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x930u + kKind);
      raise_abort(ctl, rank);
    }
  } else {
    // ------------------------------------------------------------ epilogue (both CTAs)
    regs_inc<kRegsEpi>();
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const int r = q * 32 + lane;
    const uint32_t over = ptx::mapa(ptx::smem_u32(&ctl->over), 0);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    Tiles tiles;
    for (int tile = cid; tile < total; tile += ncl) {
      const TileInfo ti = tiles.next(&ctl->seg, n_seg, g.E, n_tiles, tile, ncl, total, (int)rank);
      ok = ptx::mbar_wait(ptx::smem_u32(&ctl->tfull[acc]), acc_phase, timeout_ns, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (kKind != kSwiGLU && !ok) break;
      ptx::tc_fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kAccStep);
      // accumulator 0 shares its last 64 columns (the upper half's), accumulator 1 its first 64
      const bool shares = acc == 1 - half;
      const bool flip = acc == 0 && half == 1;  // the shared columns lie in the second piece: take it first
      const uint32_t tempty = ptx::mapa(ptx::smem_u32(&ctl->tempty[acc]), 0);
      auto arrive = [&](uint32_t bar) {  // after this warp's loads so far
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_relaxed_cluster(bar);
      };
      const bool valid = r < ti.rows;
      const int64_t p = (int64_t)ti.row0 + r;
      const int n0 = ti.n_idx * bn;
      const int vw = ti.rows - q * 32;  // rows of this warp's 32 that belong to the tile's expert
      if constexpr (kKind == kSwiGLU) {
        // This warp's 64 hidden columns: W1's products at c, W3's at 128 + c.  The side that lies in
        // the shared columns is loaded first and whole, the other 32 columns at a time.
        float h[64];
        uint32_t top = 0;
        const int c0 = half * 64;
        const uint32_t t_first = t_row + (flip ? kMmaN / 2 : 0) + c0, t_second = t_row + (flip ? 0 : kMmaN / 2) + c0;
        uint32_t f0[32], f1[32];
        ptx::tmem_ld_32cols(t_first, f0);
        ptx::tmem_ld_32cols(t_first + 32, f1);
        ptx::tmem_ld_wait();
        if (shares) arrive(over);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t s[32];
          ptx::tmem_ld_32cols(t_second + 32 * u, s);
          ptx::tmem_ld_wait();
          if (u == 1) arrive(tempty);
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = __uint_as_float(u == 0 ? f0[i] : f1[i]), y = __uint_as_float(s[i]);
            float v = silu_hidden(flip ? y : x) * (flip ? x : y);
            if (n0 + c0 + 32 * u + (i & ~15) >= g.n) v = 0.f;  // columns past the expert (n is a multiple of 16)
            h[32 * u + i] = v;
            top = max(top, abs_bits(v));
          }
        }
        top_s[half * kRowsPerCta + r] = top;
        if (half == 0 && lane == 0) bulk_wait_read();  // the quarter's last store has left its block
        if (!pair_bar_and(1 + q, ok)) {
          ok = false;
          break;
        }
        const uint32_t sb = scale_byte(__uint_as_float(max(top, top_s[(half ^ 1) * kRowsPerCta + r])));
        const float f = inv_scale_value(sb);
        const uint32_t stg = ptx::smem_u32(stg_base) + (uint32_t)(q * kStgBlockBytes);
        uint8_t* hrow = reinterpret_cast<uint8_t*>(g.out) + p * g.n + n0;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = pack_e4m3x4(h[16 * v + 4 * i] * f, h[16 * v + 4 * i + 1] * f, h[16 * v + 4 * i + 2] * f,
                               h[16 * v + 4 * i + 3] * f);
          const int j = half * 4 + v;
          if (vw >= 32)
            st_shared_v4(stg + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) * 16)), w[0], w[1], w[2], w[3]);
          else if (valid && n0 + 16 * j < g.n)
            *reinterpret_cast<uint4*>(hrow + 16 * j) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (half == 0 && valid) g.out_scales[p * scale_cols(g.n) + ti.n_idx] = (uint8_t)sb;
        if (vw >= 32) fence_async();
        pair_bar_and(1 + q, true);
        if (vw >= 32 && half == 0 && lane == 0) tma_store_2d(&tmY, n0, ti.row0 + q * 32, stg);
      } else {
        const float gate = !valid ? 0.f : g.gate ? g.gate[p] : 1.f;
        const uint32_t stg = ptx::smem_u32(stg_base) + (uint32_t)((warp - kEpiWarp0) * kStgBlockBytes);
        constexpr int kCols = kKind == kOutBf16 ? 64 : 32;  // columns of a 128-byte store row
        constexpr int kPieces = 128 / kCols;
#pragma unroll 1
        for (int u = 0; u < kPieces; ++u) {
          const int c = half * 128 + (flip ? kPieces - 1 - u : u) * kCols;
          uint32_t pk[32];
          if constexpr (kKind == kOutBf16) {
            uint32_t a[32], b[32];
            ptx::tmem_ld_32cols(t_row + c, a);
            ptx::tmem_ld_32cols(t_row + c + 32, b);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              pk[i] = pack_bf16x2(gate * __uint_as_float(a[2 * i]), gate * __uint_as_float(a[2 * i + 1]));
              pk[16 + i] = pack_bf16x2(gate * __uint_as_float(b[2 * i]), gate * __uint_as_float(b[2 * i + 1]));
            }
          } else {
            ptx::tmem_ld_32cols(t_row + c, pk);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = __float_as_uint(gate * __uint_as_float(pk[i]));
          }
          if (shares && u == 64 / kCols - 1) arrive(over);
          if (u == kPieces - 1) arrive(tempty);
          if (vw <= 0 || n0 + c >= g.n) continue;  // warp-uniform
          if (vw >= 32) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j)
              st_shared_v4(stg + (uint32_t)(lane * 128 + ((j ^ (lane & 7)) * 16)), pk[4 * j], pk[4 * j + 1], pk[4 * j + 2],
                           pk[4 * j + 3]);
            fence_async();
            __syncwarp();
            if (lane == 0) tma_store_2d(&tmY, n0 + c, ti.row0 + q * 32, stg);
          } else if (valid) {
            constexpr int kEsz = kKind == kOutBf16 ? 2 : 4;
            uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(g.out) + (p * g.n + n0 + c) * kEsz);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              if (n0 + c + v * (16 / kEsz) < g.n) d[v] = make_uint4(pk[4 * v], pk[4 * v + 1], pk[4 * v + 2], pk[4 * v + 3]);
          }
        }
      }
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    bulk_wait_all();  // the tiled stores this lane issued have been written
    if (!ok && lane == 0) {
      record_error(ws, MOE_ERR_TIMEOUT, 0x940u + kKind);
      raise_abort(ctl, rank);
    }
  }

  // ---------------------------------------------------------------- teardown
  __syncthreads();  // no warp of this CTA issues a copy any more
  if (*abort_flag && threadIdx.x == 0) {
    // copies already in flight land within microseconds; give them 200 us before the
    // shared memory they target goes away
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 200000ull) {
    }
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();  // neither CTA loads, computes or reads TMEM any more
  if (warp == 9) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// CTAs of a persistent launch: as many pairs as can be resident at once.  The kernel's attribute
// and the count are set and asked for once per kernel and device (a call of one token is shorter
// than the two questions); two threads that come first may both ask and store the same answer.
template <int kKind>
int persistent_grid(int device, int num_sms, cudaError_t* err) {
  auto kern = gemm_fp8_kernel<kKind>;
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  const bool keep = device >= 0 && device < kMaxDevices;
  *err = cudaSuccess;
  if (keep)
    if (const int g = known[device].load(std::memory_order_acquire)) return g;
  if ((*err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes)) != cudaSuccess) return 0;
  int grid = num_sms & ~1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 2;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0 && 2 * clusters < grid)
    grid = 2 * clusters;
  if (keep) known[device].store(grid, std::memory_order_release);
  return grid;
}

template <int kKind>
cudaError_t launch_kind(const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first, int device,
                        int num_sms, int64_t timeout_ns, cudaStream_t st) {
  constexpr int kEsz = kKind == kSwiGLU ? 1 : kKind == kOutBf16 ? 2 : 4;
  CUtensorMap mA, mB, mB3, mY;
  cudaError_t e;
  const uint64_t wrows = (uint64_t)g.E * (uint64_t)g.n;
  if ((e = make_tmap_rows128(&mA, g.a, 1, (uint64_t)g.rows, (uint64_t)g.K, kRowsPerCta)) != cudaSuccess) return e;
  if ((e = make_tmap_rows128(&mB, g.b, 1, wrows, (uint64_t)g.K, kMmaN / 2)) != cudaSuccess) return e;
  mB3 = mB;
  if (kKind == kSwiGLU && (e = make_tmap_rows128(&mB3, g.b3, 1, wrows, (uint64_t)g.K, kMmaN / 2)) != cudaSuccess) return e;
  if ((e = make_tmap_rows128(&mY, g.out, kEsz, (uint64_t)g.rows, (uint64_t)g.n, 32)) != cudaSuccess) return e;
  auto kern = gemm_fp8_kernel<kKind>;
  const int grid = persistent_grid<kKind>(device, num_sms, &e);
  if (e != cudaSuccess) return e;
  return launch_kernel(kern, dim3((unsigned)grid), dim3(kThreads), kSmemBytes, st, true, 2, mA, mB, mB3, mY, g, ws, seg_counts,
                       n_seg, first ? 1 : 0, timeout_ns);
}

}  // namespace

cudaError_t launch_gemm_tc(int kind, const GemmArgs& g, const Ws& ws, const int32_t* seg_counts, int n_seg, bool first,
                           int device, int num_sms, int64_t timeout_ns, cudaStream_t st) {
  switch (kind) {
    case kSwiGLU: return launch_kind<kSwiGLU>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
    case kOutBf16: return launch_kind<kOutBf16>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
    default: return launch_kind<kOutF32>(g, ws, seg_counts, n_seg, first, device, num_sms, timeout_ns, st);
  }
}

}  // namespace fp8
}  // namespace moe
