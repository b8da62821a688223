// Product of two matrices in 8 bits with a scale for each block of 128 along K (of one row, or
// of 128 rows):
//
//   S[m, n] = sum over blocks b of sA[m, b] sB[n, b] T_b[m, n],   T_b = sum in b of a b
//   D = alpha S + beta C     PostAct = act(same)        (or the backward activation epilogue)
//
// The scales are fp32, so they cannot go through the tensor core (its block
// scales are powers of two or 8 bits): a k-tile is one block, and its T_b, accumulated by
// tcgen05.mma kind::f8f6f4 in tensor memory, is read, scaled and added to fp32 sums that stay in
// registers over the whole of K.  (sA sB is rounded before it meets T_b, so a product below 2^-126
// loses up to 2^-150.  Measured and left: to look at every block's product and take the scales
// apart there, 8192^3 387 -> 412 us and the weight gradient 176 -> 208, and four times as long where
// every warp has a row of zeros, whose least scale is such a case.)  What follows from that:
//   * tensor memory holds no sums but the T_b in flight, and two warpgroups hold a tile's, a row
//     and half of the columns a thread.  A block costs a warp its waits and loads' latency, some
//     400 cycles, whatever its columns.  Large products take 256 x 256 tiles on a CTA pair: 128
//     columns a thread, 224 registers (setmaxnreg takes them from the warpgroup that loads and
//     issues), two buffers of 256 columns.  A block then takes 810 cycles, 512 of them the tensor
//     core's: 8192^3 380 us at 2.07 GHz (without the additions 335; over seconds, at the power cap's
//     1.72 GHz, 423).  Measured and left: 256 x 128 tiles with
//     four buffers (590), two MMAs of 128 columns a block, each half's buffers handed back by
//     itself (444), the next block's first load under a block's last additions (439);
//   * other products take 128 x 128 or 128 x 64 tiles on one CTA, with four buffers.  Their sums
//     go to shared memory when K ends, where a third warpgroup turns them into outputs while the
//     next tile's are added (or, split along K, while nothing else is left to do);
//   * a thread that makes outputs has a row's 128 columns, a block of an 8-bit output's scales:
//     its largest value is found without leaving the thread;
//   * a thread's row has one scale a block, and with blocks of 128 rows its columns have one,
//     too: a product and one packed fused multiply-add for two values.  With a scale for each
//     row of B (weight gradients) two packed operations, the columns' scales out of shared memory;
//     (8192^3 578 us, 4096 x 1536 x 16384 with an fp32 C 176: shared memory's loads of them);
//   * scales come through a ring of their own, by two warps' cp.async, eight blocks at a time and
//     up to sixteen ahead: they may lie anywhere (the rows of a group start on any row);
//   * few tiles are split along K over a cluster of 2 or 4 CTAs: with every rank's sums in its
//     shared memory, each reads its share of the tile out of all of them and adds in rank order
//     (16 x 8192 x 8192 20 us: 3 of launch and first loads, 10 of the weights' bytes).
//
// Tile schedule, tensor maps, bounded waits and the staged stores are those of gemm_kernel
// (gge_kernel.cuh).
#pragma once

#include "../gge_kernel.cuh"
#include "b128_launch.h"

namespace gge {
namespace b128 {

constexpr int kMaxStages = 16;
constexpr int kScaleSlots = 2;   // of the scale ring

template <int BN, int CG, bool BV>
struct GemmCfg {
  static constexpr bool kWide = BN == 256;             // the warps that hold sums finish the tile
  static constexpr int kTileM = kBM * CG;
  static constexpr int kBRows = BN / CG;
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = kBRows * kRowBytes;
  __device__ static __forceinline__ uint32_t a_bytes(const GemmParams& gp) { return kWide ? kABytes : gp.a_rows * kRowBytes; }
  __device__ static __forceinline__ uint32_t stage_bytes(const GemmParams& gp) { return a_bytes(gp) + kBBytes; }
  static constexpr int kBuffers = kWide ? 2 : 4;       // blocks' sums in tensor memory
  static constexpr int kTmemCols = kBuffers * BN;
  static constexpr int kScaleFloats = kBM + (BV ? (kWide ? 256 : 128) : 4);  // of a block
  static constexpr int kSlotBlocks = 8;                // a slot of the scale ring holds so many blocks'
  static constexpr int kSlotBytes = kSlotBlocks * kScaleFloats * 4;
  static constexpr int kHalf = BN / 2;                 // columns a holding thread has
  static constexpr int kSumsBytes = kWide ? 0 : kBM * BN * 4;
  static constexpr int kMmaWarp = 0, kLoadWarp = 1, kScaleWarp = 2;  // (and the one behind it)
  static constexpr int kFirstHold = 4, kHoldWarps = 8;
  static constexpr int kFirstFinish = 12, kFinishWarps = kWide ? 0 : 4;
  static constexpr int kStagingWarps = kWide ? kHoldWarps : kFinishWarps;
  static constexpr int kThreads = (kFirstFinish + kFinishWarps) * 32;
  // Registers of the warpgroups (setmaxnreg) that load and issue, hold sums, and finish tiles; a
  // block is launched with 168 a thread, or 128.
  static constexpr int kIssueRegs = 56, kHoldRegs = kWide ? 224 : 152, kFinishRegs = 152;
  static constexpr int kAllRegs = (kIssueRegs + 2 * kHoldRegs) * 128 + kFinishRegs * 32 * kFinishWarps;
  static_assert((BN == 256 && CG == 2) || ((BN == 128 || BN == 64) && CG == 1), "tile shapes");
  static_assert(kTmemCols <= 512, "tensor memory");
  static_assert(kAllRegs <= kThreads * (kWide ? 168 : 128), "registers");
};

// The control block's barriers and words, as offsets: one register finds them all.
enum : uint32_t {
  kFullBar = 0,                               // kMaxStages each
  kEmptyBar = kFullBar + 8 * kMaxStages,
  kSumsBar = kEmptyBar + 8 * kMaxStages,      // four buffers: a block's sums are there,
  kTakenBar = kSumsBar + 8 * 4,               // ... and have been taken
  kScaleBar = kTakenBar + 8 * 4,              // the scale ring's slots: filled,
  kUsedBar = kScaleBar + 8 * kScaleSlots,     // ... and used
  kTileBar = kUsedBar + 8 * kScaleSlots,      // a tile's sums are in shared memory,
  kFreeBar = kTileBar + 8,                    // ... and have been read
  kDrainBar = kFreeBar + 8,
  kTmemWord = kDrainBar + 8,
  kAbortWord = kTmemWord + 4,
  kCtrlBlock = 512                            // bytes, before the groups' tables
};
static_assert(kAbortWord + 4 <= kCtrlBlock, "control block");

// Bounded waits.  A block's buffers pass between the roles every few hundred cycles, so a wait
// starts with probes alone: reading the timer takes as long as most waits.
constexpr int kProbes = 64;

// ... of one thread (or of lanes that may part)
__device__ __forceinline__ bool wait_on(uint32_t bar, uint32_t parity, const Params& p, const Shared& sh, int32_t where,
                                        int32_t tile) {
#pragma unroll 1
  for (int i = 0; i < kProbes; ++i)
    if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    bool stop = *sh.abort != 0;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      record_status(p, DEV_TIMEOUT, where, tile);
      *sh.abort = 1;
      stop = true;
    }
    if (stop) return false;
  }
  return true;
}

// ... of a warp, without a call, so that its sums stay in their registers.  The answer is the
// same for all lanes.  (What is usual -- the phase is over -- has no branch to take: a taken one
// costs tens of cycles here, where the warps of a scheduler run different code.)
__device__ __forceinline__ bool wait_warp(uint32_t ctrl, uint32_t bar, uint32_t parity, const Params& p, int32_t where,
                                          int32_t tile) {
  if (__builtin_expect(__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity)), 1)) return true;
#pragma unroll 1
  for (int i = 0; i < kProbes; ++i)
    if (__all_sync(0xffffffffu, ptx::mbar_try_wait(bar, parity))) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    const bool now = ptx::mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, now)) return true;
    bool stop = ptx::ld_shared_u32(ctrl + kAbortWord) != 0u;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      record_status(p, DEV_TIMEOUT, where, tile);
      ptx::st_shared_u32(ctrl + kAbortWord, 1u);
      stop = true;
    }
    if (__any_sync(0xffffffffu, stop)) return false;
  }
}

// Is the phase over?  (Never suspends the thread.)
__device__ __forceinline__ bool probe(uint32_t bar, uint32_t parity) {
  uint32_t over;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(over)
      : "r"(bar), "r"(parity)
      : "memory");
  return over != 0u;
}

// threadIdx.x, read here (not kept in a register from one part of the kernel to another).
__device__ __forceinline__ int thread_now() {
  int tid;
  asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
  return tid;
}

// One arrival a warp.
__device__ __forceinline__ void arrive_one(uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar), "r"(threadIdx.x & 31)
      : "memory");
}
// ... at a barrier of any CTA of the cluster (nothing that the warp wrote is published).
__device__ __forceinline__ void arrive_one_remote(uint32_t cluster_bar) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.release.cta.shared::cluster.b64 _, [%0];\n\t}" ::"r"(cluster_bar), "r"(threadIdx.x & 31)
      : "memory");
}

// This CTA's blocks of K [k0, k1): all of them, or its share in a cluster split along K.
struct KSpan {
  int32_t k0, k1;
};
__device__ __forceinline__ KSpan k_span(const GemmParams& gp, uint32_t slice) {
  const int64_t k = gp.p.k_tiles;
  return KSpan{static_cast<int32_t>(slice * k / gp.splits), static_cast<int32_t>((slice + 1) * k / gp.splits)};
}

__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  return __uint_as_float(ptx::ld_shared_u32(addr));
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// ------------------------------------------------------------ loading and issuing

// A block's MMAs and the commits that hand its sums and its stage on; `next_full` and
// `next_empty` say whether the next block's stage and buffer are there.  One statement: a
// probe's answer takes longer than the MMAs take to issue, and the thread would wait for it
// before them.  (Probes at the top of the loop: 400 of its 710 cycles.)
#define GGE_B128_MMAS(CGN, COMMIT, MASK)                                                                           \
  asm volatile(                                                                                                   \
      "{\n\t.reg .pred f, e, k0, k1, k2, k3, d;\n\t.reg .b64 a, b;\n\t"                                               \
      "mbarrier.test_wait.parity.shared::cta.b64 f, [%2], %3;\n\t"                                                \
      "mbarrier.test_wait.parity.shared::cta.b64 e, [%4], %5;\n\t"                                                \
      "setp.lt.s32 k0, %10, 0;\n\tsetp.gt.s32 k1, %10, 1;\n\tsetp.gt.s32 k2, %10, 2;\n\tsetp.gt.s32 k3, %10, 3;\n\t"                      \
      "setp.ne.s32 d, %13, 0;\n\t"                                                                               \
      "tcgen05.mma.cta_group::" CGN ".kind::f8f6f4 [%6], %7, %8, %9, k0;\n\t"                                      \
      "add.s64 a, %7, 2;\n\tadd.s64 b, %8, 2;\n\t"                                                              \
      "@k1 tcgen05.mma.cta_group::" CGN ".kind::f8f6f4 [%6], a, b, %9, k1;\n\t"                                    \
      "add.s64 a, %7, 4;\n\tadd.s64 b, %8, 4;\n\t"                                                              \
      "@k2 tcgen05.mma.cta_group::" CGN ".kind::f8f6f4 [%6], a, b, %9, k2;\n\t"                                    \
      "add.s64 a, %7, 6;\n\tadd.s64 b, %8, 6;\n\t"                                                              \
      "@k3 tcgen05.mma.cta_group::" CGN ".kind::f8f6f4 [%6], a, b, %9, k3;\n\t"                                    \
      "@d " COMMIT " [%11]" MASK ";\n\t" COMMIT " [%12]" MASK ";\n\t"                                            \
      "selp.u32 %0, 1, 0, f;\n\tselp.u32 %1, 1, 0, e;\n\t}"                                                     \
      : "=r"(f), "=r"(e)                                                                                          \
      : "r"(next_full), "r"(full_phase), "r"(next_empty), "r"(empty_phase), "r"(d), "l"(adesc), "l"(bdesc),       \
        "r"(idesc), "r"(steps), "r"(tfull), "r"(empty), "r"(hand_on), "h"(static_cast<uint16_t>(0x3))               \
      : "memory")
struct Probed {
  bool full, empty;
};
template <int CG>
__device__ __forceinline__ Probed issue_block(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, int32_t steps,
                                              uint32_t tfull, uint32_t empty, int32_t hand_on, uint32_t next_full,
                                              uint32_t full_phase, uint32_t next_empty, uint32_t empty_phase) {
  uint32_t f, e;
  if constexpr (CG == 1)
    GGE_B128_MMAS("1", "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64", "");
  else
    GGE_B128_MMAS("2", "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64",
                  ", %14");
  return Probed{f != 0, e != 0};
}
#undef GGE_B128_MMAS

// Run by one thread.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void mma_role(const GemmParams& gp, const Shared& sh, uint32_t stage0, uint32_t tmem_base,
                                         const KSpan& ks, int32_t unit, int32_t units, int32_t num_tiles) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  int stage = 0, buf = 0;
  uint32_t phase = 0, buf_phase = 1;  // (the first pass over the buffers waits for nobody)
  Probed there{false, false};
  const int32_t hand_on = p.flags & FLAG_TEST_DROP_ACC_FULL ? 0 : 1;
  // (addresses in a descriptor are in 16 bytes; K advances by 32 bytes an MMA inside the swizzle)
  const uint64_t adesc = smem_desc(stage0, 16u, 1024u), bdesc = smem_desc(stage0 + Cfg::a_bytes(gp), 16u, 1024u);
  for (int32_t t = unit; t < num_tiles; t += units) {
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      const uint32_t empty = sh.empty + 8 * stage, tfull = sh.tfull + 8 * buf;
      if (__builtin_expect(!(there.full && there.empty), 0)) {
        if (!wait_on(sh.full + 8 * stage, phase, p, sh, 1, t)) return;
        if (!wait_on(sh.tempty + 8 * buf, buf_phase, p, sh, 2, t)) return;
      }
      ptx::tc_fence_after();
      const uint32_t step = static_cast<uint32_t>(stage) * (Cfg::stage_bytes(gp) / 16);
      const uint32_t d = tmem_base + buf * BN;
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      if (++buf == Cfg::kBuffers) { buf = 0; buf_phase ^= 1u; }
      there = issue_block<CG>(d, adesc + step, bdesc + step, p.idesc, min(4, (p.K - kt * kBlock + 31) / 32), tfull, empty,
                              hand_on, sh.full + 8 * stage, phase, sh.tempty + 8 * buf, buf_phase);
    }
  }
}

// Run by one thread.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void load_role(const GemmParams& gp, const Shared& sh, const CUtensorMap* tmA,
                                          const CUtensorMap* tmB, uint32_t stage0, uint32_t rank, const KSpan& ks,
                                          int32_t unit, int32_t units, int32_t num_tiles) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  int stage = 0;
  uint32_t phase = 0;
  for (int32_t t = unit; t < num_tiles; t += units) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    const int32_t row0 = tc.m_row0 + static_cast<int32_t>(rank) * kBM;
    const int32_t bn0 = tc.n0 + static_cast<int32_t>(rank) * Cfg::kBRows;
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      if (!wait_on(sh.empty + 8 * stage, phase ^ 1u, p, sh, 0, t)) return;
      const uint32_t full = sh.full + 8 * stage;
      if (CG == 1) ptx::mbar_arrive_expect_tx(full, Cfg::stage_bytes(gp));
      else if (rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * Cfg::stage_bytes(gp));
      const uint32_t bar = (CG == 1) ? full : ptx::mapa(full, 0);
      const uint32_t dst = stage0 + stage * Cfg::stage_bytes(gp);
      if (CG == 1) {
        ptx::tma_load_3d(dst, tmA, bar, kt * kBlock, row0, tc.a_batch);
        ptx::tma_load_3d(dst + Cfg::a_bytes(gp), tmB, bar, kt * kBlock, bn0, tc.b_batch);
      } else {
        ptx::tma_load_3d_pair(dst, tmA, bar, kt * kBlock, row0, tc.a_batch);
        ptx::tma_load_3d_pair(dst + Cfg::a_bytes(gp), tmB, bar, kt * kBlock, bn0, tc.b_batch);
      }
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
  }
}

// `n` scales (128 rows' or columns', one each) of a block on their way to shared memory, by one
// warp: four a lane, with one copy where they lie together on 16 bytes, else four.  What is not
// there becomes zero.  A block must not cost the warp more than a few instructions: addresses are
// worked out once a tile (once a block: 530 cycles, which bounded the whole product).
struct ScaleRow {
  const float* at[4];
  uint32_t bytes;   // together: how many there are.  Apart: a bit each
  bool together;

  __device__ __forceinline__ void init(const View& q, int64_t batch, int32_t first, int32_t end, int32_t k0) {
    const int lane = threadIdx.x & 31;
    const float* base = q.scales + batch * q.s_batch + k0 * q.s_col;
    together = q.shift == 0 && q.s_row == 1 && ((first | static_cast<int32_t>(q.s_col)) & 3) == 0 &&
               (reinterpret_cast<uintptr_t>(base) & 15u) == 0;
    if (together) {
      const int32_t row = first + 4 * lane;
      bytes = static_cast<uint32_t>(max(0, min(4, end - row))) * 4u;
      at[0] = bytes > 0u ? base + row : base;
    } else {
      bytes = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t row = first + lane + 32 * i;
        at[i] = row < end ? base + (row >> q.shift) * q.s_row : base;
        bytes |= row < end ? 1u << i : 0u;
      }
    }
  }
  // ... of one block; the next call takes the next one's.
  __device__ __forceinline__ void copy(uint32_t dst, int64_t s_col) {
    const int lane = threadIdx.x & 31;
    if (together) {
      ptx::cp_async_16(dst + 16 * lane, at[0], bytes);
      at[0] += s_col;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        cp_async_4(dst + 4 * (lane + 32 * i), at[i], (bytes >> i & 1u) != 0u);
        at[i] += s_col;
      }
    }
  }
};

// A slot of the scale ring holds, for each of its blocks, the CTA's 128 rows' scales, then the
// columns': one each (BV), or one for all.  Run by two warps, one for each part.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void scale_role(const GemmParams& gp, const Shared& sh, uint32_t ctrl, uint32_t rank,
                                           const KSpan& ks, int32_t unit, int32_t units, int32_t num_tiles, bool of_b) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  const View& q = of_b ? gp.b : gp.a;
  int slot = 0;
  uint32_t phase = 1;
  for (int32_t t = unit; t < num_tiles; t += units) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    ScaleRow row, more;  // (more: a wide tile's second 128 columns)
    if (!of_b) {
      row.init(q, tc.a_batch, tc.m_row0 + static_cast<int32_t>(rank) * kBM, p.num_groups > 0 ? tc.row_limit : p.M, ks.k0);
    } else if (BV) {
      row.init(q, tc.b_batch, tc.n0, min(p.N, tc.n0 + BN), ks.k0);
      if constexpr (Cfg::kWide) more.init(q, tc.b_batch, tc.n0 + 128, p.N, ks.k0);
    } else {
      const int32_t col = tc.n0 + (Cfg::kWide ? (threadIdx.x & 1) * 128 : 0);
      row.bytes = col < p.N ? 1u : 0u;
      row.at[0] = q.scale(col < p.N ? col : tc.n0, ks.k0, tc.b_batch);
    }
    for (int32_t kt = ks.k0; kt < ks.k1; kt += Cfg::kSlotBlocks) {
      if (!wait_on(ctrl + kUsedBar + 8 * slot, phase, p, sh, 10, t)) return;
      uint32_t dst = ctrl - (kScaleSlots - slot) * Cfg::kSlotBytes + (of_b ? 4 * kBM : 0);
      const int32_t end = min(kt + Cfg::kSlotBlocks, ks.k1);
#pragma unroll 1
      for (int32_t k = kt; k < end; ++k, dst += Cfg::kScaleFloats * 4) {
        if (BV || !of_b) {
          row.copy(dst, q.s_col);
          if constexpr (BV && Cfg::kWide) {
            if (of_b) more.copy(dst + 4 * 128, q.s_col);
          }
        } else {
          const int lane = threadIdx.x & 31;
          if (lane < (Cfg::kWide ? 2 : 1)) cp_async_4(dst + 4 * lane, row.at[0], row.bytes != 0u);
          row.at[0] += q.s_col;
        }
      }
      ptx::cp_async_mbar_arrive_noinc(ctrl + kScaleBar + 8 * slot);
      if (++slot == kScaleSlots) { slot = 0; phase ^= 1u; }
    }
  }
}

// ------------------------------------------------------------ the sums

// Add a chunk of 32 columns, scaled.  BV: the columns' scales lie at `sb`.
template <bool BV>
__device__ __forceinline__ void add_chunk(float2* acc, const uint32_t (&v)[32], float s, uint32_t sb) {
  const float2 s2 = make_float2(s, s);
  if constexpr (BV) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const uint4 w = ptx::ld_shared_v4(sb + 16 * q);
      const float2 lo = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
      const float2 hi = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
      const float2 t0 = make_float2(__uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]));
      const float2 t1 = make_float2(__uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]));
      acc[2 * q] = __ffma2_rn(t0, __fmul2_rn(lo, s2), acc[2 * q]);
      acc[2 * q + 1] = __ffma2_rn(t1, __fmul2_rn(hi, s2), acc[2 * q + 1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      acc[i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, acc[i]);
    }
  }
}

// Where a warp is in the rings.
struct Place {
  uint32_t blocks, slots;  // taken since the kernel's start
};

// A tile's blocks added to `acc`, its sums' columns from `half` of the tile on.  `idle`: none of
// the warp's rows is wanted (the buffers are only handed back).  False after a wait that ran out.
template <int BN, int CG, bool BV>
__device__ __forceinline__ bool add_blocks(const Params& p, uint32_t ctrl, uint32_t tmem, int half, int32_t blocks,
                                           int32_t t, bool idle, Place& at, float2 (&acc)[BN / 4]) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const uint32_t row = 4 * (threadIdx.x & 127);   // (a warpgroup's threads are a tile's rows)
  const uint32_t cols = 4 * (kBM + (BV ? half * Cfg::kHalf : Cfg::kWide ? half : 0));
  constexpr int kChunks = Cfg::kHalf / 32;
  constexpr uint32_t kMask = Cfg::kBuffers - 1, kShift = Cfg::kBuffers == 2 ? 1 : 2;
  uint32_t scales = 0u;
  float s = 0.f;
  bool there = false;
  const auto fetch = [&]() {
    s = ld_shared_f32(scales + row);
    if constexpr (!BV) s *= ld_shared_f32(scales + cols);
  };
  const auto leave_slot = [&]() {
    __syncwarp();
    arrive_one(ctrl + kUsedBar + 8 * (at.slots & 1u));
    ++at.slots;
  };
#pragma unroll 1
  for (int32_t n = 0; n < blocks; ++n) {
    if (n % Cfg::kSlotBlocks == 0) {
      if (n > 0) leave_slot();
      if (!wait_warp(ctrl, ctrl + kScaleBar + 8 * (at.slots & 1u), (at.slots >> 1) & 1u, p, 11, t)) return false;
      scales = ctrl - (kScaleSlots - (at.slots & 1u)) * Cfg::kSlotBytes;
      fetch();
    }
    if (!BV || !__all_sync(0xffffffffu, there))
      if (!wait_warp(ctrl, ctrl + kSumsBar + 8 * (at.blocks & kMask), (at.blocks >> kShift) & 1u, p, 3, t)) return false;
    ptx::tc_fence_after();
    const uint32_t from = tmem + (at.blocks & kMask) * BN;
    const uint32_t taken = CG == 1 ? ctrl + kTakenBar + 8 * (at.blocks & kMask) : ptx::mapa(ctrl + kTakenBar + 8 * (at.blocks & kMask), 0);
    ++at.blocks;
    const float mine = s;
    const uint32_t sb = scales + cols;
    scales += Cfg::kScaleFloats * 4;
    const auto hand_back = [&]() {
      ptx::tc_fence_before();
      if (CG == 1) arrive_one(taken);
      else arrive_one_remote(taken);
      if constexpr (BV) there = probe(ctrl + kSumsBar + 8 * (at.blocks & kMask), (at.blocks >> kShift) & 1u);
      fetch();  // (the next block's; behind a slot's last one it is not used)
    };
    if (idle) {
      hand_back();
    } else {
      // two chunks at a time, the second two's loads under the first two's additions
      uint32_t v[kChunks > 1 ? 2 : 1][32];
      ptx::tmem_ld_32x32b_x32(from, v[0]);
      if constexpr (kChunks > 1) ptx::tmem_ld_32x32b_x32(from + 32, v[1]);
#pragma unroll
      for (int c = 0; c < kChunks; c += 2) {
        ptx::tmem_wait_ld(v[0]);
        if constexpr (kChunks > 1) ptx::tmem_wait_ld(v[1]);
        if (c + 2 >= kChunks) hand_back();
        add_chunk<BV>(acc + c * 16, v[0], mine, sb + c * 128);
        if (c + 2 < kChunks) ptx::tmem_ld_32x32b_x32(from + (c + 2) * 32, v[0]);
        if constexpr (kChunks > 1) {
          add_chunk<BV>(acc + (c + 1) * 16, v[1], mine, sb + (c + 1) * 128);
          if (c + 2 < kChunks) ptx::tmem_ld_32x32b_x32(from + (c + 3) * 32, v[1]);
        }
      }
    }
  }
  if (blocks > 0) leave_slot();
  return true;
}

// Where piece q (four columns) of a row's sums lies: the pieces are XORed with the row, so that
// neighbouring rows' same piece falls into different banks.
template <int BN>
__device__ __forceinline__ uint32_t sums_at(uint32_t sums, int row, int q) {
  return sums + row * (BN * 4) + ((q ^ (row & 7)) << 4);
}

// ------------------------------------------------------------ the outputs

__device__ __forceinline__ bool has_c(const GemmParams& gp) { return gp.p.c != nullptr || gp.c8.codes != nullptr; }

// The raw bits of a lane's 32 columns of C (16 bits: 64 bytes, codes: 32); an fp32 C is read
// where it is used.
__device__ __forceinline__ void fetch_c(const GemmParams& gp, int32_t row, int32_t col0, int64_t batch, CRegs& c) {
  const Params& p = gp.p;
  if (gp.c8.codes != nullptr) {
    const uint2* at = reinterpret_cast<const uint2*>(gp.c8.codes + batch * gp.c8.batch + row * gp.c8.ld + col0);
    uint2 w[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col0 + 8 * i < p.N) w[i] = __ldg(at + i);
    c.w[0] = make_uint4(w[0].x, w[0].y, w[1].x, w[1].y);
    c.w[1] = make_uint4(w[2].x, w[2].y, w[3].x, w[3].y);
  } else if (p.c != nullptr && p.c_dtype != DT_F32) {
    const uint4* at = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.c) + batch * p.sbc + row * p.ldc + col0);
#pragma unroll
    for (int i = 0; i < 4; ++i) c.w[i] = col0 + 8 * i < p.N ? __ldg(at + i) : make_uint4(0u, 0u, 0u, 0u);
  }
}
// Eight of them (group g) as numbers.  `unit` is the codes' scale, `crow` an fp32 C's place (NULL
// for a row that is not there).
__device__ __forceinline__ void c_numbers8(const GemmParams& gp, const CRegs& c, float unit, const char* crow,
                                           int32_t col0, int g, float (&x)[8]) {
  const Params& p = gp.p;
  if (gp.c8.codes != nullptr) {
    const uint4 w = c.w[g >> 1];
    float2 f[4];
    values8_any(gp.c8.e5m2 != 0, g & 1 ? make_uint2(w.z, w.w) : make_uint2(w.x, w.y), unit, f);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = f[j].x, x[2 * j + 1] = f[j].y;
  } else if (p.c_dtype == DT_F32) {
    c_values8<DT_F32, false>(c, p, crow, col0, g, x);
  } else if (p.c_dtype == DT_BF16) {
    c_values8<DT_BF16, false>(c, p, nullptr, col0, g, x);
  } else {
    c_values8<DT_F16, false>(c, p, nullptr, col0, g, x);
  }
}

template <int ACT>
__device__ __forceinline__ void dact8_t(const float (&x)[8], float* v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= dact_one<ACT>(x[j]);
}
__device__ __forceinline__ void dact8(int act, const float (&x)[8], float* v) {
  switch (act) {
    case ACT_RELU: dact8_t<ACT_RELU>(x, v); break;
    case ACT_GELU_TANH: dact8_t<ACT_GELU_TANH>(x, v); break;
    case ACT_SILU: dact8_t<ACT_SILU>(x, v); break;
    default: dact8_t<ACT_RELU_SQ>(x, v); break;
  }
}

// A tile's place as a warp sees it.
struct Spot {
  int32_t row_base, rows_valid, col_base;
  int64_t batch;  // of C and the outputs
};

// 32 columns of a row's sums, from and back to shared memory.
template <int BN>
__device__ __forceinline__ void load32(uint32_t sums, int row, int c, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const uint4 w = ptx::ld_shared_v4(sums_at<BN>(sums, row, 8 * c + q));
    v[4 * q] = __uint_as_float(w.x), v[4 * q + 1] = __uint_as_float(w.y);
    v[4 * q + 2] = __uint_as_float(w.z), v[4 * q + 3] = __uint_as_float(w.w);
  }
}
template <int BN>
__device__ __forceinline__ void keep32(uint32_t sums, int row, int c, const float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 8; ++q)
    ptx::st_shared_v4(sums_at<BN>(sums, row, 8 * c + q),
                      make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                                 __float_as_uint(v[4 * q + 3])));
}

__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// ... of all ranks of a cluster that splits K, added in rank order.
template <int BN>
__device__ __forceinline__ void join32(uint32_t sums, int row, int c, int32_t splits, float (&v)[32]) {
#pragma unroll 1
  for (int32_t r = 0; r < splits; ++r) {
    const uint32_t from = ptx::mapa(sums, static_cast<uint32_t>(r));
    uint4 w[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) w[q] = ld_cluster_v4(sums_at<BN>(from, row, 8 * c + q));
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float f[4] = {__uint_as_float(w[q].x), __uint_as_float(w[q].y), __uint_as_float(w[q].z), __uint_as_float(w[q].w)};
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * q + j] = r == 0 ? f[j] : v[4 * q + j] + f[j];
    }
  }
}

// A warp's 32 rows of 128 codes (16-byte pieces XORed with the row) to whole lines of the output.
__device__ __forceinline__ void copy_codes_out(const GemmParams& gp, const View& q, const Spot& at, uint32_t stg) {
  const int lane = threadIdx.x & 31, piece = lane & 7;
  const int32_t n = gp.p.N - at.col_base - 16 * piece;  // (a multiple of 8)
  uint8_t* out = q.codes + at.batch * q.batch + at.row_base * q.ld + at.col_base + 16 * piece;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int r = 4 * j + (lane >> 3);
    const uint4 v = ptx::ld_shared_v4(stg + r * 128 + ((piece ^ (r & 7)) << 4));
    if (r >= at.rows_valid) continue;
    if (n >= 16) *reinterpret_cast<uint4*>(out + r * q.ld) = v;
    else if (n >= 8) *reinterpret_cast<uint2*>(out + r * q.ld) = make_uint2(v.x, v.y);
  }
  __syncwarp();  // the buffer is free again
}

// A warp's 32 rows of 8-bit output: the numbers that it keeps in shared memory, a block a row,
// quantised, through the warp's staging buffer to whole lines.
template <bool E5M2>
__device__ __forceinline__ void store_codes(const GemmParams& gp, const View& q, const Spot& at, uint32_t sums, int row,
                                            float top, uint32_t stg) {
  const int lane = threadIdx.x & 31;
  float factor;
  const float unit = block_scale<E5M2>(mx::abs_bits(top), factor);
  if (lane < at.rows_valid) *q.scale(at.row_base + lane, at.col_base >> 7, at.batch) = unit;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    float v[32];
    load32<kBlock>(sums, row, c, v);
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] = pack4<E5M2>(v[4 * j] * factor, v[4 * j + 1] * factor, v[4 * j + 2] * factor, v[4 * j + 3] * factor);
    ptx::st_shared_v4(stg + lane * 128 + (((2 * c) ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
    ptx::st_shared_v4(stg + lane * 128 + (((2 * c + 1) ^ (lane & 7)) << 4), make_uint4(w[4], w[5], w[6], w[7]));
  }
  __syncwarp();
  copy_codes_out(gp, q, at, stg);
}
__device__ __forceinline__ void store_codes_any(const GemmParams& gp, const View& q, const Spot& at, uint32_t sums,
                                                int row, float top, uint32_t stg) {
  if (q.e5m2) store_codes<true>(gp, q, at, sums, row, top, stg);
  else store_codes<false>(gp, q, at, sums, row, top, stg);
}

// 32 columns of a 16- or 32-bit output.
__device__ __forceinline__ void store32(uint32_t stg, const float (&v)[32], int dtype, void* out, int64_t ld, int64_t sb,
                                        const Spot& at, int32_t col0, int32_t N) {
  store_chunk_staged(stg, v, dtype,
                     static_cast<char*>(out) + (at.batch * sb + at.row_base * ld + col0) * dtype_bytes(dtype),
                     ld * dtype_bytes(dtype), at.rows_valid, min(32, N - col0), false);
}
// The largest |value| so far (columns past N do not count; N is a multiple of 8).
__device__ __forceinline__ float most32(float top, const float (&v)[32], int32_t left) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if ((j & ~7) < left) top = mx::max_abs(top, v[j]);
  return top;
}

// D and PostAct of a warp's 32 rows from the sums in shared memory, where the numbers of an 8-bit
// output wait for their scale.  The tile's chunks of 32 columns first,
// first + step, ... below `last` are this warp's.  Warp-collective.
template <int BN>
__device__ __forceinline__ void finish(const GemmParams& gp, const Spot& at, uint32_t sums, uint32_t stg, int32_t splits,
                                       int first, int last, int step) {
  const Params& p = gp.p;
  const int lane = threadIdx.x & 31, tile_row = threadIdx.x & 127;
  const float alpha = p.dact ? 1.f : (p.alpha_dev ? *p.alpha_dev : p.alpha);
  const float beta = p.beta_dev ? *p.beta_dev : p.beta;
  const int32_t row = at.row_base + lane;
  const bool there = lane < at.rows_valid;
  const bool d8 = gp.d8.codes != nullptr, p8 = gp.p8.codes != nullptr;
  const bool reads_c = has_c(gp), has_p = p8 || p.post != nullptr;
  float top = 0.f;
  // One pass makes both outputs, but for two in 8 bits: shared memory holds one's numbers.
#pragma unroll 1
  for (int pass = 0; pass < (d8 && p8 ? 2 : 1); ++pass) {
    const bool does_p = has_p && (pass == 1 || !(d8 && p8));
    CRegs c_raw = {};  // (the next chunk's come while this one is stored)
    const bool c_here = reads_c && (pass == 0 || p.dact) && there;
    if (c_here && at.col_base + 32 * first < p.N) fetch_c(gp, row, at.col_base + 32 * first, at.batch, c_raw);
#pragma unroll 1
    for (int c = first; c < last; c += step) {
      const int32_t col0 = at.col_base + 32 * c, left = p.N - col0;
      if (left <= 0) break;
      float v[32];
      if (splits > 1 && pass == 0) join32<BN>(sums, tile_row, c, splits, v);
      else load32<BN>(sums, tile_row, c, v);
      const CRegs now = c_raw;
      if (c_here && c + step < last && left > 32 * step) fetch_c(gp, row, col0 + 32 * step, at.batch, c_raw);
      const float unit = c_here && gp.c8.codes != nullptr ? *gp.c8.scale(row, col0 >> 7, at.batch) : 0.f;
      const char* crow = c_here && gp.c8.codes == nullptr && p.c_dtype == DT_F32
                             ? reinterpret_cast<const char*>(static_cast<const float*>(p.c) + at.batch * p.sbc +
                                                             row * p.ldc + col0)
                             : nullptr;
      if (pass == 0) {
        if (reads_c) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[8];
            c_numbers8(gp, now, unit, crow, col0, g, x);
            if (p.dact) {
              dact8(p.act, x, v + 8 * g);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) v[8 * g + j] = fmaf(beta, x[j], v[8 * g + j] * alpha);
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= alpha;
        }
        if (p.d != nullptr) store32(stg, v, p.d_dtype, p.d, p.ldd, p.sbd, at, col0, p.N);
        if (d8) {
          top = most32(top, v, left);
          keep32<BN>(sums, tile_row, c, v);
        }
      }
      if (does_p) {
        if (p.dact) {
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float x[8];
            c_numbers8(gp, now, unit, crow, col0, g, x);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[8 * g + j] = x[j];
          }
        }
        act_chunk(p.act, v);
        if (p.post != nullptr) store32(stg, v, p.p_dtype, p.post, p.ldp, p.sbp, at, col0, p.N);
        if (p8) {
          top = most32(top, v, left);
          keep32<BN>(sums, tile_row, c, v);
        }
      }
    }
    if constexpr (BN == kBlock) {
      if (d8 && pass == 0) store_codes_any(gp, gp.d8, at, sums, tile_row, top, stg);
      else if (p8) store_codes_any(gp, gp.p8, at, sums, tile_row, top, stg);
      top = 0.f;
    }
  }
}

// The same for a wide tile's thread, whose 128 columns are in registers.  It walks them in chunks
// of 32, always the first 32 of the sums, which then move round by that many: the code of a
// chunk is there once, and the sums stay in registers (walked by an index they would not).
__device__ __forceinline__ void move_round(float2 (&acc)[64]) {
  float2 first[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) first[i] = acc[i];
#pragma unroll
  for (int i = 0; i < 48; ++i) acc[i] = acc[i + 16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[48 + i] = first[i];
}

__device__ __forceinline__ void store32_pairs(uint32_t stg, const float2* v, int dtype, void* out, int64_t ld, int64_t sb,
                                              const Spot& at, int32_t col0, int32_t N) {
  // (opaque: the staging addresses are not kept in registers from chunk to chunk)
  asm volatile("" : "+r"(stg));
  float x[32];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[2 * j] = v[j].x, x[2 * j + 1] = v[j].y;
  store32(stg, x, dtype, out, ld, sb, at, col0, N);
}

// The same by TMA, so that the warp goes on with the next tile while they leave
// (4096^3 with two outputs 83 -> 78 us, 8192^3 387 -> 381).  Chunk c of a 16-bit output takes
// the buffer c % 3 of the warp's three, the codes of 32 rows the first two; what uses the buffers
// otherwise drains them first.  Warp-collective.
__device__ __forceinline__ void drain_stores() {
  if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  __syncwarp();
}
__device__ __forceinline__ void send_box(const CUtensorMap* map, uint32_t stg, int32_t col, const Spot& at) {
  ptx::fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(col),
                 "r"(at.row_base), "r"(static_cast<int32_t>(at.batch)), "r"(stg)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  }
}
__device__ __forceinline__ void store32_tma(const CUtensorMap* map, uint32_t stg, int c, const float2* v, int dtype,
                                            const Spot& at) {
  asm volatile("" : "+r"(stg));
  const int lane = threadIdx.x & 31;
  if (c == 0) {
    drain_stores();
  } else if (c == 3) {
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory");
    __syncwarp();
  }
  stg += (c % 3) * 2048;
  const bool bf16 = dtype == DT_BF16;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16 ? pack2<true>(v[4 * q + i].x, v[4 * q + i].y) : pack2<false>(v[4 * q + i].x, v[4 * q + i].y);
    ptx::st_shared_v4(stg + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
  send_box(map, stg, at.col_base + 32 * c, at);
}

// (map: not NULL where they leave by TMA)
template <bool E5M2>
__device__ __forceinline__ void store_codes_held(const GemmParams& gp, const View& q, const CUtensorMap* map,
                                                 const Spot& at, const float2 (&acc)[64], float top, uint32_t stg) {
  asm volatile("" : "+r"(stg));
  const int lane = threadIdx.x & 31;
  float factor;
  const float unit = block_scale<E5M2>(mx::abs_bits(top), factor);
  if (lane < at.rows_valid) *q.scale(at.row_base + lane, at.col_base >> 7, at.batch) = unit;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = __fmul2_rn(acc[8 * i + 2 * j], make_float2(factor, factor));
      const float2 b = __fmul2_rn(acc[8 * i + 2 * j + 1], make_float2(factor, factor));
      w[j] = pack4<E5M2>(a.x, a.y, b.x, b.y);
    }
    ptx::st_shared_v4(stg + lane * 128 + ((i ^ (lane & 7)) << 4), make_uint4(w[0], w[1], w[2], w[3]));
  }
  if (map == nullptr) {
    __syncwarp();
    copy_codes_out(gp, q, at, stg);
  } else {
    send_box(map, stg, at.col_base, at);
  }
}

template <int ACT>
__device__ __forceinline__ void act_held_t(float2 (&acc)[64]) {
#pragma unroll
  for (int j = 0; j < 64; ++j) acc[j] = make_float2(act_one<ACT>(acc[j].x), act_one<ACT>(acc[j].y));
}
__device__ __forceinline__ void act_held(int act, float2 (&acc)[64]) {
  switch (act) {
    case ACT_RELU: act_held_t<ACT_RELU>(acc); break;
    case ACT_GELU_TANH: act_held_t<ACT_GELU_TANH>(acc); break;
    case ACT_SILU: act_held_t<ACT_SILU>(acc); break;
    case ACT_RELU_SQ: act_held_t<ACT_RELU_SQ>(acc); break;
    default: break;
  }
}

__device__ __forceinline__ void finish_held(const GemmParams& gp, const CUtensorMap* tmD, const CUtensorMap* tmP,
                                            const Spot& at, float2 (&acc)[64], uint32_t stg) {
  const Params& p = gp.p;
  const float alpha = p.dact ? 1.f : (p.alpha_dev ? *p.alpha_dev : p.alpha);
  // (a group's last rows, by themselves, end before the box)
  const int tma = at.rows_valid == 32 ? gp.by_tma : 0;
  if (gp.by_tma != 0 && tma == 0) drain_stores();
  if (!has_c(gp) && p.post == nullptr && gp.d8.codes == nullptr && gp.p8.codes == nullptr) {  // D alone
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (at.col_base + 32 * c >= p.N) break;
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[16 * c + j] = __fmul2_rn(acc[16 * c + j], make_float2(alpha, alpha));
      if (tma & 1) store32_tma(tmD, stg, c, acc + 16 * c, p.d_dtype, at);
      else store32_pairs(stg, acc + 16 * c, p.d_dtype, p.d, p.ldd, p.sbd, at, at.col_base + 32 * c, p.N);
    }
    return;
  }
  const float beta = p.beta_dev ? *p.beta_dev : p.beta;
  const int lane = threadIdx.x & 31;
  const int32_t row = at.row_base + lane;
  const bool there = lane < at.rows_valid;
  // pass 0: D; pass 1: PostAct
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    const View& q = pass == 0 ? gp.d8 : gp.p8;
    void* out = pass == 0 ? p.d : p.post;
    if (pass == 1 && out == nullptr && q.codes == nullptr) break;
    const bool reads_c = has_c(gp) && (pass == 0 || p.dact);
    if (pass == 1 && !reads_c) act_held(p.act, acc);
    if (!reads_c) {  // all written out: moving the sums round costs 1300 cycles a pass
      if (pass == 0) {
#pragma unroll
        for (int j = 0; j < 64; ++j) acc[j] = __fmul2_rn(acc[j], make_float2(alpha, alpha));
      }
      if (out != nullptr) {
        if (gp.by_tma != 0 && !(tma & (1 << pass))) drain_stores();
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (at.col_base + 32 * c < p.N) {
            if (tma & (1 << pass)) store32_tma(pass == 0 ? tmD : tmP, stg, c, acc + 16 * c, pass == 0 ? p.d_dtype : p.p_dtype, at);
            else if (pass == 0) store32_pairs(stg, acc + 16 * c, p.d_dtype, p.d, p.ldd, p.sbd, at, at.col_base + 32 * c, p.N);
            else store32_pairs(stg, acc + 16 * c, p.p_dtype, p.post, p.ldp, p.sbp, at, at.col_base + 32 * c, p.N);
          }
      }
      if (q.codes != nullptr) {
        const CUtensorMap* map = tma & (4 << pass) ? (pass == 0 ? tmD : tmP) : nullptr;
        if (gp.by_tma != 0) drain_stores();
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 64; ++j) top = mx::max_abs(mx::max_abs(top, acc[j].x), acc[j].y);
        if (q.e5m2) store_codes_held<true>(gp, q, map, at, acc, top, stg);
        else store_codes_held<false>(gp, q, map, at, acc, top, stg);
      }
      continue;
    }
    float top = 0.f;
    CRegs c_raw = {};  // (the next chunk's come while this one is stored)
    if (reads_c && there && at.col_base < p.N) fetch_c(gp, row, at.col_base, at.batch, c_raw);
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
      const int32_t col0 = at.col_base + 32 * c;
      {
        const bool here = there && col0 < p.N;
        const float unit = gp.c8.codes != nullptr && here ? *gp.c8.scale(row, col0 >> 7, at.batch) : 0.f;
        const char* crow = gp.c8.codes == nullptr && p.c_dtype == DT_F32 && here
                               ? reinterpret_cast<const char*>(static_cast<const float*>(p.c) + at.batch * p.sbc +
                                                               row * p.ldc + col0)
                               : nullptr;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[8], v[8];
          c_numbers8(gp, c_raw, unit, crow, col0, g, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[2 * j] = acc[4 * g + j].x, v[2 * j + 1] = acc[4 * g + j].y;
          if (p.dact && pass == 0) {
            dact8(p.act, x, v);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = p.dact ? x[j] : fmaf(beta, x[j], v[j] * alpha);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[4 * g + j] = make_float2(v[2 * j], v[2 * j + 1]);
        }
        if (here && c + 1 < 4 && col0 + 32 < p.N) fetch_c(gp, row, col0 + 32, at.batch, c_raw);
        if (col0 >= p.N) {  // (columns past N stay zero: an 8-bit PostAct takes its scale of all 128)
#pragma unroll
          for (int j = 0; j < 16; ++j) acc[j] = make_float2(0.f, 0.f);
        }
      }
      if (pass == 1) {
        float v[32];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[2 * j] = acc[j].x, v[2 * j + 1] = acc[j].y;
        act_chunk(p.act, v);
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = make_float2(v[2 * j], v[2 * j + 1]);
      }
      if (q.codes != nullptr) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (col0 + (2 * j & ~7) < p.N) top = mx::max_abs(mx::max_abs(top, acc[j].x), acc[j].y);
      }
      if (out != nullptr && col0 < p.N) {
        if (pass == 0) store32_pairs(stg, acc, p.d_dtype, p.d, p.ldd, p.sbd, at, col0, p.N);
        else store32_pairs(stg, acc, p.p_dtype, p.post, p.ldp, p.sbp, at, col0, p.N);
      }
      move_round(acc);
    }
    if (q.codes != nullptr && at.col_base < p.N) {
      const CUtensorMap* const map = nullptr;
      if (q.e5m2) store_codes_held<true>(gp, q, map, at, acc, top, stg);
      else store_codes_held<false>(gp, q, map, at, acc, top, stg);
    }
  }
}

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// This CTA's part: its unit of tiles (a CTA, a pair, or a cluster that splits K), its rank in a
// pair, its slice of K.
struct Part {
  int32_t unit, units;
  uint32_t rank, slice;
};
// Where things lie in shared memory:
//   stages | a tile's sums | output staging | scale ring | control | groups
// Each role works its addresses out anew (the base is opaque to the compiler), so that none is
// kept in a register, or spilled, through the other roles.
struct Memory {
  Shared sh;
  uint32_t stages, sums, out_stage, ctrl;
  uint32_t* tmem_slot;
  int32_t *abort_flag, *prefix, *cu;
};
template <int BN, int CG, bool BV>
__device__ __forceinline__ Memory memory(const GemmParams& gp) {
  using Cfg = GemmCfg<BN, CG, BV>;
  extern __shared__ uint8_t smem_raw[];
  uint32_t raw = ptx::smem_addr(smem_raw);
  asm volatile("" : "+r"(raw));
  const uint32_t base = (raw + 1023u) & ~1023u;
  Memory m = {};
  m.stages = base;
  m.sums = base + gp.p.stages * Cfg::stage_bytes(gp);
  m.out_stage = m.sums + Cfg::kSumsBytes;
  // (right behind the scale ring)
  m.ctrl = m.out_stage + Cfg::kStagingWarps * gp.p.out_stage_bytes + kScaleSlots * Cfg::kSlotBytes;
  uint8_t* ctrl = static_cast<uint8_t*>(__cvta_shared_to_generic(m.ctrl));
  m.sh.full = m.ctrl + kFullBar;
  m.sh.empty = m.ctrl + kEmptyBar;
  m.sh.tfull = m.ctrl + kSumsBar;
  m.sh.tempty = m.ctrl + kTakenBar;
  m.tmem_slot = reinterpret_cast<uint32_t*>(ctrl + kTmemWord);
  m.abort_flag = reinterpret_cast<int32_t*>(ctrl + kAbortWord);
  m.prefix = reinterpret_cast<int32_t*>(ctrl + kCtrlBlock);
  m.cu = m.prefix + (kMaxGroups + 1);
  m.sh.abort = m.abort_flag;
  m.sh.prefix = m.prefix;
  m.sh.cu = m.cu;
  return m;
}

template <int CG>
__device__ __forceinline__ Part part(const GemmParams& gp) {
  const uint32_t crank = (CG == 2 || gp.splits > 1) ? ptx::cluster_ctarank() : 0u;
  int32_t cta = static_cast<int32_t>(blockIdx.x), ctas = CG == 2 ? 2 : gp.splits;
  asm volatile("" : "+r"(cta), "+r"(ctas));  // (opaque, as in memory(): quotients are not kept from role to role)
  return Part{cta / ctas, static_cast<int32_t>(gridDim.x) / ctas, CG == 2 ? crank : 0u, CG == 2 ? 0u : crank};
}
__device__ __forceinline__ int32_t tiles_of(const GemmParams& gp, const Memory& m) {
  return gp.p.num_groups > 0 ? m.prefix[gp.p.num_groups] : gp.p.num_tiles;
}

// A warp's rows of tile t.
template <int BN, int CG, bool BV>
__device__ __forceinline__ Spot spot_of(const Params& p, const Memory& m, const Part& me, int32_t t, int quad) {
  const TileCoord tc = tile_coord<BN, GemmCfg<BN, CG, BV>::kTileM>(t, p, m.sh);
  Spot s;
  s.row_base = tc.m_row0 + static_cast<int32_t>(me.rank) * kBM + quad * 32;
  s.rows_valid = min(32, tc.row_limit - s.row_base);
  s.col_base = tc.n0;
  s.batch = p.num_groups > 0 ? 0 : tc.batch;
  return s;
}

// The warps that hold the sums while K runs.  (Where they finish the tile themselves, what that
// needs is worked out after the main loop, whose registers are the sums'.)
template <int BN, int CG, bool BV>
__device__ __forceinline__ void hold_role(const GemmParams& gp, const CUtensorMap* tmD, const CUtensorMap* tmP) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  const int quad = (threadIdx.x >> 5) & 3, half = (threadIdx.x >> 7) - 1;
  Place at{0u, 0u};
  uint32_t free_phase = 1u;
#pragma unroll 1
  for (int32_t i = 0;; ++i) {
    float2 acc[Cfg::kHalf / 2];
    int32_t t;
    {
      const Memory m = memory<BN, CG, BV>(gp);
      const Part me = part<CG>(gp);
      t = me.unit + i * me.units;
      if (t >= tiles_of(gp, m)) return;
      const bool idle = spot_of<BN, CG, BV>(p, m, me, t, quad).rows_valid <= 0;
      const KSpan ks = k_span(gp, me.slice);
      const uint32_t tmem = *m.tmem_slot + (static_cast<uint32_t>(quad * 32) << 16) + half * Cfg::kHalf;
#pragma unroll
      for (int j = 0; j < Cfg::kHalf / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      if (!add_blocks<BN, CG, BV>(p, m.ctrl, tmem, half, ks.k1 - ks.k0, t, idle, at, acc)) return;
    }
    const Memory m = memory<BN, CG, BV>(gp);
    if constexpr (Cfg::kWide) {
      Spot spot = spot_of<BN, CG, BV>(p, m, part<CG>(gp), t, quad);
      spot.col_base += half * Cfg::kHalf;
      if (spot.rows_valid > 0 && spot.col_base < p.N)
        finish_held(gp, tmD, tmP, spot, acc, m.out_stage + (threadIdx.x / 32 - Cfg::kFirstHold) * p.out_stage_bytes);
    } else {
      if (!wait_warp(m.ctrl, m.ctrl + kFreeBar, free_phase, p, 12, t)) return;
      free_phase ^= 1u;
#pragma unroll
      for (int q = 0; q < Cfg::kHalf / 4; ++q)
        ptx::st_shared_v4(sums_at<BN>(m.sums, threadIdx.x & 127, half * (Cfg::kHalf / 4) + q),
                          make_uint4(__float_as_uint(acc[2 * q].x), __float_as_uint(acc[2 * q].y),
                                     __float_as_uint(acc[2 * q + 1].x), __float_as_uint(acc[2 * q + 1].y)));
      __syncwarp();
      arrive_one(m.ctrl + kTileBar);
    }
  }
}

// The warps that turn a tile's sums into outputs.
// `who`: 0 for those that do nothing else; 1 and 2 for the holding warpgroups, which join them for
// the CTA's last tile (every third chunk each; staging where the stages were).
template <int BN, int CG, bool BV>
__device__ __forceinline__ void finish_role(const GemmParams& gp, int who) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  const Memory m = memory<BN, CG, BV>(gp);
  const Part me = part<CG>(gp);
  const int quad = (threadIdx.x >> 5) & 3;
  const int32_t num_tiles = tiles_of(gp, m);
  const int32_t splits = CG == 1 ? gp.splits : 1;
  const bool codes = gp.d8.codes != nullptr || gp.p8.codes != nullptr;
  const bool shared = !codes && 8 * p.out_stage_bytes <= p.stages * static_cast<int>(Cfg::stage_bytes(gp));
  const uint32_t stg =
      who == 0 ? m.out_stage + quad * p.out_stage_bytes : m.stages + (4 * who - 4 + quad) * p.out_stage_bytes;
  uint32_t phase = 0u;
  int32_t t = me.unit;
  if (splits > 1) {  // (one tile a cluster)
    cluster_arrive();
    cluster_wait();  // every rank's sums are in its shared memory
    if (*m.abort_flag) return;
  }
  if (who > 0) {
    if (!shared || t >= num_tiles) return;
    const int32_t before = (num_tiles - 1 - t) / me.units;  // this CTA's other tiles
    t += before * me.units;
    phase = static_cast<uint32_t>(before) & 1u;
  }
#pragma unroll 1
  for (; t < num_tiles; t += me.units) {
    const Spot spot = spot_of<BN, CG, BV>(p, m, me, t, quad);
    int first = 0, last = BN / 32;
    if (splits == 1) {
      if (!wait_warp(m.ctrl, m.ctrl + kTileBar, phase, p, 13, t)) return;
      phase ^= 1u;
    } else if (!codes) {  // a share of the columns, or, where a row's block has to stay together, of the rows
      first = static_cast<int>(me.slice) * (BN / 32) / splits;
      last = static_cast<int>(me.slice + 1) * (BN / 32) / splits;
    } else if (static_cast<uint32_t>(quad * splits) / 4 != me.slice) {
      return;
    }
    const bool three = shared && t + me.units >= num_tiles;
    if (spot.rows_valid > 0)
      finish<BN>(gp, spot, m.sums, stg, splits, three ? first + who : first, last, three ? 3 : 1);
    __syncwarp();
    if (who == 0) arrive_one(m.ctrl + kFreeBar);
  }
}

template <int BN, int CG, bool BV>
__global__ void __launch_bounds__(GemmCfg<BN, CG, BV>::kThreads, 1)
    b128_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmD, const __grid_constant__ CUtensorMap tmP,
                     const __grid_constant__ GemmParams gp) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  ptx::griddep_launch_dependents();
  Memory m = memory<BN, CG, BV>(gp);

  const int tid = thread_now(), warp = tid >> 5, lane = tid & 31;
  const int S = p.stages;
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(m.sh.full + 8 * s, 1);
      ptx::mbar_init(m.sh.empty + 8 * s, 1);
    }
    for (int b = 0; b < Cfg::kBuffers; ++b) {
      ptx::mbar_init(m.sh.tfull + 8 * b, 1);
      ptx::mbar_init(m.sh.tempty + 8 * b, Cfg::kHoldWarps * CG);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      ptx::mbar_init(m.ctrl + kScaleBar + 8 * s, 64);
      ptx::mbar_init(m.ctrl + kUsedBar + 8 * s, Cfg::kHoldWarps);
    }
    ptx::mbar_init(m.ctrl + kTileBar, Cfg::kHoldWarps);
    ptx::mbar_init(m.ctrl + kFreeBar, 4);
    ptx::mbar_init((m.ctrl + kDrainBar), 1);
    *m.abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == Cfg::kLoadWarp && lane == 0 && p.k_tiles > 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == Cfg::kMmaWarp) {
    if (CG == 1) {
      ptx::tmem_alloc(ptx::smem_addr(m.tmem_slot), Cfg::kTmemCols);
      ptx::tmem_relinquish();
    } else {
      ptx::tmem_alloc_pair(ptx::smem_addr(m.tmem_slot), Cfg::kTmemCols);
      ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
  }
  ptx::griddep_wait();
  // grouped rows: the offsets, and the tiles before each group
  if (p.num_groups > 0 && warp == 0) take_groups<Cfg::kTileM>(p, m.prefix, m.cu);
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  ptx::tc_fence_after();
  if (warp >= Cfg::kFirstHold) {
    static_assert(Cfg::kWide || Cfg::kHoldRegs == Cfg::kFinishRegs, "one share for both");
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kHoldRegs));
    if constexpr (Cfg::kWide) {
      hold_role<BN, CG, BV>(gp, &tmD, &tmP);
      if ((threadIdx.x & 31) == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    } else {
      if (warp < Cfg::kFirstFinish) hold_role<BN, CG, BV>(gp, &tmD, &tmP);
      finish_role<BN, CG, BV>(gp, warp < Cfg::kFirstFinish ? (warp - Cfg::kFirstHold) / 4 + 1 : 0);
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kIssueRegs));
    const Memory m = memory<BN, CG, BV>(gp);
    const Part me = part<CG>(gp);
    const KSpan ks = k_span(gp, me.slice);
    if (warp == Cfg::kMmaWarp) {
      if (me.rank == 0 && ptx::elect_one())
        mma_role<BN, CG, BV>(gp, m.sh, m.stages, *m.tmem_slot, ks, me.unit, me.units, tiles_of(gp, m));
    } else if (warp == Cfg::kLoadWarp) {
      if (ptx::elect_one())
        load_role<BN, CG, BV>(gp, m.sh, &tmA, &tmB, m.stages, me.rank, ks, me.unit, me.units, tiles_of(gp, m));
    } else {
      scale_role<BN, CG, BV>(gp, m.sh, m.ctrl, me.rank, ks, me.unit, me.units, tiles_of(gp, m),
                             warp != Cfg::kScaleWarp);
    }
    __syncwarp();
  }
  // (worked out again: nothing is kept in registers over the main loop)
  const int last_warp = thread_now() >> 5;
  if (CG == 1 && gp.splits > 1) {
    // (the others have waited for the sums of all ranks)
    if (last_warp < Cfg::kFirstHold) {
      cluster_arrive();
      cluster_wait();
    }
    cluster_arrive();
    cluster_wait();  // nobody reads this CTA's sums any more
  }

  __syncthreads();
  m = memory<BN, CG, BV>(gp);
  // Every MMA this CTA issued has finished before TMEM is freed: its sums' holders have waited
  // for the last block's, unless a wait ran out.
  if (*m.abort_flag && last_warp == Cfg::kMmaWarp && part<CG>(gp).rank == 0) {
    if (ptx::elect_one()) {
      if (CG == 1) ptx::mma_commit((m.ctrl + kDrainBar));
      else ptx::mma_commit_pair((m.ctrl + kDrainBar), 0x1);
    }
    __syncwarp();
    wait_on(m.ctrl + kDrainBar, 0, p, m.sh, 6, -1);
  }
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  if (*m.abort_flag) {
    // let copies and MMAs that were in flight land before the memory goes away
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  if (last_warp == Cfg::kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    if (CG == 1) ptx::tmem_dealloc(*m.tmem_slot, Cfg::kTmemCols);
    else ptx::tmem_dealloc_pair(*m.tmem_slot, Cfg::kTmemCols);
  }
}

// ------------------------------------------------------------ launches

template <int BN, int CG, bool BV>
cudaLaunchConfig_t gemm_config(int grid, size_t smem, int cluster, cudaStream_t stream, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(GemmCfg<BN, CG, BV>::kThreads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 1;
  if (cluster > 1) {
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cfg;
}

template <int BN, int CG, bool BV>
cudaError_t launch_one(const GemmMaps& maps, const GemmParams& gp, const LaunchShape& shape, cudaStream_t stream) {
  const cudaError_t e = allow_smem<b128_gemm_kernel<BN, CG, BV>>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gemm_config<BN, CG, BV>(shape.grid, shape.smem, shape.cluster, stream, attr);
  return cudaLaunchKernelEx(&cfg, b128_gemm_kernel<BN, CG, BV>, maps.a, maps.b, maps.d, maps.post, gp);
}

// (Registers leave room for one CTA an SM, so tensor memory needs no count of its own.  The
// warpgroups' shares must add up to what a block is launched with: setmaxnreg would wait for
// the rest forever.)
template <int BN, int CG, bool BV>
int units_one(size_t smem, int cluster) {
  using Cfg = GemmCfg<BN, CG, BV>;
  cudaFuncAttributes fa = {};
  if (cudaFuncGetAttributes(&fa, b128_gemm_kernel<BN, CG, BV>) != cudaSuccess) return -1;
  if (fa.numRegs * Cfg::kThreads < Cfg::kAllRegs) return -1;
  if (allow_smem<b128_gemm_kernel<BN, CG, BV>>() != cudaSuccess) return -1;
  if (cluster == 1) {
    int per_sm = 0, dev = 0, sms = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, b128_gemm_kernel<BN, CG, BV>, Cfg::kThreads, smem) !=
            cudaSuccess ||
        cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return -1;
    return per_sm * sms;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = gemm_config<BN, CG, BV>(cluster * 64, smem, cluster, nullptr, attr);
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, b128_gemm_kernel<BN, CG, BV>, &cfg) != cudaSuccess) return -1;
  return n;
}

template <int BN, int CG>
cudaError_t launch_tile(const GemmMaps& maps, const GemmParams& gp, const LaunchShape& shape, cudaStream_t stream) {
  return gp.b_rows_one ? launch_one<BN, CG, true>(maps, gp, shape, stream)
                       : launch_one<BN, CG, false>(maps, gp, shape, stream);
}
template <int BN, int CG>
int units_tile(bool b_rows_one, size_t smem, int cluster) {
  return b_rows_one ? units_one<BN, CG, true>(smem, cluster) : units_one<BN, CG, false>(smem, cluster);
}

#define GGE_B128_INSTANTIATE(BN, CG)                                                                     \
  template cudaError_t launch_tile<BN, CG>(const GemmMaps&, const GemmParams&, const LaunchShape&, cudaStream_t); \
  template int units_tile<BN, CG>(bool, size_t, int);

}  // namespace b128
}  // namespace gge
