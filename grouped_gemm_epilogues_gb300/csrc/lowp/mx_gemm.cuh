// Product of two microscaled matrices on the 5th-generation tensor core:
//
//   D       = alpha * sum_k (a_k sa_k) (b_k sb_k) + beta * C
//   PostAct = act(same value, before rounding)
//
// with 8-bit (e4m3) or 4-bit (e2m1) codes and one scale per 32 (16) values of
// K.  tcgen05.mma.block_scale multiplies codes and scales inside the tensor
// core and accumulates in fp32, so no value is ever widened in a register.
//
// Roles, tile schedule, epilogue and bounded waits are those of gemm_kernel
// (gge_kernel.cuh).  What differs:
//   * one thread walks the producer's loop and one the MMA warp's, so a stage
//     costs no warp votes: with 64 rows a stage's MMAs take less time than the
//     issuing loop (16 x 8192 x 8192 nvfp4: 13.8 -> 12.4 us);
//   * few tiles are split along K over a cluster of 2 to 8 CTAs (mx_reduce): each
//     contracts a share of K into its own TMEM and hands the accumulator chunks it
//     does not own to their owner's shared memory; after one cluster barrier the
//     owners add them in rank order and run the epilogue.  (Partial sums through
//     global memory and tickets, as gemm_kernel's split last wave has them, cost
//     about 5 us here, more than the split saved.)
//   * a stage also holds the scale tiles of its k-tile (512 bytes for 128 rows x
//     4 blocks), brought by TMA like the codes;
//   * before a stage's MMAs the issuing lane copies those tiles into TMEM
//     (tcgen05.cp 32x128b.warpx4: 32 lanes x 4 columns, repeated in the four lane
//     quadrants).  Copies and MMAs of one thread run in order, so one set of
//     scale columns serves every stage;
//   * a CTA pair's peer needs its own 128 rows of A's scales but all BN rows of
//     B's, so each CTA stages all of B's scales;
//   * TMEM has 512 columns: two 256-wide accumulators and 48 scale columns do not
//     fit side by side, so the second accumulator starts at column 208 and shares
//     48 columns with the first.  The epilogue reads the shared chunks first; the
//     next tile's MMAs wait for those reads only, not for the whole tile's.
//
// What bounds it: large products run into the L2 -> SM feed and the tensor pipe at
// about the same rate (a 256 x 256 tile takes 34-38 KB a stage and SM, 512 tensor
// cycles; an SM takes in 64 bytes a cycle), and the power cap lowers the clock.
// 8192^3 nvfp4 161-165 us in short bursts (6.7-6.8 PFLOP/s, 3.5 times bf16's measured
// rate), 182-185 us under a lasting load; mxfp8 4096^3 46 us, with C, gelu and two
// outputs 54; the backward activation epilogue with silu 52, with act(C) too 64.  A few
// rows are bound by the weights' bytes: 16 x 19456 x 8192 nvfp4 18.2 us (4.9 TB/s; 3.3 us
// are the launch of any shape).
#pragma once

#include "../gge_kernel.cuh"
#include "mx_format.cuh"
#include "mx_launch.h"

namespace gge {
namespace mx {

namespace ptxmx {

// 32 lanes x 128 bits from shared memory to four TMEM columns, in all four lane
// quadrants (CG = 2: in both CTAs of the pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t sdesc) {
  if constexpr (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}

#define GGE_MX_MMA(CGN, KIND)                                                                   \
  asm volatile(                                                                                 \
      "{\n\t.reg .pred p;\n\t"                                                                  \
      "setp.ne.b32 p, %6, 0;\n\t"                                                               \
      "tcgen05.mma.cta_group::" CGN "." KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), \
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)                   \
      : "memory")

template <int FMT, int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                    uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
  if constexpr (FMT == FMT_MXFP8) {
    if constexpr (CG == 1) GGE_MX_MMA("1", "kind::mxf8f6f4.block_scale.scale_vec::1X");
    else GGE_MX_MMA("2", "kind::mxf8f6f4.block_scale.scale_vec::1X");
  } else if constexpr (FMT == FMT_MXFP4) {
    if constexpr (CG == 1) GGE_MX_MMA("1", "kind::mxf4.block_scale.scale_vec::2X");
    else GGE_MX_MMA("2", "kind::mxf4.block_scale.scale_vec::2X");
  } else {
    if constexpr (CG == 1) GGE_MX_MMA("1", "kind::mxf4nvf4.block_scale.scale_vec::4X");
    else GGE_MX_MMA("2", "kind::mxf4nvf4.block_scale.scale_vec::4X");
  }
}
#undef GGE_MX_MMA

}  // namespace ptxmx

template <int BN, int CG, int FMT>
struct MxCfg {
  static constexpr int kTileM = kBM * CG;
  static constexpr int kBRows = BN / CG;
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = kBRows * kRowBytes;
  static constexpr int kBK = kRowBytes * 8 / Fmt<FMT>::kBits;  // K values a stage
  static constexpr int kGroups = kBK / Fmt<FMT>::kGroup;       // scale words a row and stage
  static constexpr int kBTiles = (BN + 127) / 128;             // 128-row scale tiles of B
  static constexpr int kSfaBytes = kGroups * 512;
  static constexpr int kSfbBytes = kBTiles * kGroups * 512;
  static constexpr int kLoadBytes = kABytes + kBBytes + kSfaBytes + kSfbBytes;
  // (a stage starts on a 1 KiB boundary, for the swizzle atoms)
  static constexpr int kStageBytes = (kLoadBytes + 1023) / 1024 * 1024;
  static constexpr int kStep = kBK / 4;  // K values one MMA contracts (32 bytes)
  static constexpr int kEpiWarps = 8;
  static constexpr int kMmaWarp = 8, kLoadWarp = 9;
  static constexpr int kThreads = 10 * 32;
  // TMEM columns: the scales at the end, the second accumulator as far up as it goes
  static constexpr int kSfCols = 4 * kGroups * (1 + kBTiles);
  static constexpr int kTmemCols = BN == 64 ? 256 : 512;
  static constexpr int kSfBase = kTmemCols - 48;
  static constexpr bool kOverlap = BN == 256;  // the accumulators share columns
  static constexpr int kAcc1 = kOverlap ? 208 : BN;
  static_assert(kSfCols <= 48 && kAcc1 + BN <= kSfBase, "TMEM columns");
  static_assert(BN == 256 || BN == 128 || BN == 64, "tile widths");
};

constexpr int kMaxStages = 8;

// Shared-memory descriptor of one 512-byte scale tile: no swizzle, 8-row groups
// of 16-byte rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) |
         (uint64_t(128 >> 4) << 32) | (uint64_t(1) << 46);
}

// This CTA's k-tiles [k0, k1): all of them, or its share in a cluster split along K.
struct KSpan {
  int32_t k0, k1;
};
__device__ __forceinline__ KSpan k_span(const MxParams& mp, uint32_t slice) {
  const int64_t k = mp.p.k_tiles;
  return KSpan{static_cast<int32_t>(slice * k / mp.splits),
               static_cast<int32_t>((slice + 1) * k / mp.splits)};
}

// Run by one thread.
template <int BN, int CG, int FMT>
__device__ __forceinline__ void mx_mma_role(const MxParams& mp, const Shared& sh, uint32_t stage0,
                                            uint32_t tmem_base, const KSpan& ks, int32_t unit,
                                            int32_t units) {
  using Cfg = MxCfg<BN, CG, FMT>;
  const Params& p = mp.p;
  int stage = 0;
  uint32_t phase = 0;
  const uint32_t sfa_t = tmem_base + Cfg::kSfBase;
  const uint32_t sfb_t = sfa_t + 4 * Cfg::kGroups;
  int i = 0;
  for (int32_t t = unit; t < p.num_tiles; t += units, ++i) {
    const uint32_t acc = static_cast<uint32_t>(i) & 1u;
    if (Cfg::kOverlap) {
      // the columns shared with the tile before are read (and all of the one before that)
      if (i > 0 && !wait_phase<CG == 2>(sh.tempty, static_cast<uint32_t>(i - 1) & 1u, p, sh, 2, t)) return;
    } else if (i > 1) {
      // the accumulator's last tile is read.  (A barrier each: a warp may read the next
      // tile, in the other accumulator, before its neighbours have read this one.)
      if (!wait_phase<CG == 2>(sh.tempty + 8 * acc, static_cast<uint32_t>((i >> 1) - 1) & 1u, p, sh, 2, t)) return;
    }
    ptx::tc_fence_after();
    const uint32_t d_tmem = tmem_base + acc * Cfg::kAcc1;
    // 64-wide tiles: an odd one starts in the middle of a 128-row scale tile
    uint32_t sfb = sfb_t;
    if constexpr (BN == 64) sfb += (tile_coord<BN, Cfg::kTileM>(t, p, sh).n0 & 64) ? 2u : 0u;
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      if (!wait_phase<CG == 2>(sh.full + 8 * stage, phase, p, sh, 1, t)) return;
      ptx::tc_fence_after();
      const uint32_t a_addr = stage0 + stage * Cfg::kStageBytes;
      const uint32_t b_addr = a_addr + Cfg::kABytes;
      const uint32_t sfa_addr = b_addr + Cfg::kBBytes;
      const uint32_t sfb_addr = sfa_addr + Cfg::kSfaBytes;
      const int32_t nk = min(4, (p.K - kt * Cfg::kBK + Cfg::kStep - 1) / Cfg::kStep);
      // scale words are copied just before the first MMA that uses them, so that the
      // copies run under the MMA before (8192^3 nvfp4: 167 -> 164 us)
      constexpr int kPerGroup = 4 / Cfg::kGroups;  // MMAs that share a scale word
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk >= nk) break;
        const int g = kk / kPerGroup;
        if (kk % kPerGroup == 0) {
          ptxmx::copy_scales<CG>(sfa_t + 4 * g, scale_desc(sfa_addr + g * 512));
#pragma unroll
          for (int j = 0; j < Cfg::kBTiles; ++j)
            ptxmx::copy_scales<CG>(sfb_t + 4 * (g * Cfg::kBTiles + j),
                                   scale_desc(sfb_addr + (j * Cfg::kGroups + g) * 512));
        }
        const uint64_t adesc = smem_desc(a_addr + kk * 32u, 16u, 1024u);
        const uint64_t bdesc = smem_desc(b_addr + kk * 32u, 16u, 1024u);
        // which of a scale word's bytes this MMA's blocks use
        const uint32_t id = static_cast<uint32_t>(kk % kPerGroup) * (4 / kPerGroup);
        const uint32_t idesc = p.idesc | (id << 4) | (id << 29);
        ptxmx::mma<FMT, CG>(d_tmem, adesc, bdesc, idesc, sfa_t + 4 * g,
                            sfb + 4 * Cfg::kBTiles * g, (kt > ks.k0 || kk > 0) ? 1u : 0u);
      }
      if (CG == 1) ptx::mma_commit(sh.empty + 8 * stage);
      else ptx::mma_commit_pair(sh.empty + 8 * stage, 0x3);
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    if (!(p.flags & FLAG_TEST_DROP_ACC_FULL)) {
      if (CG == 1) ptx::mma_commit(sh.tfull + 8 * acc);
      else ptx::mma_commit_pair(sh.tfull + 8 * acc, 0x3);
    }
  }
}

// Run by one thread.
template <int BN, int CG, int FMT>
__device__ __forceinline__ void mx_load_role(const MxParams& mp, const Shared& sh,
                                             const CUtensorMap* tmA, const CUtensorMap* tmB,
                                             const CUtensorMap* tmSA, const CUtensorMap* tmSB,
                                             uint32_t stage0, uint32_t rank, const KSpan& ks,
                                             int32_t unit, int32_t units) {
  using Cfg = MxCfg<BN, CG, FMT>;
  const Params& p = mp.p;
  int stage = 0;
  uint32_t phase = 0;
  for (int32_t t = unit; t < p.num_tiles; t += units) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    const int32_t row0 = tc.m_row0 + static_cast<int32_t>(rank) * kBM;
    const int32_t bn0 = tc.n0 + static_cast<int32_t>(rank) * Cfg::kBRows;
    const int32_t sa = tc.a_batch * mp.sfa_batch + (row0 >> 7);
    const int32_t sb = tc.b_batch * mp.sfb_batch + (tc.n0 >> 7);
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      if (!wait_phase<CG == 2>(sh.empty + 8 * stage, phase ^ 1u, p, sh, 0, t)) return;
      const uint32_t full = sh.full + 8 * stage;
      if (CG == 1) ptx::mbar_arrive_expect_tx(full, Cfg::kLoadBytes);
      else if (rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * Cfg::kLoadBytes);
      const uint32_t bar = (CG == 1) ? full : ptx::mapa(full, 0);
      const uint32_t a_dst = stage0 + stage * Cfg::kStageBytes;
      const uint32_t b_dst = a_dst + Cfg::kABytes;
      const uint32_t sfa_dst = b_dst + Cfg::kBBytes;
      tma_load<CG>(a_dst, tmA, bar, kt * kRowBytes, row0, tc.a_batch);
      tma_load<CG>(b_dst, tmB, bar, kt * kRowBytes, bn0, tc.b_batch);
      tma_load<CG>(sfa_dst, tmSA, bar, 0, kt * Cfg::kGroups, sa);
      tma_load<CG>(sfa_dst + Cfg::kSfaBytes, tmSB, bar, 0, kt * Cfg::kGroups, sb);
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
  }
}

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A split tile's 32 x 32 accumulator chunks (lane quadrant x 32 columns) are dealt
// out to the cluster's CTAs in order; chunk `n` of 4 BN / 32 belongs to rank n S /
// (4 BN / 32).
template <int BN>
__device__ __forceinline__ uint32_t chunk_owner(int n, int32_t splits) {
  return static_cast<uint32_t>(n * splits) / (4 * (BN / 32));
}

// Where rank `from` leaves chunk n in its owner's shared memory (one float4 a lane
// and four columns, so each store instruction writes 512 contiguous bytes).
template <int BN>
__device__ __forceinline__ uint32_t chunk_slot(uint32_t red, int n, uint32_t owner, uint32_t from,
                                               int32_t splits) {
  constexpr int kChunks = 4 * (BN / 32);
  const int mine = kChunks / splits;  // chunks an owner has (both are powers of two)
  const uint32_t order = from < owner ? from : from - 1;
  return red + (order * mine + n % mine) * 4096u + (threadIdx.x & 31) * 16u;
}

// Hand the chunks of this CTA's accumulator that other ranks own to them.
template <int BN>
__device__ __forceinline__ void mx_send(const MxParams& mp, uint32_t tbase, int32_t n0, int quad, int half,
                                        uint32_t slice, uint32_t red) {
#pragma unroll 1
  for (int c = half; c < BN / 32; c += 2) {
    if (n0 + c * 32 >= mp.p.N) break;  // (no rank computes with these columns)
    const int n = quad * (BN / 32) + c;
    const uint32_t owner = chunk_owner<BN>(n, mp.splits);
    if (owner == slice) continue;
    uint32_t v[32];
    __syncwarp();
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, v);
    ptx::tmem_wait_ld(v);
    const uint32_t dst = ptx::mapa(chunk_slot<BN>(red, n, owner, slice, mp.splits), owner);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + q * 512u), "r"(v[4 * q]),
                   "r"(v[4 * q + 1]), "r"(v[4 * q + 2]), "r"(v[4 * q + 3])
                   : "memory");
  }
}

__device__ __forceinline__ float mx_alpha(const MxParams& mp) {
  float alpha = mp.p.dact ? 1.f : (mp.p.alpha_dev ? *mp.p.alpha_dev : mp.p.alpha);
  if (mp.tscale_a != nullptr) alpha *= *mp.tscale_a;
  if (mp.tscale_b != nullptr) alpha *= *mp.tscale_b;
  return alpha;
}

// A split tile's owned chunks, after the cluster barrier: the ranks' copies added in
// rank order, then the epilogue.  One tile a cluster.
template <int BN, int FMT, bool TR>
__device__ __forceinline__ void mx_reduce(const MxParams& mp, const Shared& sh, uint32_t tmem_base,
                                          uint32_t slice, uint32_t red, uint32_t stg, int32_t t,
                                          float alpha, float beta) {
  const Params& p = mp.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = warp >> 2;
  const TileCoord tc = tile_coord<BN, kBM>(t, p, sh);
  const int32_t row_base = tc.m_row0 + quad * 32;
  const int32_t rows_valid = min(32, tc.row_limit - row_base);
  const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
  for (int c = half; c < BN / 32; c += 2) {
    const int32_t col0 = tc.n0 + c * 32;
    const int n = quad * (BN / 32) + c;
    if (col0 >= p.N || rows_valid <= 0 || chunk_owner<BN>(n, mp.splits) != slice) continue;
    CRegs creg = {};
    if (p.c != nullptr && lane < rows_valid) load_c_chunk<TR>(p, row_base + lane, col0, tc.batch, creg);
    uint32_t own[32];
    __syncwarp();
    ptx::tmem_ld_32x32b_x32(tbase + c * 32, own);
    ptx::tmem_wait_ld(own);
    float sum[32];
    for (int32_t r = 0; r < mp.splits; ++r) {
      const uint32_t src = chunk_slot<BN>(red, n, slice, static_cast<uint32_t>(r), mp.splits);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        uint4 v = make_uint4(own[4 * q], own[4 * q + 1], own[4 * q + 2], own[4 * q + 3]);
        if (r != static_cast<int32_t>(slice)) v = ptx::ld_shared_v4(src + q * 512u);
        const float f[4] = {__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w)};
#pragma unroll
        for (int j = 0; j < 4; ++j) sum[4 * q + j] = r == 0 ? f[j] : sum[4 * q + j] + f[j];
      }
    }
    // (the backward epilogue takes the accumulator as it is)
    const float scale = p.dact ? alpha : 1.f;
#pragma unroll
    for (int j = 0; j < 32; ++j) own[j] = __float_as_uint(sum[j] * scale);
    epilogue_chunk_t<TR>(p, own, row_base, rows_valid, col0, tc.batch, alpha, beta, creg, stg);
  }
}

template <int BN, int CG, int FMT, bool TR>
__device__ __forceinline__ void mx_epilogue_role(const MxParams& mp, const Shared& sh,
                                                 uint32_t tmem_base, uint32_t rank, uint32_t stg,
                                                 int32_t unit, int32_t units, uint32_t slice,
                                                 uint32_t red, float alpha, float beta) {
  using Cfg = MxCfg<BN, CG, FMT>;
  const Params& p = mp.p;
  constexpr int kMine = BN / 64;  // 32-column chunks of this warp (two warps a lane quadrant)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = warp & 3, half = warp >> 2;
  const bool lean = !TR && p.c == nullptr && p.post == nullptr && p.out_stage_bytes != 0 &&
                    p.d_dtype != DT_F32;
  int i = 0;
  for (int32_t t = unit; t < p.num_tiles; t += units, ++i) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    const uint32_t acc = static_cast<uint32_t>(i) & 1u;
    const uint32_t acc_phase = static_cast<uint32_t>(i >> 1) & 1u;
    const int32_t row_base = tc.m_row0 + static_cast<int32_t>(rank) * kBM + quad * 32;
    const int32_t rows_valid = min(32, tc.row_limit - row_base);
    const int32_t row = row_base + lane;
    const bool has_c = p.c != nullptr && lane < rows_valid;
    // this warp's chunks are half, half + 2, ...; the first accumulator's walk starts at
    // its last pair, the second one's at its first: the columns both own
    const int first = (Cfg::kOverlap && acc == 0) ? kMine - 1 : 0;
    CRegs cnext = {};
    if (mp.splits == 1 && has_c && tc.n0 + (half + 2 * first) * 32 < p.N)
      load_c_chunk<TR>(p, row, tc.n0 + (half + 2 * first) * 32, tc.batch, cnext);
    // (polled: the next tile's MMAs wait for this one's first chunks)
    const bool ok = wait_phase<CG == 2>(sh.tfull + 8 * acc, acc_phase, p, sh, 3, t);
    if (!__all_sync(0xffffffffu, ok)) {
      if (CG == 1 && mp.splits > 1) cluster_wait();
      return;
    }
    ptx::tc_fence_after();
    const uint32_t tbase = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + acc * Cfg::kAcc1;
    if (CG == 1 && mp.splits > 1) {  // (one tile a cluster: mx_reduce finishes it)
      cluster_wait();  // every CTA of the cluster runs: their shared memory may be written
      mx_send<BN>(mp, tbase, tc.n0, quad, half, slice, red);
      return;
    }
#pragma unroll 1
    for (int n = 0; n < kMine; ++n) {
      const int ci = (n + first) % kMine;
      const int c = half + 2 * ci;
      const int32_t col0 = tc.n0 + c * 32;
      const CRegs ccur = cnext;
      if (has_c && n + 1 < kMine) {
        const int32_t next = tc.n0 + (half + 2 * ((ci + 1) % kMine)) * 32;
        if (next < p.N) load_c_chunk<TR>(p, row, next, tc.batch, cnext);
      }
      uint32_t v[32];
      __syncwarp();
      if (p.k_tiles > 0) {
        ptx::tmem_ld_32x32b_x32(tbase + c * 32, v);
        ptx::tmem_wait_ld(v);
      } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = 0u;
      }
      if (n == (Cfg::kOverlap ? 0 : kMine - 1)) {
        // the columns the next tile's accumulator shares are read (and, in program
        // order, all of the tile before this one): its MMAs may start.  Without shared
        // columns: this accumulator is read
        ptx::tc_fence_before();
        __syncwarp();
        const uint32_t bar = sh.tempty + (Cfg::kOverlap ? 0u : 8u * acc);
        if (lane == 0) {
          if (CG == 1) ptx::mbar_arrive(bar);
          else ptx::mbar_arrive_remote(ptx::mapa(bar, 0));
        }
      }
      if (rows_valid > 0 && col0 < p.N) {
        if (lean) {
          float x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]) * alpha;
          store_chunk_staged(stg, x, p.d_dtype,
                             out_ptr(p.d, p.ldd, p.sbd, p.d_dtype, row_base, col0, tc.batch, p),
                             2 * p.ldd, rows_valid, min(32, p.N - col0), false);
        } else {
          if (p.dact) {  // (it takes the accumulator as it is)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * alpha);
          }
          epilogue_chunk_t<TR>(p, v, row_base, rows_valid, col0, tc.batch, alpha, beta, ccur, stg);
        }
      }
    }
  }
}

template <int BN, int CG, int FMT, bool TR>
__global__ void __launch_bounds__(MxCfg<BN, CG, FMT>::kThreads, 1)
    mx_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmSA,
                   const __grid_constant__ CUtensorMap tmSB, const __grid_constant__ MxParams mp) {
  using Cfg = MxCfg<BN, CG, FMT>;
  const Params& p = mp.p;
  extern __shared__ uint8_t smem_raw[];
  ptx::griddep_launch_dependents();
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const int S = p.stages;
  const uint32_t out_stage = base + S * Cfg::kStageBytes;
  // split K: the other ranks' chunks of what this CTA owns
  const uint32_t red = out_stage + Cfg::kEpiWarps * p.out_stage_bytes;
  uint8_t* ctrl = base_ptr + S * Cfg::kStageBytes + Cfg::kEpiWarps * p.out_stage_bytes + mp.reduce_bytes;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kMaxStages + 5));
  int32_t* abort_flag = reinterpret_cast<int32_t*>(tmem_slot + 1);

  Shared sh = {};
  sh.full = ptx::smem_addr(ctrl);
  sh.empty = sh.full + 8 * kMaxStages;
  sh.tfull = sh.empty + 8 * kMaxStages;
  sh.tempty = sh.tfull + 16;
  const uint32_t drain_bar = sh.tempty + 16;
  sh.abort = abort_flag;

  const int warp = threadIdx.x >> 5;
  const uint32_t crank = (CG == 2 || mp.splits > 1) ? ptx::cluster_ctarank() : 0u;
  const uint32_t rank = (CG == 2) ? crank : 0u;      // in the pair
  const uint32_t slice = (CG == 2) ? 0u : crank;     // of K
  const int32_t ctas = CG * mp.splits;               // of the cluster
  const int32_t unit = static_cast<int32_t>(blockIdx.x) / ctas;
  const int32_t units = static_cast<int32_t>(gridDim.x) / ctas;
  const KSpan ks = k_span(mp, slice);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(sh.full + 8 * s, 1);
      ptx::mbar_init(sh.empty + 8 * s, 1);
    }
    ptx::mbar_init(sh.tfull, 1);
    ptx::mbar_init(sh.tfull + 8, 1);
    ptx::mbar_init(sh.tempty, Cfg::kEpiWarps * CG);
    ptx::mbar_init(sh.tempty + 8, Cfg::kEpiWarps * CG);
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == Cfg::kLoadWarp && (threadIdx.x & 31) == 0 && p.k_tiles > 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmSA);
    ptx::prefetch_tmap(&tmSB);
  }
  if (warp == Cfg::kMmaWarp) {
    if (CG == 1) {
      ptx::tmem_alloc(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
      ptx::tmem_relinquish();
    } else {
      ptx::tmem_alloc_pair(ptx::smem_addr(tmem_slot), Cfg::kTmemCols);
      ptx::tmem_relinquish_pair();
    }
    ptx::tc_fence_before();
  }
  ptx::griddep_wait();
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  if (CG == 1 && mp.splits > 1) cluster_arrive();  // (waited for before the first remote store)
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // (read before the main loop: they would cost the split's last step two loads' latency)
  float alpha = 1.f, beta = 0.f;
  if (warp < Cfg::kEpiWarps) {
    alpha = mx_alpha(mp);
    beta = p.beta_dev ? *p.beta_dev : p.beta;
    mx_epilogue_role<BN, CG, FMT, TR>(mp, sh, tmem_base, rank, out_stage + warp * p.out_stage_bytes,
                                      unit, units, slice, red, alpha, beta);
  } else if (warp == Cfg::kMmaWarp) {
    if (rank == 0 && ptx::elect_one()) mx_mma_role<BN, CG, FMT>(mp, sh, base, tmem_base, ks, unit, units);
  } else {
    if (ptx::elect_one())
      mx_load_role<BN, CG, FMT>(mp, sh, &tmA, &tmB, &tmSA, &tmSB, base, rank, ks, unit, units);
  }
  __syncwarp();
  if (CG == 1 && mp.splits > 1) {
    if (warp >= Cfg::kEpiWarps) cluster_wait();
    cluster_arrive();
    cluster_wait();  // every rank's chunks are where they belong
    if (warp < Cfg::kEpiWarps && !*abort_flag) {
      ptx::tc_fence_after();
      mx_reduce<BN, FMT, TR>(mp, sh, tmem_base, slice, red, out_stage + warp * p.out_stage_bytes, unit, alpha,
                             beta);
      ptx::tc_fence_before();
    }
  }

  __syncthreads();
  // Every MMA and scale copy this CTA issued has finished before TMEM is freed: its
  // epilogue has waited for the last tile's, unless a wait ran out.
  if (*abort_flag && warp == Cfg::kMmaWarp && rank == 0) {
    if (ptx::elect_one()) {
      if (CG == 1) ptx::mma_commit(drain_bar);
      else ptx::mma_commit_pair(drain_bar, 0x1);
    }
    __syncwarp();
    wait_phase<CG == 2>(drain_bar, 0, p, sh, 6, -1);
  }
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  if (*abort_flag) {
    // let copies and MMAs that were in flight land before the memory goes away
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 200000ull) __nanosleep(1000);
  }
  if (warp == Cfg::kMmaWarp) {
    __syncwarp();
    ptx::tc_fence_after();
    if (CG == 1) ptx::tmem_dealloc(tmem_base, Cfg::kTmemCols);
    else ptx::tmem_dealloc_pair(tmem_base, Cfg::kTmemCols);
  }
}

}  // namespace mx
}  // namespace gge
