// Product of two matrices in 8 bits with a scale for each block of 128 along K (of one row, or
// of 128 rows):
//
//   S[m, n] = sum over blocks b of sA[m, b] sB[n, b] T_b[m, n],   T_b = sum in b of a b
//   D = alpha S + beta C     PostAct = act(same)        (or the backward activation epilogue)
//
// The scales are fp32 of any value, so they cannot go through the tensor core (its block
// scales are powers of two or 8 bits): a k-tile is one block, and its T_b, accumulated by
// tcgen05.mma kind::f8f6f4 in tensor memory, is read, scaled and added to fp32 sums that stay in
// registers over the whole of K.  What follows from that:
//   * tensor memory holds no sums but the T_b in flight, two 256-wide or four narrower ones: the
//     MMAs of the next blocks run while one is read;
//   * two warpgroups hold the sums, a row and half of the tile's columns a thread: 128 registers
//     of 224, which setmaxnreg takes from the warpgroup that loads and issues;
//   * a thread's row has one scale a block, and with blocks of 128 rows its columns have one,
//     too: a product and one packed fused multiply-add for two values.  With a scale for each
//     row of B (weight gradients) two packed operations, the columns' scales out of shared memory;
//   * scales come through a ring of their own, by one warp's cp.async up to eight blocks ahead:
//     they may lie anywhere (the rows of a group start on any row);
//   * half of a 256-wide tile's columns is one block of an 8-bit output's scales: its largest
//     value is found without leaving the thread;
//   * few tiles are split along K over a cluster of 2 to 8 CTAs: with their sums complete, each
//     hands the pieces (32 rows x half of the columns) that it does not own to their owner's
//     shared memory, and after one cluster barrier the owners add them in rank order.
//
// Tile schedule, tensor maps, bounded waits and the staged stores are those of gemm_kernel
// (gge_kernel.cuh).
#pragma once

#include "../gge_kernel.cuh"
#include "b128_launch.h"

namespace gge {
namespace b128 {

constexpr int kMaxStages = 8;
constexpr int kScaleSlots = 8;
constexpr int kHoldRegs = 224, kIssueRegs = 56;  // of the warpgroups that hold sums, and of the other

template <int BN, int CG, bool BV>
struct GemmCfg {
  static constexpr int kTileM = kBM * CG;
  static constexpr int kBRows = BN / CG;
  static constexpr int kABytes = kBM * kRowBytes;
  static constexpr int kBBytes = kBRows * kRowBytes;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kHalf = BN / 2;                 // columns a thread holds
  static constexpr int kBuffers = BN == 256 ? 2 : 4;   // blocks' sums in tensor memory
  static constexpr int kTmemCols = kBuffers * BN;
  static constexpr int kScaleFloats = kBM + (BV ? BN : 4);
  static constexpr int kEpiWarps = 8;
  static constexpr int kMmaWarp = 8, kLoadWarp = 9, kScaleWarp = 10;
  static constexpr int kThreads = 12 * 32;
  static_assert(kTmemCols <= 512, "tensor memory");
};

struct Rings {
  uint32_t sfull, sempty;  // scale ring barriers (kScaleSlots each)
  uint32_t scales;         // its slots
  uint32_t xbar, xch;      // a quad's two warps: barriers [4], floats [2][8][32]
};

// wait_phase without a call: the sums stay in their registers.
template <bool CLUSTER>
__device__ __forceinline__ bool wait_here(uint32_t bar, uint32_t parity, const Params& p, const Shared& sh,
                                          int32_t where, int32_t tile) {
  const auto probe = [&]() {
    return CLUSTER ? ptx::mbar_try_wait_cluster(bar, parity) : ptx::mbar_try_wait(bar, parity);
  };
  if (probe()) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (!probe()) {
    if (*sh.abort) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      record_status(p, DEV_TIMEOUT, where, tile);
      *sh.abort = 1;
      return false;
    }
  }
  return true;
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

// Run by one thread.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void mma_role(const GemmParams& gp, const Shared& sh, uint32_t stage0, uint32_t tmem_base,
                                         const KSpan& ks, int32_t unit, int32_t units, int32_t num_tiles) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  int stage = 0, buf = 0;
  uint32_t phase = 0, buf_phase = 1;  // (the first pass over the buffers waits for nobody)
  for (int32_t t = unit; t < num_tiles; t += units) {
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      if (!wait_phase<CG == 2>(sh.tempty + 8 * buf, buf_phase, p, sh, 2, t)) return;
      if (!wait_phase<CG == 2>(sh.full + 8 * stage, phase, p, sh, 1, t)) return;
      ptx::tc_fence_after();
      const uint32_t a_addr = stage0 + stage * Cfg::kStageBytes;
      const uint32_t b_addr = a_addr + Cfg::kABytes;
      const uint32_t d = tmem_base + buf * BN;
      const int32_t nk = min(4, (p.K - kt * kBlock + 31) / 32);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        if (kk >= nk) break;
        const uint64_t adesc = smem_desc(a_addr + kk * 32u, 16u, 1024u);
        const uint64_t bdesc = smem_desc(b_addr + kk * 32u, 16u, 1024u);
        if (CG == 1) ptx::mma_f8(d, adesc, bdesc, p.idesc, kk > 0 ? 1u : 0u);
        else ptx::mma_f8_pair(d, adesc, bdesc, p.idesc, kk > 0 ? 1u : 0u);
      }
      if (CG == 1) ptx::mma_commit(sh.empty + 8 * stage);
      else ptx::mma_commit_pair(sh.empty + 8 * stage, 0x3);
      if (!(p.flags & FLAG_TEST_DROP_ACC_FULL)) {
        if (CG == 1) ptx::mma_commit(sh.tfull + 8 * buf);
        else ptx::mma_commit_pair(sh.tfull + 8 * buf, 0x3);
      }
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      if (++buf == Cfg::kBuffers) { buf = 0; buf_phase ^= 1u; }
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
      if (!wait_phase<CG == 2>(sh.empty + 8 * stage, phase ^ 1u, p, sh, 0, t)) return;
      const uint32_t full = sh.full + 8 * stage;
      if (CG == 1) ptx::mbar_arrive_expect_tx(full, Cfg::kStageBytes);
      else if (rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * Cfg::kStageBytes);
      const uint32_t bar = (CG == 1) ? full : ptx::mapa(full, 0);
      const uint32_t dst = stage0 + stage * Cfg::kStageBytes;
      if (CG == 1) {
        ptx::tma_load_3d(dst, tmA, bar, kt * kBlock, row0, tc.a_batch);
        ptx::tma_load_3d(dst + Cfg::kABytes, tmB, bar, kt * kBlock, bn0, tc.b_batch);
      } else {
        ptx::tma_load_3d_pair(dst, tmA, bar, kt * kBlock, row0, tc.a_batch);
        ptx::tma_load_3d_pair(dst + Cfg::kABytes, tmB, bar, kt * kBlock, bn0, tc.b_batch);
      }
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
  }
}

// A slot of the scale ring: the CTA's 128 rows' scales, then the columns': one each (BV), or one
// for each 128.  Rows and columns that are not there get zeros.  Run by one warp.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void scale_role(const GemmParams& gp, const Shared& sh, const Rings& rg, uint32_t rank,
                                           const KSpan& ks, int32_t unit, int32_t units, int32_t num_tiles) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  const int lane = threadIdx.x & 31;
  int slot = 0;
  uint32_t phase = 1;
  for (int32_t t = unit; t < num_tiles; t += units) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    const int32_t row0 = tc.m_row0 + static_cast<int32_t>(rank) * kBM;
    const int32_t row_end = p.num_groups > 0 ? tc.row_limit : p.M;
    const float* a = gp.a.scales + tc.a_batch * gp.a.s_batch + ks.k0 * gp.a.s_col;
    const float* b = gp.b.scales + tc.b_batch * gp.b.s_batch + ks.k0 * gp.b.s_col;
    for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
      if (!wait_phase(rg.sempty + 8 * slot, phase, p, sh, 10, t)) return;
      const uint32_t dst = rg.scales + slot * (Cfg::kScaleFloats * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t row = row0 + lane + 32 * i;
        const bool there = row < row_end;
        cp_async_4(dst + 4 * (lane + 32 * i), there ? a + (row >> gp.a.shift) * gp.a.s_row : a, there);
      }
      if constexpr (BV) {
#pragma unroll
        for (int i = 0; i < BN / 32; ++i) {
          const int32_t col = tc.n0 + lane + 32 * i;
          const bool there = col < p.N;
          cp_async_4(dst + 4 * (kBM + lane + 32 * i), there ? b + col * gp.b.s_row : b, there);
        }
      } else if (lane < (BN + 127) / 128) {
        const int32_t col = tc.n0 + lane * 128;
        const bool there = col < p.N;
        cp_async_4(dst + 4 * (kBM + lane), there ? b + (col >> 7) * gp.b.s_row : b, there);
      }
      a += gp.a.s_col;
      b += gp.b.s_col;
      ptx::cp_async_mbar_arrive_noinc(rg.sfull + 8 * slot);
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
    for (int i = 0; i < 16; ++i)
      acc[i] = __ffma2_rn(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), s2, acc[i]);
  }
}

// Where a promoting warp is in the rings.
struct Place {
  int slot, buf;
  uint32_t slot_phase, buf_phase;
};

// A tile's blocks [k0, k1) added to `acc`.  `idle`: none of the warp's rows is wanted (the
// buffers are only handed back).  False after a wait that ran out.
template <int BN, int CG, bool BV>
__device__ __forceinline__ bool add_blocks(const GemmParams& gp, const Shared& sh, const Rings& rg, uint32_t tmem,
                                           int quad, int half, const KSpan& ks, int32_t t, bool idle, Place& at,
                                           float2 (&acc)[GemmCfg<BN, CG, BV>::kHalf / 2]) {
  using Cfg = GemmCfg<BN, CG, BV>;
  constexpr int kChunks = Cfg::kHalf / 32;
  const Params& p = gp.p;
  const int lane = threadIdx.x & 31;
  for (int32_t kt = ks.k0; kt < ks.k1; ++kt) {
    bool ok = wait_here<false>(rg.sfull + 8 * at.slot, at.slot_phase, p, sh, 11, t);
    const uint32_t scales = rg.scales + at.slot * (Cfg::kScaleFloats * 4);
    float s = ld_shared_f32(scales + 4 * (quad * 32 + lane));
    if constexpr (!BV) s *= ld_shared_f32(scales + 4 * (kBM + (BN == 256 ? half : 0)));
    ok = ok && wait_here<CG == 2>(sh.tfull + 8 * at.buf, at.buf_phase, p, sh, 3, t);
    if (!__all_sync(0xffffffffu, ok)) return false;
    ptx::tc_fence_after();
    const uint32_t from = tmem + at.buf * BN;
    const uint32_t empty = sh.tempty + 8 * at.buf;
    const auto hand_back = [&]() {
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1) ptx::mbar_arrive(empty);
        else ptx::mbar_arrive_remote(ptx::mapa(empty, 0));
      }
    };
    if (idle) {
      hand_back();
    } else {
      uint32_t v[2][32];
      ptx::tmem_ld_32x32b_x32(from, v[0]);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        ptx::tmem_wait_ld(v[c & 1]);
        if (c + 1 < kChunks) ptx::tmem_ld_32x32b_x32(from + (c + 1) * 32, v[(c + 1) & 1]);
        else hand_back();
        add_chunk<BV>(acc + c * 16, v[c & 1], s, scales + 4 * (kBM + half * Cfg::kHalf + c * 32));
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(rg.sempty + 8 * at.slot);
    if (++at.slot == kScaleSlots) { at.slot = 0; at.slot_phase ^= 1u; }
    if (++at.buf == Cfg::kBuffers) { at.buf = 0; at.buf_phase ^= 1u; }
  }
  return true;
}

// ------------------------------------------------------------ the outputs

// The epilogue walks a thread's columns in chunks of 32, always the first 32 of the sums, which
// then move round by that many: the code of a chunk is there once, and the sums stay in
// registers (walked by an index they would not).
template <int P>
__device__ __forceinline__ void move_round(float2 (&acc)[P]) {
  if constexpr (P > 16) {
    float2 first[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) first[i] = acc[i];
#pragma unroll
    for (int i = 0; i < P - 16; ++i) acc[i] = acc[i + 16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[P - 16 + i] = first[i];
  }
}

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
// Eight of them (group g) as numbers; `unit` is the codes' scale, `crow` an fp32 C's place (NULL
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
__device__ __forceinline__ void dact8_t(const float (&x)[8], float2* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j].x *= dact_one<ACT>(x[2 * j]), v[j].y *= dact_one<ACT>(x[2 * j + 1]);
}
__device__ __forceinline__ void dact8(int act, const float (&x)[8], float2* v) {
  switch (act) {
    case ACT_RELU: dact8_t<ACT_RELU>(x, v); break;
    case ACT_GELU_TANH: dact8_t<ACT_GELU_TANH>(x, v); break;
    case ACT_SILU: dact8_t<ACT_SILU>(x, v); break;
    default: dact8_t<ACT_RELU_SQ>(x, v); break;
  }
}
template <int ACT>
__device__ __forceinline__ void act32_t(float2* v) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j].x = act_one<ACT>(v[j].x), v[j].y = act_one<ACT>(v[j].y);
}
__device__ __forceinline__ void act32(int act, float2* v) {
  switch (act) {
    case ACT_RELU: act32_t<ACT_RELU>(v); break;
    case ACT_GELU_TANH: act32_t<ACT_GELU_TANH>(v); break;
    case ACT_SILU: act32_t<ACT_SILU>(v); break;
    case ACT_RELU_SQ: act32_t<ACT_RELU_SQ>(v); break;
    default: break;
  }
}

// 32 columns of a 16- or 32-bit output.
__device__ __forceinline__ void store32(uint32_t stg, const float2* v, int dtype, void* out, int64_t ld, int64_t sb,
                                        int64_t batch, int32_t row_base, int32_t rows_valid, int32_t col0, int32_t N) {
  // (opaque: the staging addresses are not kept in registers from chunk to chunk)
  asm volatile("" : "+r"(stg));
  float x[32];
#pragma unroll
  for (int j = 0; j < 16; ++j) x[2 * j] = v[j].x, x[2 * j + 1] = v[j].y;
  store_chunk_staged(stg, x, dtype,
                     static_cast<char*>(out) + (batch * sb + row_base * ld + col0) * dtype_bytes(dtype),
                     ld * dtype_bytes(dtype), rows_valid, min(32, N - col0), false);
}

// One tile's (or piece's) place as a warp sees it.
struct Spot {
  int32_t row_base, rows_valid, col_base;
  int64_t batch;  // of C and the outputs
  int quad, half;
};

// The largest |value| over a row's block of 128 columns: a thread's own, or (128-wide tiles)
// joined with that of the warp that holds the other half.
template <int BN>
__device__ __forceinline__ bool join_halves(const GemmParams& gp, const Shared& sh, const Rings& rg, const Spot& at,
                                            uint32_t& use, uint32_t& amax) {
  if constexpr (BN == 128) {
    const int lane = threadIdx.x & 31;
    const uint32_t slots = rg.xch + (use & 1u) * 1024u;
    ptx::st_shared_u32(slots + 4u * ((at.quad * 2 + at.half) * 32 + lane), amax);
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(rg.xbar + 8 * at.quad);
    const bool ok = wait_here<false>(rg.xbar + 8 * at.quad, use & 1u, gp.p, sh, 12, -1);
    if (!__all_sync(0xffffffffu, ok)) return false;
    amax = max(amax, ptx::ld_shared_u32(slots + 4u * ((at.quad * 2 + (at.half ^ 1)) * 32 + lane)));
    ++use;
  }
  return true;
}

// A warp's 32 rows of 8-bit output: the thread's columns in `acc`, quantised, through the warp's
// staging buffer to whole lines.
template <int BN, bool E5M2, int P>
__device__ __forceinline__ void store_codes(const GemmParams& gp, const View& q, const Spot& at, const float2 (&acc)[P],
                                            uint32_t amax, uint32_t stg) {
  constexpr int kPieces = 2 * P / 16;  // 16-byte pieces of a row
  asm volatile("" : "+r"(stg));
  const int lane = threadIdx.x & 31;
  float factor;
  const float unit = block_scale<E5M2>(amax, factor);
  if (lane < at.rows_valid && at.col_base < gp.p.N && (BN == 256 || at.half == 0))
    *q.scale(at.row_base + lane, at.col_base >> 7, at.batch) = unit;
  const auto place = [&](int row, int piece) {
    return stg + row * (16 * kPieces) + ((kPieces == 8 ? piece ^ (row & 7) : piece ^ ((row >> 1) & 3)) << 4);
  };
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 a = __fmul2_rn(acc[8 * i + 2 * j], make_float2(factor, factor));
      const float2 b = __fmul2_rn(acc[8 * i + 2 * j + 1], make_float2(factor, factor));
      w[j] = pack4<E5M2>(a.x, a.y, b.x, b.y);
    }
    ptx::st_shared_v4(place(lane, i), make_uint4(w[0], w[1], w[2], w[3]));
  }
  __syncwarp();
  const int piece = lane % kPieces;
  const int32_t n = gp.p.N - at.col_base - 16 * piece;  // (a multiple of 8)
  uint8_t* out = q.codes + at.batch * q.batch + at.row_base * q.ld + at.col_base + 16 * piece;
#pragma unroll
  for (int j = 0; j < kPieces; ++j) {
    const int r = j * (32 / kPieces) + lane / kPieces;
    const uint4 v = ptx::ld_shared_v4(place(r, piece));
    if (r >= at.rows_valid) continue;
    if (n >= 16) *reinterpret_cast<uint4*>(out + r * q.ld) = v;
    else if (n >= 8) *reinterpret_cast<uint2*>(out + r * q.ld) = make_uint2(v.x, v.y);
  }
  __syncwarp();  // the buffer is free again
}

// D and PostAct of the thread's columns from the sums in `acc` (which they replace).
// Warp-collective; false after a wait that ran out.
template <int BN, int P>
__device__ __forceinline__ bool finish(const GemmParams& gp, const Shared& sh, const Rings& rg, const Spot& at,
                                       float2 (&acc)[P], float alpha, float beta, uint32_t stg, uint32_t& use) {
  constexpr int kChunks = P / 16;
  const Params& p = gp.p;
  if (!has_c(gp) && p.post == nullptr && gp.d8.codes == nullptr && gp.p8.codes == nullptr) {  // D alone
#pragma unroll
    for (int c = 0; c < kChunks; ++c) {
      if (at.col_base + 32 * c >= p.N) break;
#pragma unroll
      for (int j = 0; j < 16; ++j) acc[16 * c + j] = __fmul2_rn(acc[16 * c + j], make_float2(alpha, alpha));
      store32(stg, acc + 16 * c, p.d_dtype, p.d, p.ldd, p.sbd, at.batch, at.row_base, at.rows_valid,
              at.col_base + 32 * c, p.N);
    }
    return true;
  }
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
    float top = 0.f;
    CRegs c_raw = {};  // (the next chunk's come while this one is stored)
    if (reads_c && there && at.col_base < p.N) fetch_c(gp, row, at.col_base, at.batch, c_raw);
#pragma unroll 1
    for (int c = 0; c < kChunks; ++c) {
      const int32_t col0 = at.col_base + 32 * c;
      if (reads_c) {
        const bool here = there && col0 < p.N;
        const float unit = gp.c8.codes != nullptr && here ? *gp.c8.scale(row, col0 >> 7, at.batch) : 0.f;
        const char* crow = gp.c8.codes == nullptr && p.c_dtype == DT_F32 && here
                               ? reinterpret_cast<const char*>(static_cast<const float*>(p.c) + at.batch * p.sbc +
                                                               row * p.ldc + col0)
                               : nullptr;
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[8];
          c_numbers8(gp, c_raw, unit, crow, col0, g, x);
          float2* v = acc + 4 * g;
          if (!p.dact) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              v[j] = __ffma2_rn(make_float2(beta, beta), make_float2(x[2 * j], x[2 * j + 1]),
                                __fmul2_rn(v[j], make_float2(alpha, alpha)));
          } else if (pass == 0) {
            dact8(p.act, x, v);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_float2(x[2 * j], x[2 * j + 1]);
          }
        }
        if (here && c + 1 < kChunks && col0 + 32 < p.N) fetch_c(gp, row, col0 + 32, at.batch, c_raw);
      } else if (pass == 0) {
#pragma unroll
        for (int j = 0; j < 16; ++j) acc[j] = __fmul2_rn(acc[j], make_float2(alpha, alpha));
      }
      if (pass == 1) act32(p.act, acc);
      if (q.codes != nullptr && col0 < p.N) {
        // (columns past N are zeros: within a chunk N ends at a multiple of 8)
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (col0 + 2 * j < p.N) top = mx::max_abs(mx::max_abs(top, acc[j].x), acc[j].y);
      }
      if (out != nullptr && col0 < p.N) {
        if (pass == 0) store32(stg, acc, p.d_dtype, p.d, p.ldd, p.sbd, at.batch, at.row_base, at.rows_valid, col0, p.N);
        else store32(stg, acc, p.p_dtype, p.post, p.ldp, p.sbp, at.batch, at.row_base, at.rows_valid, col0, p.N);
      }
      move_round(acc);
    }
    if constexpr (BN >= 128) {
      if (q.codes != nullptr) {
        uint32_t amax = mx::abs_bits(top);
        if (!join_halves<BN>(gp, sh, rg, at, use, amax)) return false;
        if (q.e5m2) store_codes<BN, true>(gp, q, at, acc, amax, stg);
        else store_codes<BN, false>(gp, q, at, acc, amax, stg);
      }
    }
  }
  return true;
}

// ------------------------------------------------------------ tiles split along K

// The two halves of a cluster barrier.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }

// A tile's eight pieces (a warp's 32 rows x half of the columns) are dealt out to the cluster's
// CTAs in order.
__device__ __forceinline__ uint32_t piece_owner(int quad, int half, int32_t splits) {
  return static_cast<uint32_t>((quad * 2 + half) * splits) >> 3;
}
// Where rank `from` leaves a piece in its owner's shared memory: one float4 a lane and four
// columns, so each store writes 512 contiguous bytes.
template <int HALF>
__device__ __forceinline__ uint32_t piece_slot(uint32_t red, int quad, int half, uint32_t owner, uint32_t from,
                                               int32_t splits) {
  const int mine = 8 / splits;
  const uint32_t order = from < owner ? from : from - 1;
  return red + (order * mine + (quad * 2 + half) % mine) * (HALF * 128u) + (threadIdx.x & 31) * 16u;
}

template <int HALF>
__device__ __forceinline__ void send_piece(const GemmParams& gp, int quad, int half, uint32_t slice, uint32_t red,
                                           const float2 (&acc)[HALF / 2]) {
  const uint32_t owner = piece_owner(quad, half, gp.splits);
  const uint32_t dst = ptx::mapa(piece_slot<HALF>(red, quad, half, owner, slice, gp.splits), owner);
#pragma unroll
  for (int i = 0; i < HALF / 4; ++i)
    asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + i * 512u), "f"(acc[2 * i].x),
                 "f"(acc[2 * i].y), "f"(acc[2 * i + 1].x), "f"(acc[2 * i + 1].y)
                 : "memory");
}

// The ranks' sums, added in rank order.
template <int HALF>
__device__ __forceinline__ void join_piece(const GemmParams& gp, int quad, int half, uint32_t slice, uint32_t red,
                                           float2 (&acc)[HALF / 2]) {
  float2 sum[HALF / 2];
#pragma unroll
  for (int i = 0; i < HALF / 2; ++i) sum[i] = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int32_t r = 0; r < gp.splits; ++r) {
    if (r == static_cast<int32_t>(slice)) {
#pragma unroll
      for (int i = 0; i < HALF / 2; ++i) sum[i] = __fadd2_rn(sum[i], acc[i]);
    } else {
      const uint32_t src = piece_slot<HALF>(red, quad, half, slice, static_cast<uint32_t>(r), gp.splits);
#pragma unroll
      for (int i = 0; i < HALF / 4; ++i) {
        const uint4 v = ptx::ld_shared_v4(src + i * 512u);
        sum[2 * i] = __fadd2_rn(sum[2 * i], make_float2(__uint_as_float(v.x), __uint_as_float(v.y)));
        sum[2 * i + 1] = __fadd2_rn(sum[2 * i + 1], make_float2(__uint_as_float(v.z), __uint_as_float(v.w)));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < HALF / 2; ++i) acc[i] = sum[i];
}

// The warps that hold the sums.
template <int BN, int CG, bool BV>
__device__ __forceinline__ void hold_role(const GemmParams& gp, const Shared& sh, const Rings& rg, uint32_t tmem_base,
                                          uint32_t rank, uint32_t stg, int32_t unit, int32_t units, int32_t num_tiles,
                                          uint32_t slice, uint32_t red) {
  using Cfg = GemmCfg<BN, CG, BV>;
  constexpr int kHalf = Cfg::kHalf;
  const Params& p = gp.p;
  const int warp = threadIdx.x >> 5;
  const int quad = warp & 3, half = warp >> 2;
  const KSpan ks = k_span(gp, slice);
  const uint32_t tmem = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + half * kHalf;
  const float alpha = p.dact ? 1.f : (p.alpha_dev ? *p.alpha_dev : p.alpha);
  const float beta = p.beta_dev ? *p.beta_dev : p.beta;
  const bool split = CG == 1 && gp.splits > 1;
  Place at{0, 0, 0u, 0u};
  uint32_t use = 0;
  bool waited = false;  // (for the cluster's start)
  for (int32_t t = unit; t < num_tiles; t += units) {
    const TileCoord tc = tile_coord<BN, Cfg::kTileM>(t, p, sh);
    Spot spot;
    spot.row_base = tc.m_row0 + static_cast<int32_t>(rank) * kBM + quad * 32;
    spot.rows_valid = min(32, tc.row_limit - spot.row_base);
    spot.col_base = tc.n0 + half * kHalf;
    spot.batch = p.num_groups > 0 ? 0 : tc.batch;
    spot.quad = quad;
    spot.half = half;
    const bool idle = spot.rows_valid <= 0;
    float2 acc[kHalf / 2];
#pragma unroll
    for (int i = 0; i < kHalf / 2; ++i) acc[i] = make_float2(0.f, 0.f);
    if (!add_blocks<BN, CG, BV>(gp, sh, rg, tmem, quad, half, ks, t, idle, at, acc)) break;
    if constexpr (CG == 1) {
      if (split) {  // (one tile a cluster)
        cluster_wait();  // every CTA of the cluster runs: their shared memory may be written
        waited = true;
        const bool mine = piece_owner(quad, half, gp.splits) == slice;
        if (!mine && !idle) send_piece<kHalf>(gp, quad, half, slice, red, acc);
        cluster_arrive();
        cluster_wait();  // every rank's pieces are where they belong
        if (*sh.abort || !mine || idle) break;
        join_piece<kHalf>(gp, quad, half, slice, red, acc);
      }
    }
    if (!idle && !finish<BN>(gp, sh, rg, spot, acc, alpha, beta, stg, use)) break;
    if (split) break;
  }
  if (split && !waited) {  // (after a wait that ran out)
    cluster_wait();
    cluster_arrive();
    cluster_wait();
  }
}

template <int BN, int CG, bool BV>
__global__ void __launch_bounds__(GemmCfg<BN, CG, BV>::kThreads, 1)
    b128_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ GemmParams gp) {
  using Cfg = GemmCfg<BN, CG, BV>;
  const Params& p = gp.p;
  extern __shared__ uint8_t smem_raw[];
  ptx::griddep_launch_dependents();
  const uint32_t raw = ptx::smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* base_ptr = smem_raw + (base - raw);
  const int S = p.stages;
  // stages | output staging | split K: the other ranks' pieces | scale ring | control | groups
  const uint32_t out_stage = base + S * Cfg::kStageBytes;
  const uint32_t red = out_stage + Cfg::kEpiWarps * p.out_stage_bytes;
  uint8_t* ring = base_ptr + S * Cfg::kStageBytes + Cfg::kEpiWarps * p.out_stage_bytes + gp.reduce_bytes;
  uint8_t* ctrl = ring + kScaleSlots * Cfg::kScaleFloats * 4;
  // (barriers: two for a stage, four buffers' two, two a scale slot, four quads, the drain)
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ctrl + 8 * (2 * kMaxStages + 8 + 2 * kScaleSlots + 5));
  int32_t* abort_flag = reinterpret_cast<int32_t*>(tmem_slot + 1);
  float* xch = reinterpret_cast<float*>(ctrl + 512);
  int32_t* prefix = reinterpret_cast<int32_t*>(ctrl + 512 + 2048);
  int32_t* cu_s = prefix + (kMaxGroups + 1);

  Shared sh = {};
  sh.full = ptx::smem_addr(ctrl);
  sh.empty = sh.full + 8 * kMaxStages;
  sh.tfull = sh.empty + 8 * kMaxStages;
  sh.tempty = sh.tfull + 8 * 4;
  Rings rg;
  rg.sfull = sh.tempty + 8 * 4;
  rg.sempty = rg.sfull + 8 * kScaleSlots;
  rg.xbar = rg.sempty + 8 * kScaleSlots;
  const uint32_t drain_bar = rg.xbar + 8 * 4;
  rg.scales = ptx::smem_addr(ring);
  rg.xch = ptx::smem_addr(xch);
  sh.abort = abort_flag;
  sh.prefix = prefix;
  sh.cu = cu_s;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = (CG == 2 || gp.splits > 1) ? ptx::cluster_ctarank() : 0u;
  const uint32_t rank = (CG == 2) ? crank : 0u;   // in the pair
  const uint32_t slice = (CG == 2) ? 0u : crank;  // of K
  const int32_t ctas = CG * gp.splits;            // of the cluster
  const int32_t unit = static_cast<int32_t>(blockIdx.x) / ctas;
  const int32_t units = static_cast<int32_t>(gridDim.x) / ctas;
  const KSpan ks = k_span(gp, slice);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      ptx::mbar_init(sh.full + 8 * s, 1);
      ptx::mbar_init(sh.empty + 8 * s, 1);
    }
    for (int b = 0; b < Cfg::kBuffers; ++b) {
      ptx::mbar_init(sh.tfull + 8 * b, 1);
      ptx::mbar_init(sh.tempty + 8 * b, Cfg::kEpiWarps * CG);
    }
    for (int s = 0; s < kScaleSlots; ++s) {
      ptx::mbar_init(rg.sfull + 8 * s, 32);
      ptx::mbar_init(rg.sempty + 8 * s, Cfg::kEpiWarps);
    }
    for (int q = 0; q < 4; ++q) ptx::mbar_init(rg.xbar + 8 * q, 2);
    ptx::mbar_init(drain_bar, 1);
    *abort_flag = 0;
    ptx::fence_barrier_init();
  }
  if (warp == Cfg::kLoadWarp && lane == 0 && p.k_tiles > 0) {
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
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
  // grouped rows: the offsets, and the tiles before each group
  if (p.num_groups > 0 && warp == 0) {
    const int G = p.num_groups;
    const int per = (G + 31) / 32;
    const int g0 = min(lane * per, G), g1 = min(g0 + per, G);
    const auto group = [&](int g, int32_t& lo, int32_t& len) {
      const int32_t from = __ldg(p.cu_seqlens + g), to = __ldg(p.cu_seqlens + g + 1);
      const bool bad = from < 0 || to > p.M || to < from;
      lo = max(from, 0);
      len = max(0, min(to, p.M) - lo);
      return bad;
    };
    int32_t mine = 0, lo, len;
    for (int g = g0; g < g1; ++g) {
      if (group(g, lo, len)) record_status(p, DEV_INDEX_RANGE, 5, g);
      mine += ((len + Cfg::kTileM - 1) / Cfg::kTileM) * p.tiles_n;
    }
    int32_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    int32_t run = incl - mine;
    for (int g = g0; g < g1; ++g) {
      group(g, lo, len);
      prefix[g] = run;
      cu_s[g] = lo;
      run += ((len + Cfg::kTileM - 1) / Cfg::kTileM) * p.tiles_n;
    }
    if (lane == 31) {
      prefix[G] = incl;
      cu_s[G] = min(max(__ldg(p.cu_seqlens + G), 0), p.M);
    }
  }
  __syncthreads();
  if (CG == 2) ptx::cluster_sync();
  if (CG == 1 && gp.splits > 1) cluster_arrive();  // (waited for before the first remote store)
  ptx::tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int32_t num_tiles = p.num_groups > 0 ? prefix[p.num_groups] : p.num_tiles;

  if (warp < Cfg::kEpiWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kHoldRegs));
    hold_role<BN, CG, BV>(gp, sh, rg, tmem_base, rank, out_stage + warp * p.out_stage_bytes, unit, units, num_tiles,
                          slice, red);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
    if (warp == Cfg::kMmaWarp) {
      if (rank == 0 && ptx::elect_one()) mma_role<BN, CG, BV>(gp, sh, base, tmem_base, ks, unit, units, num_tiles);
    } else if (warp == Cfg::kLoadWarp) {
      if (ptx::elect_one()) load_role<BN, CG, BV>(gp, sh, &tmA, &tmB, base, rank, ks, unit, units, num_tiles);
    } else if (warp == Cfg::kScaleWarp) {
      scale_role<BN, CG, BV>(gp, sh, rg, rank, ks, unit, units, num_tiles);
    }
    __syncwarp();
    if (CG == 1 && gp.splits > 1) {
      cluster_wait();
      cluster_arrive();
      cluster_wait();
    }
  }

  __syncthreads();
  // Every MMA this CTA issued has finished before TMEM is freed: its sums' holders have waited
  // for the last block's, unless a wait ran out.
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
cudaError_t launch_one(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& gp, const LaunchShape& shape,
                       cudaStream_t stream) {
  const cudaError_t e = allow_smem<b128_gemm_kernel<BN, CG, BV>>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = gemm_config<BN, CG, BV>(shape.grid, shape.smem, shape.cluster, stream, attr);
  return cudaLaunchKernelEx(&cfg, b128_gemm_kernel<BN, CG, BV>, a, b, gp);
}

// (Registers leave room for one CTA an SM, so tensor memory needs no count of its own.  The
// warpgroups' shares must add up to what a block is launched with: setmaxnreg would wait for
// the rest forever.)
template <int BN, int CG, bool BV>
int units_one(size_t smem, int cluster) {
  using Cfg = GemmCfg<BN, CG, BV>;
  cudaFuncAttributes fa = {};
  if (cudaFuncGetAttributes(&fa, b128_gemm_kernel<BN, CG, BV>) != cudaSuccess) return -1;
  if (fa.numRegs * Cfg::kThreads < kHoldRegs * Cfg::kEpiWarps * 32 + kIssueRegs * 128) return -1;
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
cudaError_t launch_tile(const CUtensorMap& a, const CUtensorMap& b, const GemmParams& gp, const LaunchShape& shape,
                        cudaStream_t stream) {
  return gp.b_rows_one ? launch_one<BN, CG, true>(a, b, gp, shape, stream)
                       : launch_one<BN, CG, false>(a, b, gp, shape, stream);
}
template <int BN, int CG>
int units_tile(bool b_rows_one, size_t smem, int cluster) {
  return b_rows_one ? units_one<BN, CG, true>(smem, cluster) : units_one<BN, CG, false>(smem, cluster);
}

#define GGE_B128_INSTANTIATE(BN, CG)                                                                     \
  template cudaError_t launch_tile<BN, CG>(const CUtensorMap&, const CUtensorMap&, const GemmParams&, \
                                           const LaunchShape&, cudaStream_t);                          \
  template int units_tile<BN, CG>(bool, size_t, int);

}  // namespace b128
}  // namespace gge
