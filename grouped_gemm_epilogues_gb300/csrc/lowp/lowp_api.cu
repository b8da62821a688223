// Host side of the low-precision entry points: argument checks and launches of
// the RMS norm, microscaled quantisation and the block-scaled product.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "lowp_host.h"
#include "lowp_launch.h"
#include "mx_launch.h"

namespace gge {
namespace {

using lowp::QuantPtrs;

int mx_block(int32_t f) { return f == GGE_NVFP4 ? 16 : 32; }
int mx_bits(int32_t f) { return f == GGE_MXFP8 ? 8 : 4; }
bool mx_known(int32_t f) { return f >= GGE_MXFP8 && f <= GGE_NVFP4; }
int64_t mx_row_bytes(int32_t f, int64_t cols) { return ceil_div(cols, 32) * 32 * mx_bits(f) / 8; }
int64_t mx_kgroups(int32_t f, int64_t cols) { return ceil_div(ceil_div(cols, mx_block(f)), 4); }

gge_status check_mx(const gge_mx_tensor& q) {
  if (!mx_known(q.format) || q.reserved != 0) return GGE_ERR_INVALID_ARG;
  if (q.rows < 0 || q.cols < 0 || q.batch < 1) return GGE_ERR_INVALID_ARG;
  if (q.rows > kMaxExtent || q.cols > kMaxCols || q.batch > 65535) return GGE_ERR_UNSUPPORTED;
  if (q.tensor_scale != nullptr && q.format != GGE_NVFP4) return GGE_ERR_INVALID_ARG;
  if (q.tensor_scale != nullptr && (reinterpret_cast<uintptr_t>(q.tensor_scale) & 3u) != 0)
    return GGE_ERR_ALIGNMENT;
  if (q.rows == 0 || q.cols == 0) return GGE_OK;
  if (q.codes == nullptr || q.scales == nullptr) return GGE_ERR_INVALID_ARG;
  const int64_t need = mx_row_bytes(q.format, q.cols);
  const int64_t block_scales = mx_kgroups(q.format, q.cols) * 512;  // of 128 rows
  if (q.stride_row < need) return GGE_ERR_INVALID_ARG;
  if (q.batch > 1 && (q.stride_batch < (q.rows - 1) * q.stride_row + need ||
                      q.scale_stride_batch < ceil_div(q.rows, 128) * block_scales ||
                      q.scale_stride_batch % block_scales != 0))
    return GGE_ERR_INVALID_ARG;
  if (!aligned16(q.codes) || q.stride_row % 16 != 0 || (q.batch > 1 && q.stride_batch % 16 != 0) ||
      (reinterpret_cast<uintptr_t>(q.scales) & 127u) != 0)
    return GGE_ERR_ALIGNMENT;
  return GGE_OK;
}

// A quantised output (and its values) as the kernels take it.
gge_status quant_ptrs(const gge_mx_tensor& q, const gge_tensor* values, QuantPtrs* out) {
  gge_status s = check_mx(q);
  if (s != GGE_OK) return s;
  std::memset(out, 0, sizeof(*out));
  out->format = q.format;
  out->codes = static_cast<uint8_t*>(q.codes);
  out->ld = q.stride_row;
  out->batch_stride = q.batch > 1 ? q.stride_batch : 0;
  out->scales = static_cast<uint8_t*>(q.scales);
  out->kgroups = mx_kgroups(q.format, q.cols);
  out->scale_batch_stride = q.batch > 1 ? q.scale_stride_batch : 0;
  out->tensor_scale = q.tensor_scale;
  if (values != nullptr) {
    s = check_values(*values, false);
    if (s != GGE_OK) return s;
    if (!same_shape(*values, q.rows, q.cols, q.batch) || !rows_apart(*values)) return GGE_ERR_INVALID_ARG;
    out->values = values->ptr;
    out->ldv = values->stride_row;
    out->values_batch_stride = values->batch > 1 ? values->stride_batch : 0;
    out->v_dtype = values->dtype;
  }
  return GGE_OK;
}

// ------------------------------------------------------------ the product

struct MxPlan {
  mx::MxParams mp;
  mx::MxMaps maps;
  LaunchShape shape;
  int tile;
  bool empty;
};

// Resident CTAs (cluster 1) or clusters, cached.
int tile_units(int32_t format, int tile, size_t smem, int cluster) {
  struct Entry { int dev, format, tile, cluster; size_t smem; int units; };
  static std::mutex mu;
  static Entry cache[256];
  static int n = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  {
    std::lock_guard<std::mutex> g(mu);
    for (int i = 0; i < n; ++i)
      if (cache[i].dev == dev && cache[i].format == format && cache[i].tile == tile &&
          cache[i].cluster == cluster && cache[i].smem == smem)
        return cache[i].units;
  }
  int units;
  {
    RelaxedCaptureMode relaxed;  // the first query may run inside a stream capture
    units = format == GGE_MXFP8   ? mx::mx_units<GGE_MXFP8>(tile, smem, cluster)
            : format == GGE_MXFP4 ? mx::mx_units<GGE_MXFP4>(tile, smem, cluster)
                                  : mx::mx_units<GGE_NVFP4>(tile, smem, cluster);
  }
  if (units > 0) {
    std::lock_guard<std::mutex> g(mu);
    if (n < 256) cache[n++] = Entry{dev, format, tile, cluster, smem, units};
  }
  return units;
}

constexpr int kFlagsTaken = FLAG_TEST_DROP_ACC_FULL | FLAG_DIRECT_STORES | FLAG_NO_SPLIT | FLAG_RASTER_N;

// One way to run a product: tile shape, CTAs that share a tile's K, shared memory.
struct MxShape {
  int tile, bn, cg, splits, stages, stage_bytes, reduce_bytes, units;
  size_t smem;
  int64_t tiles_m, tiles_n, tiles;
};

// The shape `bn` (see gge_gemm_mx_args) with K over `splits` CTAs; false if it does not
// fit or its clusters would not all run at once.
bool mx_shape(int32_t format, int64_t M, int64_t N, int64_t L, int64_t k_tiles, int bn, int splits,
              int out_stage, int max_stages, int sms, MxShape* s) {
  s->bn = bn;
  s->cg = bn == 256 ? 2 : 1;
  s->tile = bn == 256 ? mx::TILE_PAIR_256 : (bn == 128 ? mx::TILE_128 : mx::TILE_SWAP_64);
  s->splits = splits;
  const int64_t rows = bn == 64 ? N : M, cols = bn == 64 ? M : N;  // (64: A and B exchanged)
  s->tiles_m = ceil_div(rows, 128 * s->cg);
  s->tiles_n = ceil_div(cols, bn);
  s->tiles = s->tiles_m * s->tiles_n * L;
  if (splits > 1 && (s->cg == 2 || splits > k_tiles || s->tiles * splits > sms)) return false;
  const int groups = 128 * 8 / mx_bits(format) / (4 * mx_block(format));
  // codes and scales of a stage, in whole KiB (MxCfg::kStageBytes)
  s->stage_bytes = (128 * 128 + bn / s->cg * 128 + 512 * groups * (1 + (bn + 127) / 128) + 1023) / 1024 * 1024;
  // the chunks (32 x 32 fp32) that the other CTAs hand over
  s->reduce_bytes = splits > 1 ? (splits - 1) * (4 * (bn / 32) / splits) * 4096 : 0;
  const int fixed = 1024 + kCtrlBytesHost + kEpiWarpsHost * out_stage + s->reduce_bytes;
  s->stages = std::min(max_stages, (kMaxSmemOptin - fixed) / s->stage_bytes);
  if (s->stages < 2) return false;
  s->smem = static_cast<size_t>(fixed + s->stages * s->stage_bytes);
  s->units = tile_units(format, s->tile, s->smem, s->cg * splits);
  if (s->units <= 0) return false;
  return splits == 1 || s->tiles <= s->units;
}

// Estimated time (ns) of a shape: rounds of tiles, each its k-tiles and an epilogue.
// Measured a k-tile (nvfp4, mxfp8): 295 / 240 ns for 128 x 64, 365 / 275 for 128 x 128
// and 380 / 330 for 256 x 256 on a pair, which is twice the work a CTA.  A split saves
// the k-tiles but costs the exchange, about 1.7 us (16 x 8192 nvfp4, whole and split by
// two: K 512 3.5 and 5.1 us, 4096 7.4 and 7.4, 8192 12.5 and 11.0; 16 x 2048 x 8192,
// by four: 11.6 and 7.1); 128 x 128 tiles exchange twice the chunks (128 x 8192: K 512
// 4.3 and 6.9 us, 4096 8.5 and 9.2, 8192 15.1 and 14.0).
double mx_cost(const MxShape& s, int64_t k_tiles) {
  const double per_k = s.bn == 64 ? 290.0 : (s.bn == 128 ? 370.0 : 380.0);
  const double tail = s.bn == 64 ? 500.0 : (s.bn == 128 ? 900.0 : 1800.0);
  const int64_t rounds = s.splits > 1 ? 1 : ceil_div(s.tiles, s.units);
  const double exchange = s.splits == 1 ? 0.0 : (s.bn == 64 ? 2000.0 : 3300.0);
  return static_cast<double>(rounds) * (static_cast<double>(ceil_div(k_tiles, s.splits)) * per_k + tail) +
         exchange;
}

gge_status plan_mx(const gge_gemm_mx_args* a, bool dact, void* ws, size_t ws_bytes, MxPlan* out) {
  if (a == nullptr) return GGE_ERR_INVALID_ARG;
  MxPlan& pl = *out;
  std::memset(&pl, 0, sizeof(pl));
  Params& p = pl.mp.p;
  const gge_config* cfg = a->config;
  if (a->reserved != 0 || a->act < GGE_ACT_NONE || a->act > GGE_ACT_RELU_SQ) return GGE_ERR_INVALID_ARG;
  if (cfg && (cfg->flags & ~kFlagsTaken)) return GGE_ERR_UNSUPPORTED;
  if (cfg && (cfg->batch_idx_permute != nullptr || cfg->cta_group != 0)) return GGE_ERR_UNSUPPORTED;
  if (a->D == nullptr && a->PostAct == nullptr) return GGE_ERR_INVALID_ARG;
  if (dact) {
    if (a->C == nullptr || a->D == nullptr || a->act == GGE_ACT_NONE) return GGE_ERR_INVALID_ARG;
  } else if (a->PostAct == nullptr && a->act != GGE_ACT_NONE) {
    return GGE_ERR_INVALID_ARG;
  }
  gge_status s = check_mx(a->A);
  if (s != GGE_OK) return s;
  s = check_mx(a->B);
  if (s != GGE_OK) return s;
  const int32_t format = a->A.format;
  if (a->B.format != format) return GGE_ERR_UNSUPPORTED;
  const gge_tensor* o = a->D ? a->D : a->PostAct;
  const int64_t M = o->rows, N = o->cols, L = o->batch, K = a->A.cols;
  if (a->A.rows != M || a->B.rows != N || a->B.cols != K || a->A.batch != L || a->B.batch != L)
    return GGE_ERR_INVALID_ARG;
  for (const gge_tensor* t : {a->D, a->PostAct, a->C}) {
    if (t == nullptr) continue;
    s = check_mn(t, M, N, L);
    if (s != GGE_OK) return s;
    if (t != a->C && !rows_apart(*t)) return GGE_ERR_INVALID_ARG;
  }
  if (N % 8 != 0) return GGE_ERR_UNSUPPORTED;
  s = check_workspace(ws, ws_bytes);
  if (s != GGE_OK) return s;
  pl.empty = M == 0 || N == 0;
  if (pl.empty) return GGE_OK;

  const int out_es = std::max(a->D ? elem_bytes(a->D->dtype) : 0,
                              a->PostAct ? elem_bytes(a->PostAct->dtype) : 0);
  p.out_stage_bytes = cfg && (cfg->flags & FLAG_DIRECT_STORES) ? 0 : 32 * 32 * out_es;
  const int bk = 128 * 8 / mx_bits(format);
  const int64_t k_tiles = ceil_div(K, bk);
  const int want = cfg ? cfg->tile_n : 0;
  if (want != 0 && want != 256 && want != 128 && want != 64) return GGE_ERR_UNSUPPORTED;
  const int max_stages = cfg && cfg->stages > 0 ? std::min(8, static_cast<int>(cfg->stages)) : 8;
  if (max_stages < 2) return GGE_ERR_UNSUPPORTED;
  const int sms = sm_count();
  if (sms <= 0) return GGE_ERR_CUDA;
  MxShape sh{};
  double best = -1.0;
  for (int bn : {256, 128, 64}) {
    if (want != 0 && bn != want) continue;
    for (int splits = 1; splits <= 8; splits *= 2) {
      if (splits > 1 && cfg && ((cfg->flags & FLAG_NO_SPLIT) || cfg->num_ctas > 0)) break;
      MxShape one;
      if (!mx_shape(format, M, N, L, k_tiles, bn, splits, p.out_stage_bytes, max_stages, sms, &one)) {
        if (splits == 1) break;
        continue;
      }
      const double cost = mx_cost(one, k_tiles);
      if (best < 0.0 || cost < best) {
        best = cost;
        sh = one;
      }
    }
  }
  if (best < 0.0) return GGE_ERR_CUDA;  // (every shape fits; the device could not be asked)
  const int bn = sh.bn;
  const bool swap = bn == 64;
  pl.tile = sh.tile;
  const gge_mx_tensor& ka = swap ? a->B : a->A;  // the kernel's A and B
  const gge_mx_tensor& kb = swap ? a->A : a->B;
  const int64_t kM = ka.rows, kN = kb.rows;
  const int tile_m = 128 * sh.cg;
  if (sh.tiles > kMaxExtent / 8) return GGE_ERR_UNSUPPORTED;
  const int groups = bk / (4 * mx_block(format));
  const int b_tiles = static_cast<int>(ceil_div(bn, 128));
  pl.shape.smem = sh.smem;
  pl.shape.cluster = sh.cg * sh.splits;
  pl.mp.splits = sh.splits;
  pl.mp.reduce_bytes = sh.reduce_bytes;

  p.M = static_cast<int32_t>(kM);
  p.N = static_cast<int32_t>(kN);
  p.K = static_cast<int32_t>(K);
  p.L = static_cast<int32_t>(L);
  p.bk = bk;
  p.k_tiles = static_cast<int32_t>(k_tiles);
  p.stages = sh.stages;
  p.tiles_n = static_cast<int32_t>(sh.tiles_n);
  if (a->D) {
    p.d = a->D->ptr; p.ldd = a->D->stride_row; p.sbd = a->D->stride_batch; p.d_dtype = a->D->dtype;
  }
  if (a->PostAct) {
    p.post = a->PostAct->ptr; p.ldp = a->PostAct->stride_row; p.sbp = a->PostAct->stride_batch;
    p.p_dtype = a->PostAct->dtype;
  }
  if (a->C) {
    p.c = a->C->ptr; p.ldc = a->C->stride_row; p.sbc = a->C->stride_batch; p.c_dtype = a->C->dtype;
  }
  p.act = a->act;
  p.dact = dact ? 1 : 0;
  p.out_trans = swap ? 1 : 0;
  p.alpha = a->alpha;
  p.beta = a->beta;
  p.alpha_dev = a->alpha_dev;
  p.beta_dev = a->beta_dev;
  // instruction descriptor of the block-scaled kinds: operand formats (e4m3 is 0,
  // e2m1 is 1 in the 4-bit kinds), N >> 3, power-of-two scales, M >> 4; the kernel
  // adds the scale bytes' index
  const uint32_t fmt = format == GGE_MXFP8 ? 0u : 1u;
  p.idesc = (fmt << 7) | (fmt << 10) | ((static_cast<uint32_t>(bn) >> 3) << 17) |
            ((format == GGE_NVFP4 ? 0u : 1u) << 23) | ((static_cast<uint32_t>(tile_m) >> 4) << 24);
  p.flags = cfg ? cfg->flags : 0;
  p.timeout_ns = (cfg && cfg->timeout_ns) ? cfg->timeout_ns : kDefaultTimeoutNs;
  p.status = static_cast<int32_t*>(ws);
  pl.mp.tscale_a = ka.tensor_scale;
  pl.mp.tscale_b = kb.tensor_scale;

  int units = sh.units;
  if (cfg && cfg->num_ctas > 0) units = std::min(units, std::max(1, cfg->num_ctas / sh.cg));
  const bool along_n = (p.flags & FLAG_RASTER_N) != 0;
  const int band = cfg && cfg->raster_band > 0 ? cfg->raster_band
                                               : auto_band(units, tile_m, bn, along_n);
  p.sched = PlainSchedule::create(static_cast<int32_t>(sh.tiles_m), static_cast<int32_t>(sh.tiles_n),
                                  static_cast<int32_t>(L), band, along_n);
  p.num_tiles = static_cast<int32_t>(sh.tiles);
  pl.shape.grid = pl.shape.cluster * static_cast<int>(std::min<int64_t>(sh.tiles, units));
  if (K == 0) return GGE_OK;  // nothing is loaded

  const auto codes_map = [&](CUtensorMap* m, const gge_mx_tensor& q, uint32_t box_rows) {
    const uint64_t sb = q.batch > 1 ? static_cast<uint64_t>(q.stride_batch)
                                    : static_cast<uint64_t>(q.rows) * static_cast<uint64_t>(q.stride_row);
    return encode_3d(m, q.codes, 1, static_cast<uint64_t>(mx_row_bytes(format, K)),
                     static_cast<uint64_t>(q.rows), static_cast<uint64_t>(q.batch),
                     static_cast<uint64_t>(q.stride_row), sb, 128, box_rows);
  };
  // scale tiles: 256 16-bit elements each, then along K, then row tiles of all batches
  const int64_t kg = mx_kgroups(format, K);
  const auto scales_map = [&](CUtensorMap* m, const gge_mx_tensor& q, uint32_t box_tiles, int32_t* a_batch) {
    const int64_t mine = ceil_div(q.rows, 128);
    const int64_t step = q.batch > 1 ? q.scale_stride_batch / (kg * 512) : mine;
    *a_batch = static_cast<int32_t>(step);
    return encode_3d(m, q.scales, 2, 256, static_cast<uint64_t>(kg),
                     static_cast<uint64_t>(step * (q.batch - 1) + mine), 512,
                     static_cast<uint64_t>(kg) * 512, 256, static_cast<uint32_t>(groups), box_tiles,
                     false);
  };
  s = codes_map(&pl.maps.a, ka, 128);
  if (s == GGE_OK) s = codes_map(&pl.maps.b, kb, static_cast<uint32_t>(bn / sh.cg));
  if (s == GGE_OK) s = scales_map(&pl.maps.sa, ka, 1, &pl.mp.sfa_batch);
  if (s == GGE_OK) s = scales_map(&pl.maps.sb, kb, static_cast<uint32_t>(b_tiles), &pl.mp.sfb_batch);
  return s;
}

gge_status run_mx(const gge_gemm_mx_args* args, bool dact, void* ws, size_t ws_bytes, gge_stream_t stream) {
  MxPlan pl;
  const gge_status s = plan_mx(args, dact, ws, ws_bytes, &pl);
  if (s != GGE_OK || pl.empty) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int32_t format = args->A.format;
  return launched(format == GGE_MXFP8   ? mx::launch_mx<GGE_MXFP8>(pl.tile, pl.maps, pl.mp, pl.shape, st)
                  : format == GGE_MXFP4 ? mx::launch_mx<GGE_MXFP4>(pl.tile, pl.maps, pl.mp, pl.shape, st)
                                        : mx::launch_mx<GGE_NVFP4>(pl.tile, pl.maps, pl.mp, pl.shape, st));
}

}  // namespace
}  // namespace gge

using namespace gge;

extern "C" {

size_t gge_mx_row_bytes(int32_t format, int64_t cols) {
  if (!mx_known(format) || cols < 0) return 0;
  return static_cast<size_t>(mx_row_bytes(format, cols));
}

size_t gge_mx_scale_bytes(int32_t format, int64_t rows, int64_t cols) {
  if (!mx_known(format) || rows < 0 || cols < 0) return 0;
  return static_cast<size_t>(ceil_div(rows, 128)) * static_cast<size_t>(mx_kgroups(format, cols)) * 512;
}

gge_status gge_mx_quantize(const gge_tensor* x, const gge_mx_tensor* q, const gge_tensor* values,
                           gge_stream_t stream) {
  if (x == nullptr || q == nullptr) return GGE_ERR_INVALID_ARG;
  gge_status s = check_values(*x, true);
  if (s != GGE_OK) return s;
  lowp::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  s = quant_ptrs(*q, values, &p.q);
  if (s != GGE_OK) return s;
  if (!same_shape(*x, q->rows, q->cols, q->batch)) return GGE_ERR_INVALID_ARG;
  if (x->rows == 0 || x->cols == 0) return GGE_OK;
  p.rows = x->rows;
  p.cols = x->cols;
  p.batch = x->batch;
  p.dtype = x->dtype;
  p.x = x->ptr;
  p.stride_row = x->stride_row;
  p.stride_col = x->stride_col;
  p.stride_batch = x->batch > 1 ? x->stride_batch : 0;
  p.aligned = x->cols == 1 || x->stride_col == 1
                  ? rows_aligned(*x) && (values == nullptr || rows_aligned(*values))
                  : aligned16(x->ptr) && x->stride_col * elem_bytes(x->dtype) % 16 == 0 &&
                        (x->batch <= 1 || x->stride_batch * elem_bytes(x->dtype) % 16 == 0);
  // (a transposed view takes the rows' tiles as a second grid dimension)
  if (x->cols != 1 && x->stride_col != 1 && x->rows > 65535 * int64_t(64)) return GGE_ERR_UNSUPPORTED;
  return launched(lowp::launch_quantize(p, reinterpret_cast<cudaStream_t>(stream)));
}

gge_status gge_mx_dequantize(const gge_mx_tensor* q, const gge_tensor* y, gge_stream_t stream) {
  if (q == nullptr || y == nullptr) return GGE_ERR_INVALID_ARG;
  gge_status s = check_mx(*q);
  if (s != GGE_OK) return s;
  s = check_values(*y, false);
  if (s != GGE_OK) return s;
  if (!same_shape(*y, q->rows, q->cols, q->batch) || !rows_apart(*y)) return GGE_ERR_INVALID_ARG;
  if (q->rows == 0 || q->cols == 0) return GGE_OK;
  lowp::DequantParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = q->rows;
  p.cols = q->cols;
  p.batch = q->batch;
  p.format = q->format;
  p.codes = static_cast<const uint8_t*>(q->codes);
  p.scales = static_cast<const uint8_t*>(q->scales);
  p.ld = q->stride_row;
  p.batch_stride = q->batch > 1 ? q->stride_batch : 0;
  p.kgroups = mx_kgroups(q->format, q->cols);
  p.scale_batch_stride = q->batch > 1 ? q->scale_stride_batch : 0;
  p.tensor_scale = q->tensor_scale;
  p.y = y->ptr;
  p.ldy = y->stride_row;
  p.y_batch_stride = y->batch > 1 ? y->stride_batch : 0;
  p.dtype = y->dtype;
  p.aligned = rows_aligned(*y) ? 1 : 0;
  return launched(lowp::launch_dequantize(p, reinterpret_cast<cudaStream_t>(stream)));
}

gge_status gge_gemm_mx(const gge_gemm_mx_args* args, void* ws, size_t ws_bytes, gge_stream_t stream) {
  return run_mx(args, false, ws, ws_bytes, stream);
}

gge_status gge_gemm_mx_dact(const gge_gemm_mx_args* args, void* ws, size_t ws_bytes, gge_stream_t stream) {
  return run_mx(args, true, ws, ws_bytes, stream);
}

gge_status gge_rmsnorm(const gge_rmsnorm_args* a, gge_stream_t stream) {
  if (a == nullptr) return GGE_ERR_INVALID_ARG;
  const gge_tensor& x = a->x;
  gge_status s = check_values(x, false);
  if (s != GGE_OK) return s;
  if (x.batch != 1) return GGE_ERR_UNSUPPORTED;
  if (!is_value_type(a->weight_dtype)) return GGE_ERR_UNSUPPORTED;
  lowp::NormParams p;
  std::memset(&p, 0, sizeof(p));
  p.q.format = 3;  // no quantised output
  bool aligned = rows_aligned(x) && (a->values == nullptr || rows_aligned(*a->values));
  bool alike = a->q == nullptr;
  const auto take = [&](const gge_tensor* t, bool output) {
    if (t == nullptr) return GGE_OK;
    const gge_status r = check_values(*t, false);
    if (r != GGE_OK) return r;
    if (t->dtype != x.dtype) return GGE_ERR_UNSUPPORTED;
    if (!same_shape(*t, x.rows, x.cols, 1) || (output && !rows_apart(*t))) return GGE_ERR_INVALID_ARG;
    aligned = aligned && rows_aligned(*t);
    alike = alike && rows_alike(*t, x);
    return GGE_OK;
  };
  if ((s = take(a->residual, false)) != GGE_OK) return s;
  if ((s = take(a->residual_out, true)) != GGE_OK) return s;
  if ((s = take(a->y, true)) != GGE_OK) return s;
  if (a->residual_out != nullptr && a->residual == nullptr) return GGE_ERR_INVALID_ARG;
  if (a->values != nullptr && a->q == nullptr) return GGE_ERR_INVALID_ARG;
  if (a->q != nullptr) {
    s = quant_ptrs(*a->q, a->values, &p.q);
    if (s != GGE_OK) return s;
    if (a->q->rows != x.rows || a->q->cols != x.cols || a->q->batch != 1) return GGE_ERR_INVALID_ARG;
  }
  if (x.rows == 0 || x.cols == 0) return GGE_OK;
  if (a->weight == nullptr) return GGE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a->weight) & (elem_bytes(a->weight_dtype) - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(a->inv_rms) & 3u) != 0)
    return GGE_ERR_ALIGNMENT;
  p.rows = x.rows;
  p.cols = static_cast<int32_t>(x.cols);
  p.dtype = x.dtype;
  p.x = x.ptr;
  p.ldx = x.stride_row;
  if (a->residual) { p.residual = a->residual->ptr; p.ldr = a->residual->stride_row; }
  if (a->residual_out) { p.h = a->residual_out->ptr; p.ldh = a->residual_out->stride_row; }
  if (a->y) { p.y = a->y->ptr; p.ldy = a->y->stride_row; }
  p.weight = a->weight;
  p.w_dtype = a->weight_dtype;
  p.eps = a->eps;
  p.inv = a->inv_rms;
  p.w_vec = aligned16(a->weight) ? 1 : 0;
  p.rows_lie = aligned ? lowp::ROWS_ALIGNED : (alike ? lowp::ROWS_ALIKE : lowp::ROWS_ANY);
  const int sms = sm_count();
  if (sms <= 0) return GGE_ERR_CUDA;
  return launched(lowp::launch_norm(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gge_workspace_size_rmsnorm_bwd(int64_t cols) {
  const int sms = sm_count();
  if (sms <= 0 || cols < 0) return 0;
  return kTailBase + static_cast<size_t>(lowp::norm_bwd_blocks(kMaxExtent, sms)) *
                         static_cast<size_t>(cols) * sizeof(float);
}

gge_status gge_rmsnorm_bwd(const gge_rmsnorm_bwd_args* a, void* ws, size_t ws_bytes,
                           gge_stream_t stream) {
  if (a == nullptr || a->reserved != 0) return GGE_ERR_INVALID_ARG;
  const gge_tensor& dy = a->dy;
  gge_status s = check_values(dy, false);
  if (s != GGE_OK) return s;
  if (dy.batch != 1) return GGE_ERR_UNSUPPORTED;
  if (!is_value_type(a->weight_dtype)) return GGE_ERR_UNSUPPORTED;
  bool aligned = rows_aligned(dy), alike = true;
  for (const gge_tensor* t : {&a->h, a->dh, &a->dx}) {
    if (t == nullptr) continue;
    s = check_values(*t, false);
    if (s != GGE_OK) return s;
    if (t->dtype != dy.dtype) return GGE_ERR_UNSUPPORTED;
    if (!same_shape(*t, dy.rows, dy.cols, 1)) return GGE_ERR_INVALID_ARG;
    aligned = aligned && rows_aligned(*t);
    alike = alike && rows_alike(*t, dy);
  }
  if (!rows_apart(a->dx)) return GGE_ERR_INVALID_ARG;
  if (dy.cols == 0 || (dy.rows == 0 && a->dweight == nullptr)) return GGE_OK;
  if (a->weight == nullptr || (a->inv_rms == nullptr && dy.rows > 0)) return GGE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(a->weight) & (elem_bytes(a->weight_dtype) - 1)) != 0 ||
      (reinterpret_cast<uintptr_t>(a->inv_rms) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(a->dweight) & 3u) != 0)
    return GGE_ERR_ALIGNMENT;
  lowp::NormBwdParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = dy.rows;
  p.cols = static_cast<int32_t>(dy.cols);
  p.dtype = dy.dtype;
  p.dy = dy.ptr;
  p.lddy = dy.stride_row;
  p.h = a->h.ptr;
  p.ldh = a->h.stride_row;
  if (a->dh) { p.dh = a->dh->ptr; p.lddh = a->dh->stride_row; }
  p.dx = a->dx.ptr;
  p.lddx = a->dx.stride_row;
  p.weight = a->weight;
  p.w_dtype = a->weight_dtype;
  p.inv = a->inv_rms;
  p.dw = a->dweight;
  p.w_vec = aligned16(a->weight) ? 1 : 0;
  p.rows_lie = aligned ? lowp::ROWS_ALIGNED : (alike ? lowp::ROWS_ALIKE : lowp::ROWS_ANY);
  const int sms = sm_count();
  if (sms <= 0) return GGE_ERR_CUDA;
  if (a->dweight != nullptr) {
    if (ws == nullptr) return GGE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return GGE_ERR_ALIGNMENT;
    if (ws_bytes < kTailBase + static_cast<size_t>(lowp::norm_bwd_blocks(dy.rows, sms)) *
                                   static_cast<size_t>(dy.cols) * sizeof(float))
      return GGE_ERR_WORKSPACE;
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kTailBase);
  }
  return launched(lowp::launch_norm_bwd(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
