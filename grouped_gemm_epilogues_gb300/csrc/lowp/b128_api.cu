// Host side of the operators on 8 bits with a scale for each block of 128: argument checks and
// launches of quantisation, transposition, layer norm and the product.
#include <algorithm>
#include <cstring>
#include <mutex>

#include "b128_launch.h"
#include "lowp_host.h"

namespace gge {
namespace {

using b128::View;

// The same rules as rows_apart, for up to three strides: no two indices share a place.
bool scales_apart(int64_t e0, int64_t s0, int64_t e1, int64_t s1, int64_t e2, int64_t s2) {
  int64_t e[3] = {e0, e1, e2}, s[3] = {s0, s1, s2};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (s[j] > s[j + 1]) std::swap(s[j], s[j + 1]), std::swap(e[j], e[j + 1]);
  int64_t span = 0;  // the last place of the dimensions so far
  for (int i = 0; i < 3; ++i) {
    if (e[i] <= 1) continue;
    if (s[i] <= span) return false;
    span += (e[i] - 1) * s[i];
  }
  return true;
}

gge_status check_b128(const gge_b128_tensor& q, bool output) {
  if (q.dtype != GGE_E4M3 && q.dtype != GGE_E5M2) return GGE_ERR_UNSUPPORTED;
  if (q.block_rows != 1 && q.block_rows != 128) return GGE_ERR_UNSUPPORTED;
  if (q.rows < 0 || q.cols < 0 || q.batch < 1) return GGE_ERR_INVALID_ARG;
  if (q.rows > kMaxCols || q.cols > kMaxCols || q.batch > 65535) return GGE_ERR_UNSUPPORTED;
  if (q.rows == 0 || q.cols == 0) return GGE_OK;
  if (q.codes == nullptr || q.scales == nullptr) return GGE_ERR_INVALID_ARG;
  const int64_t span = (q.rows - 1) * q.stride_row + q.cols;
  if (q.rows > 1 && q.stride_row < q.cols) return GGE_ERR_INVALID_ARG;
  if (q.batch > 1 && q.stride_batch < (q.rows > 1 ? span : q.cols)) return GGE_ERR_INVALID_ARG;
  if (q.scale_stride_row < 0 || q.scale_stride_col < 0 || q.scale_stride_batch < 0) return GGE_ERR_INVALID_ARG;
  if (output && !scales_apart(ceil_div(q.rows, q.block_rows), q.scale_stride_row, ceil_div(q.cols, 128),
                              q.scale_stride_col, q.batch, q.scale_stride_batch))
    return GGE_ERR_INVALID_ARG;
  if (!aligned16(q.codes) || (q.rows > 1 && q.stride_row % 16 != 0) || (q.batch > 1 && q.stride_batch % 16 != 0) ||
      (reinterpret_cast<uintptr_t>(q.scales) & 3u) != 0)
    return GGE_ERR_ALIGNMENT;
  return GGE_OK;
}

bool shape_is(const gge_b128_tensor& q, int64_t rows, int64_t cols, int64_t batch) {
  return q.rows == rows && q.cols == cols && q.batch == batch;
}

View view_of(const gge_b128_tensor& q) {
  return View{static_cast<uint8_t*>(q.codes), q.scales, q.rows > 1 ? q.stride_row : (q.cols + 15) / 16 * 16,
              q.batch > 1 ? q.stride_batch : 0, q.scale_stride_row, q.scale_stride_col,
              q.batch > 1 ? q.scale_stride_batch : 0, q.block_rows == 128 ? 7 : 0, q.dtype == GGE_E5M2 ? 1 : 0};
}

gge_status take_values(const gge_tensor* values, int64_t rows, int64_t cols, int64_t batch,
                       b128::QuantParams* p) {
  if (values == nullptr) return GGE_OK;
  const gge_status s = check_values(*values, false);
  if (s != GGE_OK) return s;
  if (!same_shape(*values, rows, cols, batch) || !rows_apart(*values)) return GGE_ERR_INVALID_ARG;
  p->values = values->ptr;
  p->ldv = values->stride_row;
  p->v_batch = values->batch > 1 ? values->stride_batch : 0;
  p->v_dtype = values->dtype;
  p->v_aligned = rows_aligned(*values) ? 1 : 0;
  return GGE_OK;
}

// ------------------------------------------------------------ the product

struct GemmPlan {
  b128::GemmParams gp;
  b128::GemmMaps maps;
  LaunchShape shape;
  int tile;
  bool empty;
};

int shape_units(int tile, bool bv, size_t smem, int cluster) {
  return tile == 256   ? b128::units_tile<256, 2>(bv, smem, cluster)
         : tile == 128 ? b128::units_tile<128, 1>(bv, smem, cluster)
                       : b128::units_tile<64, 1>(bv, smem, cluster);
}

// Resident CTAs (cluster 1) or clusters, cached.
int tile_units(int tile, bool bv, size_t smem, int cluster) {
  struct Entry { int dev, tile, cluster; bool bv; size_t smem; int units; };
  static std::mutex mu;
  static Entry cache[256];
  static int n = 0;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  {
    std::lock_guard<std::mutex> g(mu);
    for (int i = 0; i < n; ++i)
      if (cache[i].dev == dev && cache[i].tile == tile && cache[i].bv == bv && cache[i].cluster == cluster &&
          cache[i].smem == smem)
        return cache[i].units;
  }
  int units;
  {
    RelaxedCaptureMode relaxed;  // the first query may run inside a stream capture
    units = shape_units(tile, bv, smem, cluster);
  }
  if (units > 0) {
    std::lock_guard<std::mutex> g(mu);
    if (n < 256) cache[n++] = Entry{dev, tile, cluster, bv, smem, units};
  }
  return units;
}

constexpr int kFlagsTaken = FLAG_TEST_DROP_ACC_FULL | FLAG_NO_SPLIT | FLAG_RASTER_N;
constexpr int kMaxGroupsHost = 1024;

// One way to run a product: tile shape (256 x 256 on a CTA pair, 128 x 128 or 128 x 64 on one
// CTA), CTAs that share a tile's K, shared memory.
struct Shape {
  int a_rows, bn, cg, splits, stages, stage_bytes, units;
  size_t smem;
  int64_t tiles_m, tiles_n, tiles;  // (grouped rows: tiles_m and tiles as expected)
};

struct Problem {
  int64_t M, N, L, k_tiles;
  int groups;
  bool bv, codes_out;
  int out_stage, wide_stage, max_stages, sms;
};

bool try_shape(const Problem& q, int bn, int splits, Shape* s) {
  s->bn = bn;
  s->cg = bn == 256 ? 2 : 1;
  s->splits = splits;
  s->tiles_m = ceil_div(q.M, 128 * s->cg) + q.groups / 2;
  s->tiles_n = ceil_div(q.N, bn);
  s->tiles = s->tiles_m * s->tiles_n * (q.groups > 0 ? 1 : q.L);
  if (splits > 1 && (s->cg == 2 || splits > q.k_tiles || s->tiles * splits > q.sms)) return false;
  s->a_rows = bn < 256 && q.groups == 0 && q.M <= b128::kFewRows ? b128::kFewRows : 128;
  s->stage_bytes = (s->a_rows + bn / s->cg) * 128;
  const int ring = 2 * 8 * (128 + (q.bv ? std::max(bn, 128) : 4)) * 4;  // (kScaleSlots, kSlotBytes)
  const int outputs = bn == 256 ? 8 * q.wide_stage : 128 * bn * 4 + 4 * q.out_stage;  // (a tile's sums, staging)
  const int fixed = 1024 + 512 + outputs + ring +
                    (q.groups > 0 ? 2 * (kMaxGroupsHost + 1) * 4 : 0);
  s->stages = std::min(q.max_stages, (kMaxSmemOptin - fixed) / s->stage_bytes);
  if (s->stages < 2) return false;
  s->smem = static_cast<size_t>(fixed + s->stages * s->stage_bytes);
  s->units = tile_units(bn, q.bv, s->smem, s->cg * splits);
  if (s->units <= 0) return false;
  return splits == 1 || s->tiles <= s->units;
}

// Estimated time (ns) of a shape, from measured products: a block of K costs 400, 345 or 245 with
// tiles 256, 128 or 64 wide, more with a scale for each row of B; a 256-wide tile's outputs are
// made between its K and the next one's, small tiles' beside it; ranks that split K exchange sums.
// (Two rounds of 256 x 256 tiles, 4096 x 1536 x 16384 with a scale for each row: 193 us; three
// rounds of 128 x 128: 175.)
double cost(const Shape& s, const Problem& q) {
  const double per_k = s.bn == 64 ? (q.bv ? 295.0 : 245.0)
                       : s.bn == 128 ? (q.bv ? 440.0 : s.a_rows < 128 ? 240.0 : 345.0)
                                     : (q.bv ? 700.0 : 400.0);
  const int64_t rounds = s.splits > 1 ? 1 : ceil_div(s.tiles, s.units);
  const double outputs = s.bn == 256 ? 2000.0 * static_cast<double>(rounds) : 1500.0;
  const double exchange = s.splits == 1 ? 0.0 : 2500.0;
  return static_cast<double>(rounds) * static_cast<double>(ceil_div(q.k_tiles, s.splits)) * per_k + outputs + exchange;
}

// One of C, D and PostAct in either form.
gge_status check_out(const gge_tensor* t, const gge_b128_tensor* q, int64_t M, int64_t N, int64_t L, bool output) {
  if (t != nullptr && q != nullptr) return GGE_ERR_INVALID_ARG;
  if (t != nullptr) {
    const gge_status s = check_mn(t, M, N, L);
    if (s != GGE_OK) return s;
    if (output && !rows_apart(*t)) return GGE_ERR_INVALID_ARG;
  }
  if (q != nullptr) {
    const gge_status s = check_b128(*q, output);
    if (s != GGE_OK) return s;
    if (!shape_is(*q, M, N, L)) return GGE_ERR_INVALID_ARG;
    if (q->block_rows != 1) return GGE_ERR_UNSUPPORTED;
  }
  return GGE_OK;
}

gge_status plan_b128(const gge_gemm_b128_args* a, bool dact, void* ws, size_t ws_bytes, GemmPlan* out) {
  if (a == nullptr) return GGE_ERR_INVALID_ARG;
  GemmPlan& pl = *out;
  std::memset(&pl, 0, sizeof(pl));
  Params& p = pl.gp.p;
  const gge_config* cfg = a->config;
  if (a->act < GGE_ACT_NONE || a->act > GGE_ACT_RELU_SQ) return GGE_ERR_INVALID_ARG;
  if (cfg && (cfg->flags & ~kFlagsTaken)) return GGE_ERR_UNSUPPORTED;
  if (cfg && (cfg->batch_idx_permute != nullptr || cfg->cta_group != 0)) return GGE_ERR_UNSUPPORTED;
  const bool has_d = a->D != nullptr || a->D8 != nullptr, has_p = a->PostAct != nullptr || a->PostAct8 != nullptr;
  if (!has_d && !has_p) return GGE_ERR_INVALID_ARG;
  if (dact) {
    if ((a->C == nullptr && a->C8 == nullptr) || !has_d || a->act == GGE_ACT_NONE) return GGE_ERR_INVALID_ARG;
  } else if (!has_p && a->act != GGE_ACT_NONE) {
    return GGE_ERR_INVALID_ARG;
  }
  gge_status s = check_b128(a->A, false);
  if (s != GGE_OK) return s;
  s = check_b128(a->B, false);
  if (s != GGE_OK) return s;
  const int32_t G = a->num_groups;
  if (G < 0 || (G > 0) != (a->cu_seqlens_m != nullptr)) return GGE_ERR_INVALID_ARG;
  if (G > kMaxGroupsHost) return GGE_ERR_UNSUPPORTED;
  if ((reinterpret_cast<uintptr_t>(a->cu_seqlens_m) & 3u) != 0) return GGE_ERR_ALIGNMENT;
  const int64_t M = a->A.rows, N = a->B.rows, L = a->A.batch, K = a->A.cols;
  if (a->B.cols != K || a->B.batch != (G > 0 ? G : L) || (G > 0 && L != 1)) return GGE_ERR_INVALID_ARG;
  if ((s = check_out(a->C, a->C8, M, N, L, false)) != GGE_OK) return s;
  if ((s = check_out(a->D, a->D8, M, N, L, true)) != GGE_OK) return s;
  if ((s = check_out(a->PostAct, a->PostAct8, M, N, L, true)) != GGE_OK) return s;
  if (N % 8 != 0) return GGE_ERR_UNSUPPORTED;
  pl.empty = M == 0 || N == 0;
  if (dact && !pl.empty) {  // C is read again after D is written
    const void* c = a->C ? a->C->ptr : a->C8->codes;
    for (const gge_tensor* t : {a->D, a->PostAct})
      if (t != nullptr && t->ptr == c) return GGE_ERR_INVALID_ARG;
    for (const gge_b128_tensor* t : {a->D8, a->PostAct8})
      if (t != nullptr && t->codes == c) return GGE_ERR_INVALID_ARG;
  }
  s = check_workspace(ws, ws_bytes);
  if (s != GGE_OK) return s;
  if (pl.empty) return GGE_OK;

  const int out_es = std::max(a->D ? elem_bytes(a->D->dtype) : 0, a->PostAct ? elem_bytes(a->PostAct->dtype) : 0);
  Problem q{};
  q.M = M, q.N = N, q.L = L, q.groups = G;
  q.k_tiles = ceil_div(K, 128);
  q.bv = a->B.block_rows == 1;
  q.codes_out = a->D8 != nullptr || a->PostAct8 != nullptr;
  q.out_stage = out_es == 4 || q.codes_out ? 4096 : 2048;
  // 16- and 8-bit outputs of 256-wide tiles leave by TMA, up to three chunks of a warp on their way
  const bool c_read = a->C != nullptr || a->C8 != nullptr;
  const auto by_tma = [&](const gge_tensor* t) {
    return t != nullptr && !c_read && elem_bytes(t->dtype) == 2 && M > 1 && aligned16(t->ptr) && t->stride_row % 8 == 0 &&
           (L == 1 || t->stride_batch % 8 == 0);
  };
  // (a row's end is exact to 16 bytes only: 72 columns of codes wrote 80)
  const bool codes_tma = !c_read && M > 1 && N % 16 == 0;
  const int tma = (by_tma(a->D) ? 1 : 0) | (by_tma(a->PostAct) ? 2 : 0) | (a->D8 && codes_tma ? 4 : 0) |
                  (a->PostAct8 && codes_tma ? 8 : 0);
  q.wide_stage = (tma & 3) != 0 ? 3 * 2048 : q.out_stage;
  const int want = cfg ? cfg->tile_n : 0;
  if (want != 0 && want != 256 && want != 128 && (want != 64 || q.codes_out)) return GGE_ERR_UNSUPPORTED;
  q.max_stages = cfg && cfg->stages > 0 ? std::min(8, static_cast<int>(cfg->stages)) : 16;
  if (q.max_stages < 2) return GGE_ERR_UNSUPPORTED;
  q.sms = sm_count();
  if (q.sms <= 0) return GGE_ERR_CUDA;
  Shape sh{};
  double best = -1.0;
  for (int tile : {256, 128, 64}) {
    if ((want != 0 && tile != want) || (tile == 64 && q.codes_out)) continue;
    for (int splits = 1; splits <= 4; splits *= 2) {
      if (splits > 1 && (G > 0 || (cfg && ((cfg->flags & FLAG_NO_SPLIT) || cfg->num_ctas > 0)))) break;
      Shape one;
      if (!try_shape(q, tile, splits, &one)) {
        if (splits == 1) break;
        continue;
      }
      const double c = cost(one, q);
      if (best < 0.0 || c < best) {
        best = c;
        sh = one;
      }
    }
  }
  if (best < 0.0) return GGE_ERR_CUDA;  // (every shape fits; the device could not be asked)
  const int tile_m = 128 * sh.cg;
  if (sh.tiles > kMaxExtent / 8) return GGE_ERR_UNSUPPORTED;
  pl.tile = sh.bn;
  pl.shape.smem = sh.smem;
  pl.shape.cluster = sh.cg * sh.splits;
  pl.gp.splits = sh.splits;
  pl.gp.a_rows = sh.a_rows;
  pl.gp.b_rows_one = q.bv ? 1 : 0;
  pl.gp.a = view_of(a->A);
  pl.gp.b = view_of(a->B);
  if (a->C8) pl.gp.c8 = view_of(*a->C8);
  if (a->D8) pl.gp.d8 = view_of(*a->D8);
  if (a->PostAct8) pl.gp.p8 = view_of(*a->PostAct8);

  p.M = static_cast<int32_t>(M);
  p.N = static_cast<int32_t>(N);
  p.K = static_cast<int32_t>(K);
  p.L = static_cast<int32_t>(L);
  p.bk = 128;
  p.k_tiles = static_cast<int32_t>(q.k_tiles);
  p.stages = sh.stages;
  p.tiles_n = static_cast<int32_t>(sh.tiles_n);
  p.num_groups = G;
  p.cu_seqlens = a->cu_seqlens_m;
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
  p.alpha = a->alpha;
  p.beta = a->beta;
  p.alpha_dev = a->alpha_dev;
  p.beta_dev = a->beta_dev;
  p.out_stage_bytes = sh.bn == 256 ? q.wide_stage : q.out_stage;
  pl.gp.by_tma = sh.bn == 256 ? tma : 0;
  p.f8 = 1;
  // instruction descriptor: fp32 sums, operand types (e4m3 is 0, e5m2 is 1), N >> 3, M >> 4
  p.idesc = (1u << 4) | ((a->A.dtype == GGE_E5M2 ? 1u : 0u) << 7) | ((a->B.dtype == GGE_E5M2 ? 1u : 0u) << 10) |
            ((static_cast<uint32_t>(sh.bn) >> 3) << 17) | ((static_cast<uint32_t>(tile_m) >> 4) << 24);
  p.flags = cfg ? cfg->flags : 0;
  p.timeout_ns = (cfg && cfg->timeout_ns) ? cfg->timeout_ns : kDefaultTimeoutNs;
  p.status = static_cast<int32_t*>(ws);

  int units = sh.units;
  if (cfg && cfg->num_ctas > 0) units = std::min(units, std::max(1, cfg->num_ctas / sh.cg));
  int64_t most = sh.tiles;  // tiles there can be
  if (G > 0) {
    most = (ceil_div(M, tile_m) + G) * sh.tiles_n;
    if (most > kMaxExtent / 8) return GGE_ERR_UNSUPPORTED;
    p.tiles_n_div = FastDivmod::create(p.tiles_n);
  } else {
    const bool along_n = (p.flags & FLAG_RASTER_N) != 0;
    const int band = cfg && cfg->raster_band > 0 ? cfg->raster_band : auto_band(units, tile_m, sh.bn, along_n);
    p.sched = PlainSchedule::create(static_cast<int32_t>(sh.tiles_m), static_cast<int32_t>(sh.tiles_n),
                                    static_cast<int32_t>(L), band, along_n);
    p.num_tiles = static_cast<int32_t>(sh.tiles);
  }
  pl.shape.grid = pl.shape.cluster * static_cast<int>(std::min<int64_t>(most, units));
  if (K == 0) {  // nothing is loaded
    pl.gp.by_tma = 0;
    return GGE_OK;
  }

  const auto map = [&](CUtensorMap* m, const gge_b128_tensor& t, uint32_t box_rows) {
    const uint64_t ld = t.rows > 1 ? static_cast<uint64_t>(t.stride_row) : static_cast<uint64_t>((t.cols + 15) / 16 * 16);
    const uint64_t sb = t.batch > 1 ? static_cast<uint64_t>(t.stride_batch) : static_cast<uint64_t>(t.rows) * ld;
    return encode_3d(m, t.codes, 1, static_cast<uint64_t>(K), static_cast<uint64_t>(t.rows),
                     static_cast<uint64_t>(t.batch), ld, sb, 128, box_rows);
  };
  s = map(&pl.maps.a, a->A, static_cast<uint32_t>(sh.a_rows));
  if (s == GGE_OK) s = map(&pl.maps.b, a->B, static_cast<uint32_t>(sh.bn / sh.cg));
  const auto out_map = [&](CUtensorMap* m, const gge_tensor& t) {
    const uint64_t ld = static_cast<uint64_t>(t.stride_row) * 2;
    return encode_3d(m, t.ptr, 2, static_cast<uint64_t>(N), static_cast<uint64_t>(M), static_cast<uint64_t>(L), ld,
                     L > 1 ? static_cast<uint64_t>(t.stride_batch) * 2 : static_cast<uint64_t>(M) * ld, 32, 32, 1, 2);
  };
  if (s == GGE_OK && (pl.gp.by_tma & 1)) s = out_map(&pl.maps.d, *a->D);
  if (s == GGE_OK && (pl.gp.by_tma & 2)) s = out_map(&pl.maps.post, *a->PostAct);
  const auto codes_map = [&](CUtensorMap* m, const gge_b128_tensor& t) {
    const uint64_t ld = static_cast<uint64_t>(t.stride_row);
    return encode_3d(m, t.codes, 1, static_cast<uint64_t>(N), static_cast<uint64_t>(M), static_cast<uint64_t>(L), ld,
                     L > 1 ? static_cast<uint64_t>(t.stride_batch) : static_cast<uint64_t>(M) * ld, 128, 32);
  };
  if (s == GGE_OK && (pl.gp.by_tma & 4)) s = codes_map(&pl.maps.d, *a->D8);
  if (s == GGE_OK && (pl.gp.by_tma & 8)) s = codes_map(&pl.maps.post, *a->PostAct8);
  return s;
}

gge_status run_b128(const gge_gemm_b128_args* args, bool dact, void* ws, size_t ws_bytes, gge_stream_t stream) {
  GemmPlan pl;
  const gge_status s = plan_b128(args, dact, ws, ws_bytes, &pl);
  if (s != GGE_OK || pl.empty) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return launched(pl.tile == 256   ? b128::launch_tile<256, 2>(pl.maps, pl.gp, pl.shape, st)
                  : pl.tile == 128 ? b128::launch_tile<128, 1>(pl.maps, pl.gp, pl.shape, st)
                                   : b128::launch_tile<64, 1>(pl.maps, pl.gp, pl.shape, st));
}

// ------------------------------------------------------------ layer norm

// A parameter vector (NULL is fine).
bool param_aligned(const void* p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) & (elem_bytes(dtype) - 1)) == 0;
}
bool float_aligned(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

gge_status take_codes(const gge_b128_tensor* q, const gge_tensor& x, bool output, View* out) {
  if (q == nullptr) return GGE_OK;
  const gge_status s = check_b128(*q, output);
  if (s != GGE_OK) return s;
  if (!shape_is(*q, x.rows, x.cols, 1)) return GGE_ERR_INVALID_ARG;
  if (output && q->block_rows != 1) return GGE_ERR_UNSUPPORTED;
  *out = view_of(*q);
  return GGE_OK;
}

}  // namespace
}  // namespace gge

using namespace gge;

extern "C" {

gge_status gge_b128_quantize(const gge_tensor* x, const gge_b128_tensor* q, const gge_tensor* values,
                             gge_stream_t stream) {
  if (x == nullptr || q == nullptr) return GGE_ERR_INVALID_ARG;
  gge_status s = check_values(*x, true);
  if (s != GGE_OK) return s;
  s = check_b128(*q, true);
  if (s != GGE_OK) return s;
  if (!shape_is(*q, x->rows, x->cols, x->batch)) return GGE_ERR_INVALID_ARG;
  b128::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  s = take_values(values, x->rows, x->cols, x->batch, &p);
  if (s != GGE_OK) return s;
  if (x->rows == 0 || x->cols == 0) return GGE_OK;
  p.rows = x->rows;
  p.cols = x->cols;
  p.batch = x->batch;
  p.x = x->ptr;
  p.dtype = x->dtype;
  p.stride_row = x->stride_row;
  p.stride_col = x->stride_col;
  p.stride_batch = x->batch > 1 ? x->stride_batch : 0;
  p.aligned = x->cols == 1 || x->stride_col == 1
                  ? rows_aligned(*x)
                  : aligned16(x->ptr) && x->stride_col * elem_bytes(x->dtype) % 16 == 0 &&
                        (x->batch <= 1 || x->stride_batch * elem_bytes(x->dtype) % 16 == 0);
  p.q = view_of(*q);
  return launched(b128::launch_quantize(p, reinterpret_cast<cudaStream_t>(stream)));
}

gge_status gge_b128_transpose(const gge_b128_tensor* x, const gge_b128_tensor* q, const gge_tensor* values,
                              gge_stream_t stream) {
  if (x == nullptr || q == nullptr) return GGE_ERR_INVALID_ARG;
  gge_status s = check_b128(*x, false);
  if (s != GGE_OK) return s;
  s = check_b128(*q, true);
  if (s != GGE_OK) return s;
  if (!shape_is(*q, x->cols, x->rows, x->batch)) return GGE_ERR_INVALID_ARG;
  b128::QuantParams p;
  std::memset(&p, 0, sizeof(p));
  s = take_values(values, q->rows, q->cols, q->batch, &p);
  if (s != GGE_OK) return s;
  if (x->rows == 0 || x->cols == 0) return GGE_OK;
  p.rows = q->rows;
  p.cols = q->cols;
  p.batch = q->batch;
  p.x = x->codes;
  p.dtype = x->dtype;
  p.from = view_of(*x);
  p.stride_row = 1;
  p.stride_col = p.from.ld;
  p.stride_batch = p.from.batch;
  p.aligned = 1;
  p.q = view_of(*q);
  return launched(b128::launch_quantize(p, reinterpret_cast<cudaStream_t>(stream)));
}

gge_status gge_b128_dequantize(const gge_b128_tensor* q, const gge_tensor* y, gge_stream_t stream) {
  if (q == nullptr || y == nullptr) return GGE_ERR_INVALID_ARG;
  gge_status s = check_b128(*q, false);
  if (s != GGE_OK) return s;
  s = check_values(*y, false);
  if (s != GGE_OK) return s;
  if (!shape_is(*q, y->rows, y->cols, y->batch) || !rows_apart(*y)) return GGE_ERR_INVALID_ARG;
  if (q->rows == 0 || q->cols == 0) return GGE_OK;
  b128::DequantParams p;
  std::memset(&p, 0, sizeof(p));
  p.rows = q->rows;
  p.cols = q->cols;
  p.batch = q->batch;
  p.q = view_of(*q);
  p.y = y->ptr;
  p.ldy = y->stride_row;
  p.y_batch = y->batch > 1 ? y->stride_batch : 0;
  p.dtype = y->dtype;
  p.aligned = rows_aligned(*y) ? 1 : 0;
  return launched(b128::launch_dequantize(p, reinterpret_cast<cudaStream_t>(stream)));
}

gge_status gge_gemm_b128(const gge_gemm_b128_args* args, void* ws, size_t ws_bytes, gge_stream_t stream) {
  return run_b128(args, false, ws, ws_bytes, stream);
}

gge_status gge_gemm_b128_dact(const gge_gemm_b128_args* args, void* ws, size_t ws_bytes, gge_stream_t stream) {
  return run_b128(args, true, ws, ws_bytes, stream);
}

gge_status gge_layernorm(const gge_layernorm_args* a, gge_stream_t stream) {
  if (a == nullptr) return GGE_ERR_INVALID_ARG;
  const gge_tensor& x = a->x;
  gge_status s = check_values(x, false);
  if (s != GGE_OK) return s;
  if (x.batch != 1) return GGE_ERR_UNSUPPORTED;
  if (!is_value_type(a->param_dtype)) return GGE_ERR_UNSUPPORTED;
  b128::LnParams p;
  std::memset(&p, 0, sizeof(p));
  bool aligned = rows_aligned(x), alike = a->q == nullptr && a->h8 == nullptr;
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
  if (a->values != nullptr) {
    if (a->q == nullptr) return GGE_ERR_INVALID_ARG;
    if ((s = check_values(*a->values, false)) != GGE_OK) return s;
    if (!same_shape(*a->values, x.rows, x.cols, 1) || !rows_apart(*a->values)) return GGE_ERR_INVALID_ARG;
    aligned = aligned && rows_aligned(*a->values);
  }
  if ((s = take_codes(a->q, x, true, &p.q)) != GGE_OK) return s;
  if ((s = take_codes(a->h8, x, true, &p.h8)) != GGE_OK) return s;
  if (x.rows == 0 || x.cols == 0) return GGE_OK;
  if (!param_aligned(a->weight, a->param_dtype) || !param_aligned(a->bias, a->param_dtype) ||
      !float_aligned(a->mean) || !float_aligned(a->rstd))
    return GGE_ERR_ALIGNMENT;
  p.rows = x.rows;
  p.cols = static_cast<int32_t>(x.cols);
  p.dtype = x.dtype;
  p.x = x.ptr;
  p.ldx = x.stride_row;
  if (a->residual) { p.residual = a->residual->ptr; p.ldr = a->residual->stride_row; }
  if (a->residual_out) { p.h = a->residual_out->ptr; p.ldh = a->residual_out->stride_row; }
  if (a->y) { p.y = a->y->ptr; p.ldy = a->y->stride_row; }
  if (a->values) { p.values = a->values->ptr; p.ldv = a->values->stride_row; p.v_dtype = a->values->dtype; }
  p.weight = a->weight;
  p.bias = a->bias;
  p.p_dtype = a->param_dtype;
  p.eps = a->eps;
  p.mean = a->mean;
  p.rstd = a->rstd;
  p.w_vec = aligned16(a->weight) && aligned16(a->bias) ? 1 : 0;
  p.rows_lie = aligned ? lowp::ROWS_ALIGNED : (alike ? lowp::ROWS_ALIKE : lowp::ROWS_ANY);
  const int sms = sm_count();
  if (sms <= 0) return GGE_ERR_CUDA;
  return launched(b128::launch_ln(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

size_t gge_workspace_size_layernorm_bwd(int64_t cols) {
  const int sms = sm_count();
  if (sms <= 0 || cols < 0) return 0;
  return kTailBase + static_cast<size_t>(b128::ln_bwd_blocks(kMaxExtent, sms)) * 2 * static_cast<size_t>(cols) *
                         sizeof(float);
}

gge_status gge_layernorm_bwd(const gge_layernorm_bwd_args* a, void* ws, size_t ws_bytes, gge_stream_t stream) {
  if (a == nullptr || a->reserved != 0) return GGE_ERR_INVALID_ARG;
  const gge_tensor& dy = a->dy;
  gge_status s = check_values(dy, false);
  if (s != GGE_OK) return s;
  if (dy.batch != 1) return GGE_ERR_UNSUPPORTED;
  if (!is_value_type(a->weight_dtype)) return GGE_ERR_UNSUPPORTED;
  if ((a->h != nullptr) == (a->h8 != nullptr)) return GGE_ERR_INVALID_ARG;
  bool aligned = rows_aligned(dy), alike = a->h8 == nullptr;
  for (const gge_tensor* t : {a->h, a->dh, &a->dx}) {
    if (t == nullptr) continue;
    s = check_values(*t, false);
    if (s != GGE_OK) return s;
    if (t->dtype != dy.dtype) return GGE_ERR_UNSUPPORTED;
    if (!same_shape(*t, dy.rows, dy.cols, 1)) return GGE_ERR_INVALID_ARG;
    aligned = aligned && rows_aligned(*t);
    alike = alike && rows_alike(*t, dy);
  }
  if (!rows_apart(a->dx)) return GGE_ERR_INVALID_ARG;
  b128::LnBwdParams p;
  std::memset(&p, 0, sizeof(p));
  if ((s = take_codes(a->h8, dy, false, &p.h8)) != GGE_OK) return s;
  const bool sums = a->dweight != nullptr || a->dbias != nullptr;
  if (dy.cols == 0 || (dy.rows == 0 && !sums)) return GGE_OK;
  if (dy.rows > 0 && (a->mean == nullptr || a->rstd == nullptr)) return GGE_ERR_INVALID_ARG;
  if (!param_aligned(a->weight, a->weight_dtype) || !float_aligned(a->mean) || !float_aligned(a->rstd) ||
      !float_aligned(a->dweight) || !float_aligned(a->dbias))
    return GGE_ERR_ALIGNMENT;
  p.rows = dy.rows;
  p.cols = static_cast<int32_t>(dy.cols);
  p.dtype = dy.dtype;
  p.dy = dy.ptr;
  p.lddy = dy.stride_row;
  if (a->h) { p.h = a->h->ptr; p.ldh = a->h->stride_row; }
  if (a->dh) { p.dh = a->dh->ptr; p.lddh = a->dh->stride_row; }
  p.dx = a->dx.ptr;
  p.lddx = a->dx.stride_row;
  p.weight = a->weight;
  p.w_dtype = a->weight_dtype;
  p.mean = a->mean;
  p.rstd = a->rstd;
  p.dw = a->dweight;
  p.db = a->dbias;
  p.w_vec = aligned16(a->weight) ? 1 : 0;
  p.rows_lie = aligned ? lowp::ROWS_ALIGNED : (alike ? lowp::ROWS_ALIKE : lowp::ROWS_ANY);
  const int sms = sm_count();
  if (sms <= 0) return GGE_ERR_CUDA;
  if (sums) {
    if (ws == nullptr) return GGE_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return GGE_ERR_ALIGNMENT;
    if (ws_bytes < kTailBase + static_cast<size_t>(b128::ln_bwd_blocks(dy.rows, sms)) * 2 *
                                   static_cast<size_t>(dy.cols) * sizeof(float))
      return GGE_ERR_WORKSPACE;
    p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kTailBase);
  }
  return launched(b128::launch_ln_bwd(p, sms, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
