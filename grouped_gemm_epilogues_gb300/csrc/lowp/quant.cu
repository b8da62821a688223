// Microscaled quantisation and its inverse.
//
// The blocks of a quantised matrix run along its columns (a product's K).  The
// source may hold those contiguously (stride_col 1) or be the transpose of a
// row-major matrix (stride_row 1), as the weight-gradient products need it: a
// tile then goes through shared memory.  Both forms read the source once and
// are bound by memory.  Measured with the codes' values written too: 8192 x 8192 bf16
// to nvfp4 54 us (5.7 TB/s, 85 % of a copy's rate; issue 83 % busy, two divisions a
// block), transposed 59 us; 4096 x 32768 to mxfp8 transposed 128 us (5.3 TB/s, 79 %).
// Codes and scales alone: 40, 37 and 77 us.  Back to bf16, 8192 x 8192: mxfp8 35 us (5.8
// TB/s, 86 %), nvfp4 32.
#include "lowp_launch.h"
#include "rows.cuh"

namespace gge {
namespace lowp {
namespace {

using namespace mx;

__device__ __forceinline__ QuantOut quant_out(const QuantPtrs& q, int64_t batch) {
  const int vs = q.v_dtype == 4 ? 4 : 2;
  return QuantOut{q.codes + batch * q.batch_stride, q.ld, q.scales + batch * q.scale_batch_stride,
                  q.kgroups, q.tensor_scale,
                  q.values == nullptr
                      ? nullptr
                      : static_cast<void*>(static_cast<uint8_t*>(q.values) + batch * q.values_batch_stride * vs),
                  q.ldv, q.v_dtype};
}

// A block's eight warps cover 256 columns each: `wx` of them side by side, the
// others below, and U rows a warp, whose loads are in flight together.  Four rows
// where they start on 16-byte boundaries (8192 x 8192 to nvfp4 54 us; 60 with two, 77
// with one), two elsewhere, where a row takes more registers (4000 x 4001 25.7 us; 29.7
// with four, 27.3 with one).
template <bool AL>
constexpr int rows_a_warp() {
  return AL ? 4 : 2;
}

struct RowTiles {
  int32_t wx;         // warps along the columns: 1, 2, 4 or 8
  int32_t across;     // blocks along the columns
  int32_t rows;       // rows a warp
};

__host__ __device__ __forceinline__ int64_t rows_a_block(const RowTiles& r) { return 8 / r.wx * r.rows; }

RowTiles row_tiles(int64_t span, bool aligned) {
  RowTiles r{1, 1, aligned ? rows_a_warp<true>() : rows_a_warp<false>()};
  while (r.wx < 8 && r.wx * 256 < span) r.wx *= 2;
  r.across = static_cast<int32_t>((span + r.wx * 256 - 1) / (r.wx * 256));
  return r;
}

dim3 row_grid(const RowTiles& r, int64_t rows, int64_t batch) {
  const int64_t down = (rows + rows_a_block(r) - 1) / rows_a_block(r);
  return dim3(static_cast<unsigned>(down * r.across), static_cast<unsigned>(batch));
}

// This warp's first row and this lane's first column.
__device__ __forceinline__ void warp_place(const RowTiles& r, int64_t& row, int32_t& col) {
  const int warp = threadIdx.x >> 5;
  const uint32_t down = blockIdx.x / static_cast<uint32_t>(r.across);
  const uint32_t over = blockIdx.x - down * static_cast<uint32_t>(r.across);
  row = down * rows_a_block(r) + warp / r.wx * r.rows;
  col = (static_cast<int32_t>(over) * r.wx + warp % r.wx) * 256 + (threadIdx.x & 31) * 8;
}

// Columns contiguous.  AL: every row of the source (and of the values) starts on a
// 16-byte boundary.
template <typename T, int FMT, bool AL>
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const __grid_constant__ QuantParams p, RowTiles tiles) {
  constexpr int B = Fmt<FMT>::kBlock, U = rows_a_warp<AL>();
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.y;
  const QuantOut q = quant_out(p.q, batch);
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const int32_t cols = static_cast<int32_t>(p.cols);
  int64_t row0;
  int32_t col;
  warp_place(tiles, row0, col);
  if (col - (threadIdx.x & 31) * 8 >= cols) return;
  const int32_t rows = static_cast<int32_t>(min(p.rows - row0, static_cast<int64_t>(U)));
  const T* src = x + row0 * p.stride_row;
  uint8_t* codes = q.codes + row0 * q.ld + static_cast<int64_t>(col) * Fmt<FMT>::kBits / 8;
  // (a warp's rows share a scale tile's 32-row stretch: U divides 32)
  uint8_t* scales = q.scales + scale_word(row0, col / Fmt<FMT>::kGroup, q.kgroups);
  const bool word = holds_word<FMT>() && col < q.kgroups * Fmt<FMT>::kGroup;
  const bool code = col < ((cols + 31) & ~31);
  const bool past = col >= (cols + B - 1) / B * B;
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && q.tensor_scale) ? *q.tensor_scale : 1.f;
  Raw8<T> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int j = 0; j < WarpRow<T>::kPieces; ++j) raw[u].w[j] = make_uint4(0u, 0u, 0u, 0u);
    if (u < rows && col < cols) {
      const T* row = src + u * p.stride_row;
      if (AL && col + 8 <= cols) raw[u] = load8(row + col);
      else raw[u] = load_row8(row, col, cols, x);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= rows) break;  // (the whole warp)
    float2 v[4];
    widen(raw[u], v);
    const Quantised z = quantise8<FMT>(v, tscale, past);
    if (word) *reinterpret_cast<uint32_t*>(scales + u * 16) = z.word;
    if (code) store_codes<FMT>(codes + u * q.ld, z.codes);
    if (q.values != nullptr) {
      code_values<FMT>(z.codes, z.unit, tscale, v);
      store_row8_any<AL>(q.values, (row0 + u) * q.ldv, q.v_dtype, col, cols, v);
    }
  }
}

// Rows contiguous (the transpose of a row-major source): a block takes a tile of
// 128 rows (64 of 32-bit values) x 128 columns through shared memory.  A thread
// then holds 32 columns of the row pair (row) that one shared-memory word holds,
// whole blocks, and finds their scales by itself.  A word's column is kPitch words
// from the next, an odd number, so reads along either direction of the tile are
// free of bank conflicts.
constexpr int kTCols = 128, kTWords = 64, kTPitch = kTWords + 1;

// 32 columns of the V rows that words[0..31] hold, quantised: a row's codes to w[row],
// a scale byte a block to bytes[row * pitch], and, where wanted, the numbers that the
// codes stand for (rounded to O) back to the words (V = 2) or to their floats (V = 1).
template <typename T, int FMT, typename O>
__device__ __forceinline__ void quantise_words(uint32_t (&words)[32], float tscale, int32_t col, int32_t cols,
                                               uint32_t (&w)[4 / sizeof(T)][8], uint8_t* bytes, int pitch,
                                               bool values) {
  constexpr int V = 4 / sizeof(T), B = Fmt<FMT>::kBlock;
#pragma unroll
  for (int k = 0; k < 32; k += B) {
    float factor[V], unit[V];
    uint32_t amax[V];
    if constexpr (V == 2) {
      using T2 = typename Pair<T>::type;
      T2 m = __habs2(*reinterpret_cast<const T2*>(&words[k]));
#pragma unroll
      for (int i = 1; i < B; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const T2*>(&words[k + i])));
      const float2 f = widen_pair<T>(*reinterpret_cast<const uint32_t*>(&m));
      amax[0] = abs_bits(f.x);
      amax[1] = abs_bits(f.y);
    } else {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < B; ++i) m = max_abs(m, __uint_as_float(words[k + i]));
      amax[0] = abs_bits(m);
    }
#pragma unroll
    for (int h = 0; h < V; ++h) {
      const uint32_t s = block_scale<FMT>(amax[h], tscale, factor[h]);
      unit[h] = scale_value<FMT>(s);
      bytes[h * pitch + k / B] = static_cast<uint8_t>(col + k < cols ? s : 0u);
    }
#pragma unroll
    for (int i = k; i < k + B; i += 8) {
      float2 back[V][4];
#pragma unroll
      for (int h = 0; h < V; ++h) {
        float c[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float x;
          if constexpr (V == 1) x = __uint_as_float(words[i + j]);
          else x = h == 0 ? widen_pair<T>(words[i + j]).x : widen_pair<T>(words[i + j]).y;
          c[j] = x * factor[h];
        }
        const uint2 codes = pack8<FMT>(c);
        if constexpr (FMT == FMT_MXFP8) {
          w[h][i / 4] = codes.x;
          w[h][i / 4 + 1] = codes.y;
        } else {
          w[h][i / 8] = codes.x;
        }
        if (values) code_values<FMT>(codes, unit[h], tscale, back[h]);
      }
      if (values) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if constexpr (V == 1) {
            words[i + 2 * j] = __float_as_uint(back[0][j].x);
            words[i + 2 * j + 1] = __float_as_uint(back[0][j].y);
          } else {
            words[i + 2 * j] = narrow_pair<O>(make_float2(back[0][j].x, back[1][j].x));
            words[i + 2 * j + 1] = narrow_pair<O>(make_float2(back[0][j].y, back[1][j].y));
          }
        }
      }
    }
  }
}

// O: the type of the values (what a 16-bit source's words take; bf16 where none).
template <typename T, int FMT, bool AL, typename O>
__global__ void __launch_bounds__(256, 4) quantize_cols_kernel(const __grid_constant__ QuantParams p) {
  constexpr int V = 4 / sizeof(T);         // rows a word holds
  constexpr int kRows = kTWords * V;       // rows of the tile
  constexpr int kBytes = kTCols / Fmt<FMT>::kBlock;  // scale bytes of a row of the tile
  constexpr int kCodes = kTCols * Fmt<FMT>::kBits / 8;  // bytes of codes of a row of the tile
  constexpr int kPiecesARow = kCodes / 16;
  extern __shared__ __align__(16) uint8_t shared[];
  uint32_t* tile = reinterpret_cast<uint32_t*>(shared);                    // [column][word]
  uint32_t* words = tile + kTCols * kTPitch;                               // scale bytes
  uint4* pieces = reinterpret_cast<uint4*>(words + kRows * kBytes / 4);    // codes, [row][kPiecesARow + 1]
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.z;
  const QuantOut q = quant_out(p.q, batch);
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const int64_t row0 = static_cast<int64_t>(blockIdx.y) * kRows;
  const int32_t rows = static_cast<int32_t>(p.rows), cols = static_cast<int32_t>(p.cols);
  const int32_t col0 = blockIdx.x * kTCols;
  ptx::griddep_wait();
  const float tscale = (FMT == FMT_NVFP4 && q.tensor_scale) ? *q.tensor_scale : 1.f;
  {
    // 8 rows of one column a piece; kTCols * kRows / 8 pieces
    constexpr int kAcross = kRows / 8, kDown = 256 / kAcross, kPieces = kTCols / kDown;
    const int r = threadIdx.x % kAcross * 8, c = threadIdx.x / kAcross;
    const int32_t row = static_cast<int32_t>(row0) + r;
    Raw8<T> raw[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
#pragma unroll
      for (int j = 0; j < WarpRow<T>::kPieces; ++j) raw[u].w[j] = make_uint4(0u, 0u, 0u, 0u);
      const int32_t col = col0 + c + kDown * u;
      if (row < rows && col < cols) {
        const T* line = x + col * p.stride_col;
        if (AL && row + 8 <= rows) raw[u] = load8(line + row);
        else raw[u] = load_row8(line, row, rows, x);
      }
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(&raw[u]);
#pragma unroll
      for (int i = 0; i < 8 / V; ++i) tile[(c + kDown * u) * kTPitch + r / V + i] = w[i];
    }
  }
  __syncthreads();
  const int part = threadIdx.x / kTWords, at = threadIdx.x % kTWords;  // 32 columns a part
  const int32_t col = col0 + part * 32;
  uint32_t* mine = tile + part * 32 * kTPitch + at;
  uint32_t held[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) held[i] = mine[i * kTPitch];
  uint32_t w[V][8];
  quantise_words<T, FMT, O>(held, tscale, col, cols, w,
                            reinterpret_cast<uint8_t*>(words) + at * V * kBytes + part * (kBytes / 4), kBytes,
                            q.values != nullptr);
#pragma unroll
  for (int h = 0; h < V; ++h) {
    uint4* dst = pieces + (at * V + h) * (kPiecesARow + 1) + part * (kPiecesARow / 4);
    dst[0] = make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
    if constexpr (FMT == FMT_MXFP8) dst[1] = make_uint4(w[h][4], w[h][5], w[h][6], w[h][7]);
  }
  if (q.values != nullptr) {  // the values take the source's place in the tile
#pragma unroll
    for (int i = 0; i < 32; ++i) mine[i * kTPitch] = held[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * kBytes / 4; i += 256) {
    const int rr = i % kRows, kw = i / kRows;
    const int64_t kg = col0 / Fmt<FMT>::kGroup + kw;
    if (row0 + rr < p.rows && kg < q.kgroups)
      *reinterpret_cast<uint32_t*>(q.scales + scale_word(row0 + rr, kg, q.kgroups)) = words[rr * (kBytes / 4) + kw];
  }
  // whole lines of codes
  for (int i = threadIdx.x; i < kRows * kPiecesARow; i += 256) {
    const int rr = i / kPiecesARow, piece = i % kPiecesARow;
    const int32_t c = col0 + piece * (128 / Fmt<FMT>::kBits);
    if (row0 + rr < p.rows && c < ((cols + 31) & ~31))
      *reinterpret_cast<uint4*>(q.codes + (row0 + rr) * q.ld + static_cast<int64_t>(c) * Fmt<FMT>::kBits / 8) =
          pieces[rr * (kPiecesARow + 1) + piece];
  }
  if (q.values == nullptr) return;
  // values: a warp a word of rows.  Two columns a lane where a row's pairs start on four
  // bytes, else one: whole lines at any alignment
  const int lane = threadIdx.x & 31;
  if (V == 2 && q.ldv % 2 == 0 && (reinterpret_cast<uintptr_t>(q.values) & 3u) == 0) {
    uint16_t* values = static_cast<uint16_t*>(q.values);
    for (int r = threadIdx.x >> 5; r < kTWords; r += 8) {
      const int64_t row = row0 + r * V;
      if (row >= p.rows) break;
#pragma unroll
      for (int c = lane * 2; c < kTCols; c += 64) {
        if (col0 + c >= cols) break;
        const uint32_t a = tile[c * kTPitch + r], b = tile[(c + 1) * kTPitch + r];
        uint16_t* out = values + row * q.ldv + col0 + c;
        if (col0 + c + 1 < cols) {
          *reinterpret_cast<uint32_t*>(out) = __byte_perm(a, b, 0x5410);
          if (row + 1 < p.rows) *reinterpret_cast<uint32_t*>(out + q.ldv) = __byte_perm(a, b, 0x7632);
        } else {
          out[0] = static_cast<uint16_t>(a);
          if (row + 1 < p.rows) out[q.ldv] = static_cast<uint16_t>(a >> 16);
        }
      }
    }
    return;
  }
  for (int r = threadIdx.x >> 5; r < kTWords; r += 8) {
    const int64_t row = row0 + r * V;
    if (row >= p.rows) break;
#pragma unroll
    for (int c = lane; c < kTCols; c += 32) {
      if (col0 + c >= cols) break;
      const uint32_t w = tile[c * kTPitch + r];
      const int64_t out = row * q.ldv + col0 + c;
      if constexpr (V == 1) {
        store_any(q.values, out, q.v_dtype, __uint_as_float(w));
      } else {
        static_cast<uint16_t*>(q.values)[out] = static_cast<uint16_t>(w);
        if (row + 1 < p.rows) static_cast<uint16_t*>(q.values)[out + q.ldv] = static_cast<uint16_t>(w >> 16);
      }
    }
  }
}

template <typename T, int FMT, bool AL>
cudaError_t launch_quantize_t(const QuantParams& p, cudaStream_t st) {
  const int64_t span = scale_span<FMT>(p.q.kgroups);
  if (p.stride_col == 1 || p.cols == 1) {
    const RowTiles tiles = row_tiles(span, AL);
    return launch_pdl(quantize_rows_kernel<T, FMT, AL>, row_grid(tiles, p.rows, p.batch), dim3(256), 0, st,
                      p, tiles);
  }
  constexpr int kRows = kTWords * (4 / sizeof(T));
  constexpr size_t smem = kTCols * kTPitch * 4 + kRows * (kTCols / Fmt<FMT>::kBlock) +
                          kRows * (kTCols * Fmt<FMT>::kBits / 8 + 16);
  const bool half = p.q.values != nullptr && p.q.v_dtype == 1;
  const auto kern = half ? quantize_cols_kernel<T, FMT, AL, __half> : quantize_cols_kernel<T, FMT, AL, __nv_bfloat16>;
  const cudaError_t e = half ? allow_smem<quantize_cols_kernel<T, FMT, AL, __half>>()
                             : allow_smem<quantize_cols_kernel<T, FMT, AL, __nv_bfloat16>>();
  if (e != cudaSuccess) return e;
  return launch_pdl(kern,
                    dim3(static_cast<unsigned>((span + kTCols - 1) / kTCols),
                         static_cast<unsigned>((p.rows + kRows - 1) / kRows),
                         static_cast<unsigned>(p.batch)),
                    dim3(256), smem, st, p);
}

template <typename T>
cudaError_t launch_quantize_f(const QuantParams& p, cudaStream_t st) {
  switch (p.q.format) {
    case FMT_MXFP8: return p.aligned ? launch_quantize_t<T, FMT_MXFP8, true>(p, st)
                                     : launch_quantize_t<T, FMT_MXFP8, false>(p, st);
    case FMT_MXFP4: return p.aligned ? launch_quantize_t<T, FMT_MXFP4, true>(p, st)
                                     : launch_quantize_t<T, FMT_MXFP4, false>(p, st);
    default: return p.aligned ? launch_quantize_t<T, FMT_NVFP4, true>(p, st)
                                     : launch_quantize_t<T, FMT_NVFP4, false>(p, st);
  }
}

// ------------------------------------------------------------- and back

template <int FMT, bool AL>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const __grid_constant__ DequantParams p, RowTiles tiles) {
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int64_t batch = blockIdx.y;
  const uint8_t* codes = p.codes + batch * p.batch_stride;
  const uint8_t* scales = p.scales + batch * p.scale_batch_stride;
  const float tscale = (FMT == FMT_NVFP4 && p.tensor_scale) ? *p.tensor_scale : 1.f;
  const int32_t cols = static_cast<int32_t>(p.cols);
  int64_t row0;
  int32_t col;
  warp_place(tiles, row0, col);
  constexpr int U = rows_a_warp<AL>();
  uint2 w[U];
  float unit[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + u;
    w[u] = make_uint2(0u, 0u);
    unit[u] = 0.f;
    if (row >= p.rows || col >= cols) continue;
    const uint8_t* c = codes + row * p.ld + static_cast<int64_t>(col) * Fmt<FMT>::kBits / 8;
    if constexpr (FMT == FMT_MXFP8) w[u] = *reinterpret_cast<const uint2*>(c);
    else w[u].x = *reinterpret_cast<const uint32_t*>(c);
    const int64_t block = col / Fmt<FMT>::kBlock;
    unit[u] = scale_value<FMT>(scales[scale_word(row, block >> 2, p.kgroups) + (block & 3)]);
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row0 + u >= p.rows) break;
    float2 v[4];
    code_values<FMT>(w[u], unit[u], tscale, v);
    store_row8_any<AL>(p.y, batch * p.y_batch_stride + (row0 + u) * p.ldy, p.dtype, col, cols, v);
  }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams& p, cudaStream_t st) {
  if (p.dtype != 4 && p.q.values != nullptr && p.q.v_dtype == 4 && p.stride_col != 1 && p.cols != 1) {
    // the transposing kernel passes a 16-bit source's values on in 16 bits: 32-bit ones
    // are read back from the codes
    QuantParams codes = p;
    codes.q.values = nullptr;
    const cudaError_t e = launch_quantize(codes, st);
    if (e != cudaSuccess) return e;
    DequantParams d{};
    d.rows = p.rows, d.cols = p.cols, d.batch = p.batch;
    d.format = p.q.format;
    d.codes = p.q.codes, d.scales = p.q.scales;
    d.ld = p.q.ld, d.batch_stride = p.q.batch_stride;
    d.kgroups = p.q.kgroups, d.scale_batch_stride = p.q.scale_batch_stride;
    d.tensor_scale = p.q.tensor_scale;
    d.y = p.q.values, d.ldy = p.q.ldv, d.y_batch_stride = p.q.values_batch_stride;
    d.dtype = 4;
    return launch_dequantize(d, st);  // (any alignment)
  }
  if (p.dtype == 0) return launch_quantize_f<__nv_bfloat16>(p, st);
  if (p.dtype == 1) return launch_quantize_f<__half>(p, st);
  return launch_quantize_f<float>(p, st);
}

cudaError_t launch_dequantize(const DequantParams& p, cudaStream_t st) {
  const RowTiles tiles = row_tiles(p.cols, p.aligned != 0);
  const dim3 grid = row_grid(tiles, p.rows, p.batch);
  switch (p.format) {
    case FMT_MXFP8: return launch_pdl(p.aligned ? dequantize_kernel<FMT_MXFP8, true> : dequantize_kernel<FMT_MXFP8, false>, grid,
                                      dim3(256), 0, st, p, tiles);
    case FMT_MXFP4: return launch_pdl(p.aligned ? dequantize_kernel<FMT_MXFP4, true> : dequantize_kernel<FMT_MXFP4, false>, grid,
                                      dim3(256), 0, st, p, tiles);
    default: return launch_pdl(p.aligned ? dequantize_kernel<FMT_NVFP4, true> : dequantize_kernel<FMT_NVFP4, false>, grid,
                                      dim3(256), 0, st, p, tiles);
  }
}

}  // namespace lowp
}  // namespace gge
