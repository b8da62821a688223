// Quantisation to 8 bits with a scale for each block of 128, its inverse, and the
// transposition of a matrix that is in this form already.
//
// Blocks run along a result's columns.  The source may hold those contiguously, or be the
// transpose of a row-major matrix (its own columns contiguous along the result's rows), in
// 16 or 32 bits or as codes: a 128 x 128 tile then goes through shared memory.  Every form
// reads the source once.  8192 x 8192 bf16 in 44 us either way, rows as they lie 38 (201 MB, 4.6 and 5.3
// TB/s; with the values written too 60, 5.6 TB/s); codes of 16384 x 4096 turned in 38 us (138 MB, 3.7
// TB/s; with values 52), bound by the phases of a tile: load, scales, codes, store.
#include "b128_launch.h"
#include "rows.cuh"

namespace gge {
namespace b128 {
namespace {

using namespace mx;
using lowp::WarpRow;

// n values of 8, in columns [col, col + 8) of a row at `row` of a runtime type.  AL: 16-byte
// stores; else single values (neighbouring lanes store neighbouring ones).
template <typename O>
__device__ __forceinline__ void store_values8_t(O* at, int32_t n, const float2 (&v)[4]) {
  const Raw8<O> r = narrow<O>(v);
  if (n >= 8) {
    store8(at, r);
  } else {
    const O* o = reinterpret_cast<const O*>(&r);
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) at[i] = o[i];
  }
}
__device__ __forceinline__ void store_values8(void* base, int64_t at, int32_t dtype, int32_t n, const float2 (&v)[4]) {
  if (dtype == 0) store_values8_t(static_cast<__nv_bfloat16*>(base) + at, n, v);
  else if (dtype == 1) store_values8_t(static_cast<__half*>(base) + at, n, v);
  else store_values8_t(static_cast<float*>(base) + at, n, v);
}

__device__ __forceinline__ int64_t value_at(const QuantParams& p, int64_t batch, int64_t row, int64_t col) {
  return batch * p.v_batch + row * p.ldv + col;
}

// ------------------------------------------------- columns contiguous, blocks of a row

// A block's eight warps cover 256 columns each: `wx` of them side by side, the others
// below, U rows a warp, whose loads are in flight together.
constexpr int kRowsAWarp = 4;

struct RowTiles {
  int32_t wx, across;
};
__host__ __device__ __forceinline__ int64_t rows_a_block(const RowTiles& r) { return 8 / r.wx * kRowsAWarp; }

RowTiles row_tiles(int64_t cols) {
  RowTiles r{1, 1};
  while (r.wx < 8 && r.wx * 256 < cols) r.wx *= 2;
  r.across = static_cast<int32_t>((cols + r.wx * 256 - 1) / (r.wx * 256));
  return r;
}
dim3 row_grid(const RowTiles& r, int64_t rows, int64_t batch) {
  const int64_t down = (rows + rows_a_block(r) - 1) / rows_a_block(r);
  return dim3(static_cast<unsigned>(down * r.across), static_cast<unsigned>(batch));
}
__device__ __forceinline__ void warp_place(const RowTiles& r, int64_t& row, int32_t& col) {
  const int warp = threadIdx.x >> 5;
  const uint32_t down = blockIdx.x / static_cast<uint32_t>(r.across);
  const uint32_t over = blockIdx.x - down * static_cast<uint32_t>(r.across);
  row = down * rows_a_block(r) + warp / r.wx * kRowsAWarp;
  col = (static_cast<int32_t>(over) * r.wx + warp % r.wx) * 256 + (threadIdx.x & 31) * 8;
}

template <typename T, bool E5M2, bool AL>
__global__ void __launch_bounds__(256)
    quantize_rows_kernel(const __grid_constant__ QuantParams p, RowTiles tiles) {
  constexpr int U = kRowsAWarp;
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.y;
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const int32_t cols = static_cast<int32_t>(p.cols);
  int64_t row0;
  int32_t col;
  warp_place(tiles, row0, col);
  const int lane = threadIdx.x & 31;
  if (col - lane * 8 >= cols) return;
  const int32_t rows = static_cast<int32_t>(min(p.rows - row0, static_cast<int64_t>(U)));
  const T* src = x + row0 * p.stride_row;
  uint8_t* codes = p.q.codes + batch * p.q.batch + row0 * p.q.ld + col;
  float* scale = p.q.scale(row0, col >> 7, batch);
  ptx::griddep_wait();
  Raw8<T> raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int j = 0; j < WarpRow<T>::kPieces; ++j) raw[u].w[j] = make_uint4(0u, 0u, 0u, 0u);
    if (u < rows && col < cols) {
      const T* row = src + u * p.stride_row;
      if (AL && col + 8 <= cols) raw[u] = load8(row + col);
      else raw[u] = lowp::load_row8(row, col, cols, x);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= rows) break;  // (the whole warp)
    float2 v[4];
    widen(raw[u], v);
    float unit;
    const uint2 z = quantise8<E5M2>(v, unit);
    if ((lane & 15) == 0 && col < cols) scale[u * p.q.s_row] = unit;
    store_codes8(codes + u * p.q.ld, z, cols - col);
    if (p.values != nullptr) {
      values8<E5M2>(z, unit, v);
      lowp::store_row8_any<AL>(p.values, value_at(p, batch, row0 + u, 0), p.v_dtype, col, cols, v);
    }
  }
}

// ---------------------------------------------- columns contiguous, blocks of 128 rows

// A thread block takes a block: sixteen lanes a row, sixteen rows at a time, held in
// registers while the largest value is found.
template <typename T, bool E5M2, bool AL>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(const __grid_constant__ QuantParams p, uint32_t across) {
  __shared__ uint32_t most[8];
  constexpr int U = 8;
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.y;
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  const int32_t cols = static_cast<int32_t>(p.cols);
  const int lane = threadIdx.x & 31;
  const uint32_t down = blockIdx.x / across, over = blockIdx.x - down * across;
  const int64_t row0 = static_cast<int64_t>(down) * 128 + (threadIdx.x >> 4);
  const int32_t col = over * 128 + (threadIdx.x & 15) * 8;
  ptx::griddep_wait();
  Raw8<T> raw[U];
  uint32_t amax = 0u;
#pragma unroll
  for (int u = 0; u < U; ++u) {
#pragma unroll
    for (int j = 0; j < WarpRow<T>::kPieces; ++j) raw[u].w[j] = make_uint4(0u, 0u, 0u, 0u);
    const int64_t row = row0 + 16 * u;
    if (row < p.rows && col < cols) {
      const T* at = x + row * p.stride_row;
      if (AL && col + 8 <= cols) raw[u] = load8(at + col);
      else raw[u] = lowp::load_row8(at, col, cols, x);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float2 v[4];
    widen(raw[u], v);
    amax = max(amax, amax8(v));
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  if (lane == 0) most[threadIdx.x >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = max(amax, most[i]);
  float factor;
  const float unit = block_scale<E5M2>(amax, factor);
  if (threadIdx.x == 0) *p.q.scale(row0, over, batch) = unit;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t row = row0 + 16 * u;
    if (row >= p.rows) break;
    float2 v[4];
    widen(raw[u], v);
    const uint2 z = codes8<E5M2>(v, factor);
    store_codes8(p.q.codes + batch * p.q.batch + row * p.q.ld + col, z, cols - col);
    if (p.values != nullptr && col < cols) {
      values8<E5M2>(z, unit, v);
      const int64_t at = value_at(p, batch, row, col);
      if (p.v_aligned) {
        store_values8(p.values, at, p.v_dtype, cols - col, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (col + i < cols) store_any(p.values, at + i, p.v_dtype, i & 1 ? v[i / 2].y : v[i / 2].x);
      }
    }
  }
}

// -------------------------------------------------------- rows contiguous (transposed)

// What a 32-bit word of the source's storage holds: V rows of one column.
template <typename T> struct Word { static constexpr int V = 4 / sizeof(T); };
struct Code8 { uint8_t b; };  // codes, whose numbers are the product with their block's scale

// A block takes 128 rows x 128 columns.  While the tile's words come in, each thread keeps the
// largest value of the rows it loads; with the scales known, a thread turns the words of one
// place (V rows) and 64 / V columns into codes, which leave through shared memory in whole
// lines, as do the values they stand for.  A column's words are one more than an even number
// apart, so both directions of the tile are free of bank conflicts.
template <typename T, bool E5M2, bool AL>
struct ColsTile {
  static constexpr int V = Word<T>::V;
  static constexpr int kWords = 128 / V;
  static constexpr int kPitch = kWords + 1;
  static constexpr int kCodePitch = 128 + 16;
  // tile words, codes, the warps' maxima, factors and scales, the source's scales
  static constexpr size_t kBytes = 128 * kPitch * 4 + 128 * kCodePitch + 8 * 128 * 4 + 2 * 128 * 4 + 128 * 4 + 16;
};

template <typename T, bool E5M2, bool AL, bool FROM5>
__global__ void __launch_bounds__(256) quantize_cols_kernel(const __grid_constant__ QuantParams p, uint32_t down) {
  using Tile = ColsTile<T, E5M2, AL>;
  constexpr bool kCodes = sizeof(T) == 1;
  constexpr int V = Tile::V;
  extern __shared__ __align__(16) uint8_t shared[];
  uint32_t* tile = reinterpret_cast<uint32_t*>(shared);
  uint8_t* codes = shared + 128 * Tile::kPitch * 4;                      // [row][kCodePitch]
  uint32_t* most = reinterpret_cast<uint32_t*>(codes + 128 * Tile::kCodePitch);  // [warp][row]
  float* factors = reinterpret_cast<float*>(most + 8 * 128);
  float* units = factors + 128;
  float* from = units + 128;                                              // [column]
  uint32_t* all = reinterpret_cast<uint32_t*>(from + 128);                // [4]
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.y;
  const int32_t rows = static_cast<int32_t>(p.rows), cols = static_cast<int32_t>(p.cols);
  const uint32_t over = blockIdx.x / down;  // (tiles down the rows first: the source's lines)
  const int32_t row0 = (blockIdx.x - over * down) * 128, col0 = over * 128;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* x = static_cast<const T*>(p.x) + batch * p.stride_batch;
  ptx::griddep_wait();
  // 16 bytes a thread and pass: kRun rows of a column (32 bytes of a 32-bit source)
  constexpr int kRun = kCodes ? 16 : 8;
  constexpr int kAcross = 128 / kRun;       // threads a column
  constexpr int kDown = 256 / kAcross;      // columns a pass
  constexpr int kPasses = 128 / kDown;
  constexpr int kW = kRun / V;              // words a thread and pass
  const int r = threadIdx.x % kAcross * kRun, c0 = threadIdx.x / kAcross;
  const int32_t row = row0 + r;
  uint32_t raw[kPasses][kW];
  float scale[kCodes ? kPasses : 1];
#pragma unroll
  for (int u = 0; u < kPasses; ++u) {
#pragma unroll
    for (int i = 0; i < kW; ++i) raw[u][i] = 0u;
    const int32_t col = col0 + c0 + kDown * u;
    if constexpr (kCodes) scale[u] = 0.f;
    if (row < rows && col < cols) {
      const T* line = x + static_cast<int64_t>(col) * p.stride_col;
      if constexpr (kCodes) {
        scale[u] = *p.from.scale(col, row0 >> 7, batch);
        // (lines of codes start on 16 bytes; past the row's end single codes are taken)
        const uint8_t* at = reinterpret_cast<const uint8_t*>(line) + row;
        if (row + 16 <= rows) {
          const uint4 w = *reinterpret_cast<const uint4*>(at);
          raw[u][0] = w.x, raw[u][1] = w.y, raw[u][2] = w.z, raw[u][3] = w.w;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (row + i < rows) raw[u][i / 4] |= static_cast<uint32_t>(at[i]) << (8 * (i & 3));
        }
      } else {
        const Raw8<T> v = AL && row + 8 <= rows ? load8(line + row) : lowp::load_row8(line, row, rows, x);
        const uint32_t* w = reinterpret_cast<const uint32_t*>(&v);
#pragma unroll
        for (int i = 0; i < kW; ++i) raw[u][i] = w[i];
      }
    }
  }
  // the numbers of one word
  const auto numbers = [](uint32_t w, float s, float (&v)[V]) {
    if constexpr (kCodes) {
      float2 f[2];
      values4<FROM5>(w, s, f);
      v[0] = f[0].x, v[1] = f[0].y, v[2] = f[1].x, v[3] = f[1].y;
    } else if constexpr (V == 2) {
      const float2 f = widen_pair<T>(w);
      v[0] = f.x, v[1] = f.y;
    } else {
      v[0] = __uint_as_float(w);
    }
  };
  {
    float top[kRun];
#pragma unroll
    for (int i = 0; i < kRun; ++i) top[i] = 0.f;
#pragma unroll
    for (int u = 0; u < kPasses; ++u)
#pragma unroll
      for (int i = 0; i < kW; ++i) {
        float v[V];
        numbers(raw[u][i], kCodes ? scale[u] : 0.f, v);
#pragma unroll
        for (int h = 0; h < V; ++h) top[i * V + h] = max_abs(top[i * V + h], v[h]);
      }
    // lanes that load the same rows are kAcross apart
#pragma unroll
    for (int o = kAcross; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < kRun; ++i) top[i] = max_abs(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    if (lane < kAcross) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) most[warp * 128 + r + i] = abs_bits(top[i]);
    }
#pragma unroll
    for (int u = 0; u < kPasses; ++u) {
      const int c = c0 + kDown * u;
      if (kCodes && r == 0) from[c] = scale[u];
#pragma unroll
      for (int i = 0; i < kW; ++i) tile[c * Tile::kPitch + r / V + i] = raw[u][i];
    }
  }
  __syncthreads();
  uint32_t amax = 0u;
  if (threadIdx.x < 128) {
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, most[i * 128 + threadIdx.x]);
    if (p.q.shift != 0) {
      const uint32_t m = __reduce_max_sync(0xffffffffu, amax);
      if (lane == 0) all[warp] = m;
    }
  }
  if (p.q.shift != 0) __syncthreads();
  if (threadIdx.x < 128) {
    if (p.q.shift != 0) amax = max(max(all[0], all[1]), max(all[2], all[3]));
    float factor;
    const float unit = block_scale<E5M2>(amax, factor);
    factors[threadIdx.x] = factor;
    units[threadIdx.x] = unit;
    if (p.q.shift == 0 ? row0 + static_cast<int32_t>(threadIdx.x) < rows : threadIdx.x == 0)
      *p.q.scale(row0 + threadIdx.x, col0 >> 7, batch) = unit;
  }
  __syncthreads();
  {
    constexpr int kCols = 64 / V;             // columns a thread
    const int at = threadIdx.x % Tile::kWords, part = threadIdx.x / Tile::kWords;
    const uint32_t* mine = tile + part * kCols * Tile::kPitch + at;
    float f[V];
#pragma unroll
    for (int h = 0; h < V; ++h) f[h] = factors[at * V + h];
#pragma unroll
    for (int i = 0; i < kCols; i += 16) {
      uint32_t w[V][4];
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        float v[4][V];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int c = i + j + k;
          numbers(mine[c * Tile::kPitch], kCodes ? from[part * kCols + c] : 0.f, v[k]);
        }
#pragma unroll
        for (int h = 0; h < V; ++h)
          w[h][j / 4] = pack4<E5M2>(v[0][h] * f[h], v[1][h] * f[h], v[2][h] * f[h], v[3][h] * f[h]);
      }
#pragma unroll
      for (int h = 0; h < V; ++h)
        *reinterpret_cast<uint4*>(codes + (at * V + h) * Tile::kCodePitch + part * kCols + i) =
            make_uint4(w[h][0], w[h][1], w[h][2], w[h][3]);
    }
  }
  __syncthreads();
  // whole lines of codes: eight lanes a row
  uint8_t* out = p.q.codes + batch * p.q.batch + static_cast<int64_t>(row0) * p.q.ld + col0;
#pragma unroll
  for (int i = threadIdx.x; i < 128 * 8; i += 256) {
    const int rr = i >> 3, c = (i & 7) * 16;
    if (row0 + rr >= rows) break;
    const int32_t n = cols - col0 - c;
    const uint4 w = *reinterpret_cast<const uint4*>(codes + rr * Tile::kCodePitch + c);
    if (n >= 16) {
      *reinterpret_cast<uint4*>(out + rr * p.q.ld + c) = w;
    } else {
      store_codes8(out + rr * p.q.ld + c, make_uint2(w.x, w.y), n);
      store_codes8(out + rr * p.q.ld + c + 8, make_uint2(w.z, w.w), n - 8);
    }
  }
  if (p.values == nullptr) return;
  // sixteen lanes a row
#pragma unroll 2
  for (int i = threadIdx.x; i < 128 * 16; i += 256) {
    const int rr = i >> 4, c = (i & 15) * 8;
    if (row0 + rr >= rows) break;
    if (!p.v_aligned) break;
    float2 v[4];
    values8<E5M2>(*reinterpret_cast<const uint2*>(codes + rr * Tile::kCodePitch + c), units[rr], v);
    if (col0 + c < cols) store_values8(p.values, value_at(p, batch, row0 + rr, col0 + c), p.v_dtype, cols - col0 - c, v);
  }
  if (p.v_aligned) return;
  // rows that start anywhere: a value a lane
  for (int i = threadIdx.x; i < 128 * 128; i += 256) {
    const int rr = i >> 7, c = i & 127;
    if (row0 + rr >= rows) break;
    if (col0 + c < cols)
      store_any(p.values, value_at(p, batch, row0 + rr, col0 + c), p.v_dtype,
                unpack2<E5M2>(codes[rr * Tile::kCodePitch + c]).x * units[rr]);
  }
}

// ------------------------------------------------------------------ and back

template <bool E5M2, bool AL>
__global__ void __launch_bounds__(256)
    dequantize_kernel(const __grid_constant__ DequantParams p, RowTiles tiles) {
  constexpr int U = kRowsAWarp;
  ptx::griddep_launch_dependents();
  const int64_t batch = blockIdx.y;
  const int32_t cols = static_cast<int32_t>(p.cols);
  int64_t row0;
  int32_t col;
  warp_place(tiles, row0, col);
  if (col - (threadIdx.x & 31) * 8 >= cols) return;
  const uint8_t* codes = p.q.codes + batch * p.q.batch + row0 * p.q.ld + col;
  ptx::griddep_wait();
  uint2 w[U];
  float unit[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    w[u] = make_uint2(0u, 0u);
    unit[u] = 0.f;
    if (row0 + u >= p.rows || col >= cols) continue;
    unit[u] = *p.q.scale(row0 + u, col >> 7, batch);
    const uint8_t* at = codes + u * p.q.ld;
    if (col + 8 <= cols) {
      w[u] = *reinterpret_cast<const uint2*>(at);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (col + i < cols) (i < 4 ? w[u].x : w[u].y) |= static_cast<uint32_t>(at[i]) << (8 * (i & 3));
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (row0 + u >= p.rows) break;
    float2 v[4];
    values8<E5M2>(w[u], unit[u], v);
    lowp::store_row8_any<AL>(p.y, batch * p.y_batch + (row0 + u) * p.ldy, p.dtype, col, cols, v);
  }
}

// ------------------------------------------------------------------ launches

using lowp::launch_pdl;

// (a matrix that fits the device's memory has fewer than 2^26 tiles)
dim3 tile_grid(const QuantParams& p) {
  return dim3(static_cast<unsigned>((p.rows + 127) / 128 * ((p.cols + 127) / 128)), static_cast<unsigned>(p.batch));
}

template <typename T, bool E5M2, bool FROM5>
cudaError_t launch_cols(const QuantParams& p, cudaStream_t st) {
  const uint32_t down = static_cast<uint32_t>((p.rows + 127) / 128);
  const dim3 grid = tile_grid(p);
  if (p.aligned) {
    const cudaError_t e = allow_smem<quantize_cols_kernel<T, E5M2, true, FROM5>>();
    if (e != cudaSuccess) return e;
    return launch_pdl(quantize_cols_kernel<T, E5M2, true, FROM5>, grid, dim3(256), ColsTile<T, E5M2, true>::kBytes, st, p, down);
  }
  const cudaError_t e = allow_smem<quantize_cols_kernel<T, E5M2, false, FROM5>>();
  if (e != cudaSuccess) return e;
  return launch_pdl(quantize_cols_kernel<T, E5M2, false, FROM5>, grid, dim3(256), ColsTile<T, E5M2, false>::kBytes, st, p, down);
}

template <typename T, bool E5M2, bool AL>
cudaError_t launch_straight(const QuantParams& p, cudaStream_t st) {
  if (p.q.shift != 0) {
    return launch_pdl(quantize_tiles_kernel<T, E5M2, AL>, tile_grid(p), dim3(256), 0, st, p,
                      static_cast<uint32_t>((p.cols + 127) / 128));
  }
  const RowTiles tiles = row_tiles(p.cols);
  return launch_pdl(quantize_rows_kernel<T, E5M2, AL>, row_grid(tiles, p.rows, p.batch), dim3(256), 0, st, p, tiles);
}

template <typename T, bool E5M2>
cudaError_t launch_quantize_t(const QuantParams& p, cudaStream_t st) {
  if (p.stride_col != 1 && p.cols != 1) return launch_cols<T, E5M2, false>(p, st);
  const bool al = p.aligned && (p.values == nullptr || p.v_aligned);
  return al ? launch_straight<T, E5M2, true>(p, st) : launch_straight<T, E5M2, false>(p, st);
}

template <bool E5M2>
cudaError_t launch_quantize_f(const QuantParams& p, cudaStream_t st) {
  switch (p.dtype) {
    case 0: return launch_quantize_t<__nv_bfloat16, E5M2>(p, st);
    case 1: return launch_quantize_t<__half, E5M2>(p, st);
    case 2: return launch_cols<Code8, E5M2, false>(p, st);
    case 3: return launch_cols<Code8, E5M2, true>(p, st);
    default: return launch_quantize_t<float, E5M2>(p, st);
  }
}

}  // namespace

cudaError_t launch_quantize(const QuantParams& p, cudaStream_t st) {
  return p.q.e5m2 ? launch_quantize_f<true>(p, st) : launch_quantize_f<false>(p, st);
}

cudaError_t launch_dequantize(const DequantParams& p, cudaStream_t st) {
  const RowTiles tiles = row_tiles(p.cols);
  const dim3 grid = row_grid(tiles, p.rows, p.batch);
  const auto kern = p.q.e5m2 ? (p.aligned ? dequantize_kernel<true, true> : dequantize_kernel<true, false>)
                             : (p.aligned ? dequantize_kernel<false, true> : dequantize_kernel<false, false>);
  return launch_pdl(kern, grid, dim3(256), 0, st, p, tiles);
}

}  // namespace b128
}  // namespace gge
