// Launch entry points of the block-scaled product's instances (one translation
// unit a format).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "../gge_launch.h"
#include "../gge_params.h"

namespace gge {
namespace mx {

// gemm_kernel's parameters and what the block scales add
struct MxParams {
  Params p;
  const float *tscale_a, *tscale_b;  // fp32 scales of the whole operands, or NULL
  int32_t sfa_batch, sfb_batch;      // scale row tiles a batch
  int32_t splits;                    // CTAs of a cluster that share a tile's K: 1, 2, 4 or 8
  int32_t reduce_bytes;              // shared memory for the chunks they exchange
};

struct MxMaps {
  CUtensorMap a, b, sa, sb;
};

// Tile shapes: 256 x 256 on a CTA pair, 128 x 128 on one CTA, and 128 x 64 with
// the operands exchanged and the outputs stored transposed (few rows of A).
enum MxTile { TILE_PAIR_256 = 0, TILE_128 = 1, TILE_SWAP_64 = 2 };

template <int FMT>
cudaError_t launch_mx(int tile, const MxMaps& maps, const MxParams& mp, const LaunchShape& shape,
                      cudaStream_t stream);
// Resident CTAs, or clusters of `cluster` CTAs, on the current device, or -1.
template <int FMT>
int mx_units(int tile, size_t smem, int cluster);

}  // namespace mx
}  // namespace gge
