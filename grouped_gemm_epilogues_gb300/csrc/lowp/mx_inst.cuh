// Shared body of the block-scaled product's translation units.
#pragma once

#include "mx_gemm.cuh"

namespace gge {
namespace mx {

template <int BN, int CG, int FMT, bool TR>
cudaLaunchConfig_t mx_config(int grid, size_t smem, int cluster, cudaStream_t stream,
                             cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(MxCfg<BN, CG, FMT>::kThreads, 1, 1);
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

template <int BN, int CG, int FMT, bool TR>
cudaError_t mx_launch_one(const MxMaps& m, const MxParams& mp, const LaunchShape& shape,
                          cudaStream_t stream) {
  const cudaError_t e = allow_smem<mx_gemm_kernel<BN, CG, FMT, TR>>();
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  const cudaLaunchConfig_t cfg = mx_config<BN, CG, FMT, TR>(shape.grid, shape.smem, shape.cluster, stream, attr);
  return cudaLaunchKernelEx(&cfg, mx_gemm_kernel<BN, CG, FMT, TR>, m.a, m.b, m.sa, m.sb, mp);
}

// (Shared memory and registers; the tensor memory's columns need no count of their own: the
// registers leave room for one CTA an SM.)
template <int BN, int CG, int FMT, bool TR>
int mx_units_one(size_t smem, int cluster) {
  if (allow_smem<mx_gemm_kernel<BN, CG, FMT, TR>>() != cudaSuccess) return -1;
  if (cluster == 1) {
    int per_sm = 0, dev = 0, sms = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, mx_gemm_kernel<BN, CG, FMT, TR>,
                                                      MxCfg<BN, CG, FMT>::kThreads, smem) != cudaSuccess ||
        cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return -1;
    return per_sm * sms;
  }
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg = mx_config<BN, CG, FMT, TR>(cluster * 64, smem, cluster, nullptr, attr);
  cfg.attrs = attr + 1;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, mx_gemm_kernel<BN, CG, FMT, TR>, &cfg) != cudaSuccess) return -1;
  return n;
}

template <int FMT>
cudaError_t launch_mx(int tile, const MxMaps& maps, const MxParams& mp, const LaunchShape& shape,
                      cudaStream_t stream) {
  switch (tile) {
    case TILE_PAIR_256: return mx_launch_one<256, 2, FMT, false>(maps, mp, shape, stream);
    case TILE_128: return mx_launch_one<128, 1, FMT, false>(maps, mp, shape, stream);
    default: return mx_launch_one<64, 1, FMT, true>(maps, mp, shape, stream);
  }
}

template <int FMT>
int mx_units(int tile, size_t smem, int cluster) {
  switch (tile) {
    case TILE_PAIR_256: return mx_units_one<256, 2, FMT, false>(smem, cluster);
    case TILE_128: return mx_units_one<128, 1, FMT, false>(smem, cluster);
    default: return mx_units_one<64, 1, FMT, true>(smem, cluster);
  }
}

#define GGE_MX_INSTANTIATE(FMT)                                                                    \
  template cudaError_t launch_mx<FMT>(int, const MxMaps&, const MxParams&, const LaunchShape&,   \
                                      cudaStream_t);                                              \
  template int mx_units<FMT>(int, size_t, int);

}  // namespace mx
}  // namespace gge
