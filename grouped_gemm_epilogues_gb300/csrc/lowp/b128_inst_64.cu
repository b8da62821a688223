// Product with a scale for each block of 128, 64-wide tiles on one CTA.
#include "b128_gemm.cuh"

namespace gge {
namespace b128 {
GGE_B128_INSTANTIATE(64, 1)
}  // namespace b128
}  // namespace gge
