// Product with a scale for each block of 128, 128-wide tiles on one CTA.
#include "b128_gemm.cuh"

namespace gge {
namespace b128 {
GGE_B128_INSTANTIATE(128, 1)
}  // namespace b128
}  // namespace gge
