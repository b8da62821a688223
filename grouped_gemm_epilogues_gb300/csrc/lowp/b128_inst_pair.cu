// Product with a scale for each block of 128, 256-wide tiles on a CTA pair.
#include "b128_gemm.cuh"

namespace gge {
namespace b128 {
GGE_B128_INSTANTIATE(256, 2)
}  // namespace b128
}  // namespace gge
