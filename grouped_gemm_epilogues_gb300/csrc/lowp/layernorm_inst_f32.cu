// Layer norm, float rows.
#include "layernorm.cuh"

namespace gge {
namespace b128 {
GGE_LN_INSTANTIATE(float)
}  // namespace b128
}  // namespace gge
