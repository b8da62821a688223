// Layer norm, __half rows.
#include "layernorm.cuh"

namespace gge {
namespace b128 {
GGE_LN_INSTANTIATE(__half)
}  // namespace b128
}  // namespace gge
