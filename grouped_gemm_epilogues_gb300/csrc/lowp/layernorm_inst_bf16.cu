// Layer norm, __nv_bfloat16 rows.
#include "layernorm.cuh"

namespace gge {
namespace b128 {
GGE_LN_INSTANTIATE(__nv_bfloat16)
}  // namespace b128
}  // namespace gge
