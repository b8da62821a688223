// Block-scaled product, mxfp8 operands.
#include "mx_inst.cuh"

namespace gge {
namespace mx {
GGE_MX_INSTANTIATE(FMT_MXFP8)
}  // namespace mx
}  // namespace gge
