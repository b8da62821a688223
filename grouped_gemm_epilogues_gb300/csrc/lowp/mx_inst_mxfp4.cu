// Block-scaled product, mxfp4 operands.
#include "mx_inst.cuh"

namespace gge {
namespace mx {
GGE_MX_INSTANTIATE(FMT_MXFP4)
}  // namespace mx
}  // namespace gge
