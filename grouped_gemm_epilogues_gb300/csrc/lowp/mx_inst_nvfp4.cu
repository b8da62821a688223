// Block-scaled product, nvfp4 operands.
#include "mx_inst.cuh"

namespace gge {
namespace mx {
GGE_MX_INSTANTIATE(FMT_NVFP4)
}  // namespace mx
}  // namespace gge
