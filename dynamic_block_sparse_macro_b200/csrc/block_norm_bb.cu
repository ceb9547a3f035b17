// Block norms: the kernels for a bf16 residual stream and bf16 branches.
#include "block_norm.cuh"

namespace prism {
namespace bn {
PRISM_BN_INSTANTIATE(__nv_bfloat16, __nv_bfloat16)
}  // namespace bn
}  // namespace prism
