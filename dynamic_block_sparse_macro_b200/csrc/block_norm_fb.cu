// Block norms: the kernels for an f32 residual stream and bf16 branches.
#include "block_norm.cuh"

namespace prism {
namespace bn {
PRISM_BN_INSTANTIATE(float, __nv_bfloat16)
}  // namespace bn
}  // namespace prism
