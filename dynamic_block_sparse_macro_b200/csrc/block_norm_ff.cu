// Block norms: the kernels for an f32 residual stream and f32 branches.
#include "block_norm.cuh"

namespace prism {
namespace bn {
PRISM_BN_INSTANTIATE(float, float)
}  // namespace bn
}  // namespace prism
