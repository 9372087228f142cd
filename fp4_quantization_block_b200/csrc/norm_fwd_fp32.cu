// norm_fwd_fp32.cu -- layer norm forward for fp32 matrices.
#include "norm_fwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t forward<float>(const NormFwdArgs &, cudaStream_t);
}
}  // namespace fa4
