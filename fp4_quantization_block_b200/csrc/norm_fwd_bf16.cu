// norm_fwd_bf16.cu -- layer norm forward for bf16 matrices.
#include "norm_fwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t forward<__nv_bfloat16>(const NormFwdArgs &, cudaStream_t);
}
}  // namespace fa4
