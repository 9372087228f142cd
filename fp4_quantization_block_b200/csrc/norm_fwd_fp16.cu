// norm_fwd_fp16.cu -- layer norm forward for fp16 matrices.
#include "norm_fwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t forward<__half>(const NormFwdArgs &, cudaStream_t);
}
}  // namespace fa4
