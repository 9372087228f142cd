// norm_bwd_bf16.cu -- layer norm backward for bf16 matrices.
#include "norm_bwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t backward<__nv_bfloat16>(const NormBwdArgs &, int *, cudaStream_t);
}
}  // namespace fa4
