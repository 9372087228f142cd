// norm_bwd_fp32.cu -- layer norm backward for fp32 matrices.
#include "norm_bwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t backward<float>(const NormBwdArgs &, int *, cudaStream_t);
}
}  // namespace fa4
