// norm_bwd_fp16.cu -- layer norm backward for fp16 matrices.
#include "norm_bwd.cuh"

namespace fa4 {
namespace norm {
template cudaError_t backward<__half>(const NormBwdArgs &, int *, cudaStream_t);
}
}  // namespace fa4
