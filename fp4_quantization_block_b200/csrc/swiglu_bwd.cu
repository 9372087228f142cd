// swiglu_bwd.cu -- backward pass of the SwiGLU activation whose forward pass
// is the producer of the down projection's input (quantize.cu).
//
// h = silu(g) u, silu(g) = g sg, sg = 1 / (1 + exp(-g)):
//   du = dh silu(g),   dg = dh u sg (1 + g (1 - sg)),
// in binary32, each rounded once to bf16.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace {

using namespace rows;

// One chunk of eight channels of h per thread and step.
__global__ void __launch_bounds__(256) swiglu_bwd_kernel(const SwigluBwdArgs p) {
  using T = __nv_bfloat16;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t chunks = p.F >> 3, total = p.T * chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / chunks, c = 8 * (i - r * chunks);
    const T *z = reinterpret_cast<const T *>(p.z) + r * p.ldz;
    T *dz = reinterpret_cast<T *>(p.dz) + r * p.lddz;
    float g[8], u[8], d[8];
    load8<T, true>(z, c, p.F, g);
    load8<T, true>(z + p.F, c, p.F, u);
    load8<T, true>(reinterpret_cast<const T *>(p.dh) + r * p.lddh, c, p.F, d);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float e = expf(-g[j]), sg = 1.0f / (1.0f + e);
      const float du = d[j] * (g[j] * sg);
      g[j] = d[j] * u[j] * (sg * fmaf(g[j], 1.0f - sg, 1.0f));
      u[j] = du;
    }
    store8<T, true>(dz, c, p.F, g);
    store8<T, true>(dz + p.F, c, p.F, u);
  }
}

}  // namespace

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs &a, cudaStream_t st) {
  const int64_t ctas = (a.T * (a.F >> 3) + 255) / 256;
  return launch_pdl(swiglu_bwd_kernel, dim3((unsigned)(ctas < 148 * 8 ? ctas : 148 * 8)), dim3(256), 0,
                    st, a);
}

}  // namespace fa4
