// dropout.cu -- dropout from the counter-based generator, with or without the
// residual addition: y = [res +] (kept ? x * scale : 0), the mask computed
// from (key, row, column) where it is needed (rows.cuh) and never stored.
// The backward pass is the same map of dy under the same key.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace {

using namespace rows;

struct DropoutParams {
  const void *x, *res;
  void *y;
  int64_t ldx, ldres, ldy, T, N, chunks;
  Drop drop;
};

// One chunk of eight columns per thread and step.  y may be x or res itself:
// a thread reads its elements before it writes them.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) dropout_kernel(const DropoutParams p) {
  grid_dependency_wait();
  grid_dependents_launch();
  const uint64_t key = p.drop.key();
  const int64_t total = p.T * p.chunks;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / p.chunks, c = 8 * (i - r * p.chunks);
    float f[8];
    load8<T, VEC>(static_cast<const T *>(p.x) + r * p.ldx, c, p.N, f);
    drop8(p.drop, key, (uint32_t)r, (uint32_t)c, f);
    if (p.res) {
      float g[8];
      load8<T, VEC>(static_cast<const T *>(p.res) + r * p.ldres, c, p.N, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] += g[j];
    }
    store8<T, VEC>(static_cast<T *>(p.y) + r * p.ldy, c, p.N, f);
  }
}

inline bool vec_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

template <typename T>
cudaError_t launch(const DropoutArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.y, a.ldy) &&
                   (!a.res || vec_ok(a.res, a.ldres));
  const int64_t chunks = (a.N + 7) / 8;
  const DropoutParams p = {a.x, a.res, a.y, a.ldx, a.ldres, a.ldy, a.T, a.N, chunks,
                           {a.drop.seed, a.drop.step, a.drop.threshold, a.drop.scale}};
  const int64_t ctas = (a.T * chunks + 255) / 256;
  return launch_pdl(vec ? dropout_kernel<T, true> : dropout_kernel<T, false>,
                    dim3((unsigned)(ctas < 148 * 8 ? ctas : 148 * 8)), dim3(256), 0, st, p);
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs &a, cudaStream_t st) {
  switch (a.dtype) {
    case kBF16: return launch<__nv_bfloat16>(a, st);
    case kFP16: return launch<__half>(a, st);
    default: return launch<float>(a, st);
  }
}

}  // namespace fa4
