// norm.cu -- the layer norm calls: by the matrices' type to their kernels, and
// the last sums of the weight's and the bias's gradients.
#include "norm.cuh"

namespace fa4 {
namespace {

// dw[c] and db[c] = the sums of n partials [n][2][N]: 32 columns per CTA, 16
// threads to a column, ten partials of a thread in flight at a time.
constexpr int kSumThreads = 512;
__global__ void __launch_bounds__(kSumThreads)
    norm_colsum_kernel(const float *partials, int n, int64_t N, float *dw, float *db) {
  __shared__ float part[16][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int cx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = 32 * (int64_t)blockIdx.x + cx, k = blockIdx.y;
  float v = 0.0f;
  if (c < N)
#pragma unroll 10
    for (int i = ty; i < n; i += 16) v += partials[((int64_t)i * 2 + k) * N + c];
  part[ty][cx] = v;
  __syncthreads();
  if (ty == 0 && c < N) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][cx];
    (k ? db : dw)[c] = v;
  }
}

}  // namespace

// As many partial sums as there can be clusters at once (launch_bwd), or row
// groups where rows are too long for a cluster; never more than rows.
int norm_partials_count(int64_t T, int64_t N) {
  int n = norm::wide_splits(T, N);
  for (int log = 3; log >= 0; --log)
    if (N <= (int64_t)norm::kBwdRow << log) n = norm::kMaxClusters[log];
  return T < n ? (int)T : n;
}

cudaError_t launch_norm_fwd(const NormFwdArgs &a, cudaStream_t st) {
  switch (a.dtype) {
    case kBF16: return norm::forward<__nv_bfloat16>(a, st);
    case kFP16: return norm::forward<__half>(a, st);
    default: return norm::forward<float>(a, st);
  }
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t st) {
  int n = 0;
  cudaError_t e;
  switch (a.dtype) {
    case kBF16: e = norm::backward<__nv_bfloat16>(a, &n, st); break;
    case kFP16: e = norm::backward<__half>(a, &n, st); break;
    default: e = norm::backward<float>(a, &n, st);
  }
  if (e != cudaSuccess || n == 0) return e;
  return launch_pdl(norm_colsum_kernel, dim3((unsigned)((a.N + 31) / 32), a.db ? 2u : 1u), dim3(kSumThreads),
                    0, st, a.partials, n, a.N, a.dw, a.db);
}

}  // namespace fa4
