// norm.cu -- the layer norm calls: by the matrices' type to their kernels, and
// the last sums of the weight's and the bias's gradients.
#include "norm.cuh"

namespace fa4 {
namespace {

// dw[c] and db[c] = the sums of n partials [n][2][N]: 32 V columns per CTA, V
// (consecutive) per thread, kSplits threads to a column, so that of the 148
// partials a thread has its five in flight at once.  What it costs is its
// latency: 3 us of the 48 at 8192 x 4096 (with 16 threads to a column 4).
constexpr int kSplits = 32;
constexpr int kSumThreads = 32 * kSplits;
template <int V>
__global__ void __launch_bounds__(kSumThreads)
    norm_colsum_kernel(const float *partials, int n, int64_t N, float *dw, float *db) {
  __shared__ float part[kSplits][32 * V];
  grid_dependency_wait();
  grid_dependents_launch();
  const int cx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = V * (32 * (int64_t)blockIdx.x + cx), k = blockIdx.y;
  float v[V] = {};
  if (c < N)
#pragma unroll 5
    for (int i = ty; i < n; i += kSplits) {
      const float *p = partials + ((int64_t)i * 2 + k) * N + c;
      if constexpr (V == 2) {
        const float2 q = *reinterpret_cast<const float2 *>(p);
        v[0] += q.x, v[1] += q.y;
      } else {
        v[0] += *p;
      }
    }
#pragma unroll
  for (int j = 0; j < V; ++j) part[ty][V * cx + j] = v[j];
  __syncthreads();
  const int64_t base = 32 * V * (int64_t)blockIdx.x;
  for (int j = threadIdx.x; j < 32 * V; j += kSumThreads)
    if (base + j < N) {
      float t = 0.0f;
#pragma unroll
      for (int i = 0; i < kSplits; ++i) t += part[i][j];
      (k ? db : dw)[base + j] = t;
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
  const int v = a.N % 2 == 0 ? 2 : 1;
  return launch_pdl(v == 2 ? norm_colsum_kernel<2> : norm_colsum_kernel<1>,
                    dim3((unsigned)((a.N + 32 * v - 1) / (32 * v)), a.db ? 2u : 1u), dim3(kSumThreads), 0, st,
                    a.partials, n, a.N, a.dw, a.db);
}

}  // namespace fa4
