// norm.cuh -- layer normalisation forward and backward, alone or fused with
// dropout and the residual addition in front of it: what its kernels
// (norm_fwd.cuh, norm_bwd.cuh) share.
//
// A row x of N values (binary32 arithmetic, each stored value rounded once):
//   mu = mean(x) (0 in the RMS form), r = (mean((x - mu)^2) + eps)^-1/2,
//   xh = (x - mu) r,  y = w xh + b.
// Backward, with g = w dy:
//   dx = r (g - mean(g) - xh mean(g xh)) [+ dres]   (no mean(g) in the RMS form)
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
// Fused: s = residual + dropout(x), stored, and x = the stored s above;
// backward: dres = the dx above, and dx = dropout of it.
//
// The variance is a second pass over the row's values, which stay on the
// chip: one-pass sums of squares lose the variance of rows whose mean is
// large.  The weight's and the bias's gradients are summed in a fixed order
// (per CTA, then over the CTAs), with no atomics, so a call repeats bit for
// bit.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace norm {

using namespace rows;

// How a launch lays rows over threads.
struct Layout {
  int warps;    // of a team (one row, or a cluster's CTA's share of it)
  int teams;    // of a CTA
  int stages;   // of the ring
  int cluster;  // CTAs that share rows (backward)
  int wvec;     // weight and bias start on 16-byte boundaries
  // Team q of all takes the rows q, q + step, ...: base of them, one more
  // where q < extra.
  uint32_t step;
  int base;
  uint32_t extra;
  __device__ __forceinline__ int rows(uint32_t q) const { return base + (q < extra ? 1 : 0); }
  void share(int64_t T, int64_t all_teams) {
    step = (uint32_t)all_teams;
    base = (int)(T / all_teams);
    extra = (uint32_t)(T % all_teams);
  }
};

constexpr int kSms = 148;
constexpr int kMaxClusters[4] = {148, 74, 33, 15};  // of 1, 2, 4 and 8 CTAs that run at once, one per SM
constexpr size_t kMaxSmem = 224 * 1024;  // the static arrays' share left out
constexpr int kBwdWarps = 16;                // of a CTA of the backward pass
constexpr int kBwdRow = kBwdWarps * 2 * kTile;  // the columns that it holds at most
constexpr int kWideThreads = 512;

// Sum over the CTA's threads, the same bits in each of them.
__device__ __forceinline__ float cta_sum(float v, float *red) {
  v = warp_sum(v);
  __syncthreads();  // the last sum's readers are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.0f);
}

inline int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }
inline bool vec_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}
inline unsigned row_ctas(int64_t T) { return (unsigned)(T < kSms * 4 ? T : kSms * 4); }
// Row groups of the wide dw pass, so that its CTAs fill the GPU twice over.
inline int wide_splits(int64_t T, int64_t N) {
  const int64_t strips = (N + 255) / 256, groups = (T + 7) / 8;
  int64_t s = (kSms * 8 + strips - 1) / strips;
  s = s < groups ? s : groups;
  return (int)(s < 1 ? 1 : s > kMaxNormPartials ? kMaxNormPartials : s);
}
inline Drop make_drop(const DropArgs &d) { return {d.seed, d.step, d.threshold, d.scale}; }

template <typename K, typename P>
cudaError_t launch_rows(K kern, const P &p, const Layout &g, size_t smem, int ctas, cudaStream_t st) {
  // The limit belongs to the kernel, not to the launch: every call sets the
  // same one, so that a call from another thread, for other rows, cannot lower
  // it between here and the launch.
  if (smem > 40 * 1024) {  // static shared memory counts towards the default 48 KB too
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(32 * g.warps * g.teams);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {pdl_attribute()};
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)g.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = g.cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, p, g);
}

// The calls for one type of the matrices (norm_fwd_bf16.cu, norm_bwd_bf16.cu
// and their like for fp16 and fp32).  backward: *n partial sums of dw and db are left in
// a.partials, none where they are done.
template <typename T>
cudaError_t forward(const NormFwdArgs &a, cudaStream_t st);
template <typename T>
cudaError_t backward(const NormBwdArgs &a, int *n, cudaStream_t st);

}  // namespace norm
}  // namespace fa4
