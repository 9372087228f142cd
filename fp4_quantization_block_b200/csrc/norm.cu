// norm.cu -- layer normalisation forward and backward, alone or fused with
// dropout and the residual addition in front of it.
//
// A row x of N values (binary32 arithmetic, each stored value rounded once):
//   mu = mean(x) (0 in the RMS form), r = (mean((x - mu)^2) + eps)^-1/2,
//   xh = (x - mu) r,  y = w xh + b.
// Backward, with g = w dy:
//   dx = r (g - mean(g) - xh mean(g xh)) [+ dres]   (no mean(g) in the RMS form)
//   dw = sum over rows of dy xh,  db = sum over rows of dy.
// Fused: s = residual + dropout(x), stored, and x = the stored s above;
// backward: dres = the dx above, and dx = dropout(dres).
//
// The variance is a second pass over the row's values, which stay on the
// chip: one-pass sums of squares lose the variance of rows whose mean is
// large.  The weight's and the bias's gradients are summed in a fixed order
// (per CTA, then over the CTAs), with no atomics, so a call repeats bit for
// bit.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace {

using namespace rows;

struct FwdParams {
  const void *x, *res;
  int64_t ldx, ldres, T, N;
  const void *w, *b;
  int w_f32, center;
  float eps;
  void *y, *s;
  int64_t ldy, lds;
  float *mean, *rstd;
  Drop drop;
};
struct BwdParams {
  const void *dy, *x, *ds;
  int64_t lddy, ldx, ldds, T, N;
  const void *w;
  int w_f32, center;
  const float *mean, *rstd;
  void *dx, *dres;
  int64_t lddx, lddres;
  float *partials;  // [CTA][2][N]
  Drop drop;
};

// Sum over the CTA's threads, the same bits in each of them.
__device__ __forceinline__ float cta_sum(float v, float *red) {
  v = warp_sum(v);
  __syncthreads();  // the last sum's readers are done
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  return warp_sum((threadIdx.x & 31) < (blockDim.x >> 5) ? red[threadIdx.x & 31] : 0.0f);
}

constexpr int kWideThreads = 512;

// One CTA per row, the row read again for each pass.
template <typename T, bool VEC, bool FUSED>
__global__ void __launch_bounds__(kWideThreads) norm_fwd_wide_kernel(const FwdParams p) {
  __shared__ float red[32];
  grid_dependency_wait();
  grid_dependents_launch();
  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  const Vec<T> w{p.w, p.w_f32}, b{p.b, p.w_f32};
  for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + r * p.ldx;
    T *y = static_cast<T *>(p.y) + r * p.ldy;
    float sum = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kWideThreads) {
      float f[8];
      load8<T, VEC>(x, c, p.N, f);
      if constexpr (FUSED) {
        float g[8];
        drop8(p.drop, key, (uint32_t)r, (uint32_t)c, f);
        load8<T, VEC>(static_cast<const T *>(p.res) + r * p.ldres, c, p.N, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += g[i];
        round8<T>(f);
        store8<T, VEC>(static_cast<T *>(p.s) + r * p.lds, c, p.N, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < p.N ? f[i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += f[i];
    }
    // a thread reads back the columns of s that it wrote
    const T *v = FUSED ? static_cast<const T *>(p.s) + r * p.lds : x;
    const float mean = p.center ? cta_sum(sum, red) / (float)p.N : 0.0f;
    float m2 = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kWideThreads) {
      float f[8];
      load8<T, VEC>(v, c, p.N, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = f[i] - mean;
        m2 += c + i < p.N ? d * d : 0.0f;
      }
    }
    const float rstd = __frsqrt_rn(cta_sum(m2, red) / (float)p.N + p.eps);
    if (threadIdx.x == 0) {
      if (p.center) p.mean[r] = mean;
      p.rstd[r] = rstd;
    }
    for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kWideThreads) {
      float f[8];
      load8<T, VEC>(v, c, p.N, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int64_t k = c + i < p.N ? c + i : 0;
        f[i] = fmaf((f[i] - mean) * rstd, w.at(k), p.b ? b.at(k) : 0.0f);
      }
      store8<T, VEC>(y, c, p.N, f);
    }
  }
}

// dx of one row per CTA.
template <typename T, bool VEC, bool FUSED>
__global__ void __launch_bounds__(kWideThreads) norm_dx_wide_kernel(const BwdParams p) {
  __shared__ float red[32];
  grid_dependency_wait();
  grid_dependents_launch();
  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  const Vec<T> w{p.w, p.w_f32};
  for (int64_t r = blockIdx.x; r < p.T; r += gridDim.x) {
    const T *x = static_cast<const T *>(p.x) + r * p.ldx;
    const T *dy = static_cast<const T *>(p.dy) + r * p.lddy;
    const float mean = p.center ? p.mean[r] : 0.0f, rstd = p.rstd[r];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kWideThreads) {
      float f[8], g[8];
      load8<T, VEC>(x, c, p.N, f);
      load8<T, VEC>(dy, c, p.N, g);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < p.N) {
          const float gi = g[i] * w.at(c + i);
          c1 += gi;
          c2 = fmaf(gi, (f[i] - mean) * rstd, c2);
        }
    }
    c1 = p.center ? cta_sum(c1, red) / (float)p.N : 0.0f;
    c2 = cta_sum(c2, red) / (float)p.N;
    for (int64_t c = 8 * threadIdx.x; c < p.N; c += 8 * kWideThreads) {
      float f[8], g[8], d[8];
      load8<T, VEC>(x, c, p.N, f);
      load8<T, VEC>(dy, c, p.N, g);
      if (p.ds) load8<T, VEC>(static_cast<const T *>(p.ds) + r * p.ldds, c, p.N, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * w.at(c + i < p.N ? c + i : 0);
        f[i] = fmaf(-(f[i] - mean) * rstd, c2, gi - c1) * rstd + (p.ds ? d[i] : 0.0f);
      }
      if constexpr (FUSED) {
        store8<T, VEC>(static_cast<T *>(p.dres) + r * p.lddres, c, p.N, f);
        drop8(p.drop, key, (uint32_t)r, (uint32_t)c, f);
      }
      store8<T, VEC>(static_cast<T *>(p.dx) + r * p.lddx, c, p.N, f);
    }
  }
}

// Partial sums of dw and db: CTA (bx, by) takes the columns 256 bx .. 256 bx
// + 255 and every gridDim.y-th group of eight rows; a warp takes one row of
// the group.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) norm_dw_wide_kernel(const BwdParams p) {
  __shared__ float part[8][2][256];
  grid_dependency_wait();
  grid_dependents_launch();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t c = 256 * (int64_t)blockIdx.x + 8 * lane;
  float dw[8] = {}, db[8] = {};
  for (int64_t r = 8 * (int64_t)blockIdx.y + warp; r < p.T; r += 8 * (int64_t)gridDim.y) {
    float f[8], g[8];
    load8<T, VEC>(static_cast<const T *>(p.x) + r * p.ldx, c, p.N, f);
    load8<T, VEC>(static_cast<const T *>(p.dy) + r * p.lddy, c, p.N, g);
    const float mean = p.center ? p.mean[r] : 0.0f, rstd = p.rstd[r];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[i] = fmaf(g[i], (f[i] - mean) * rstd, dw[i]);
      db[i] += g[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    part[warp][0][8 * lane + i] = dw[i];
    part[warp][1][8 * lane + i] = db[i];
  }
  __syncthreads();
  const int64_t col = 256 * (int64_t)blockIdx.x + threadIdx.x;
  if (col >= p.N) return;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][k][threadIdx.x];
    p.partials[((int64_t)blockIdx.y * 2 + k) * p.N + col] = v;
  }
}

// dw[c] and db[c] = the sums of n partials [n][2][N]: 32 columns per CTA,
// eight threads to a column.
__global__ void __launch_bounds__(256)
    norm_colsum_kernel(const float *partials, int n, int64_t N, float *dw, float *db) {
  __shared__ float part[8][32];
  grid_dependency_wait();
  grid_dependents_launch();
  const int cx = threadIdx.x & 31, ty = threadIdx.x >> 5;
  const int64_t c = 32 * (int64_t)blockIdx.x + cx, k = blockIdx.y;
  float v = 0.0f;
  if (c < N)
    for (int i = ty; i < n; i += 8) v += partials[((int64_t)i * 2 + k) * N + c];
  part[ty][cx] = v;
  __syncthreads();
  if (ty == 0 && c < N) {
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i][cx];
    (k ? db : dw)[c] = v;
  }
}

Drop make_drop(const DropArgs &d) { return {d.seed, d.step, d.threshold, d.scale}; }

inline bool vec_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

template <typename F>
cudaError_t by_type(int dtype, F &&f) {
  switch (dtype) {
    case kBF16: return f(__nv_bfloat16());
    case kFP16: return f(__half());
    default: return f(float());
  }
}

unsigned row_ctas(int64_t T) { return (unsigned)(T < 148 * 4 ? T : 148 * 4); }
// row groups of the dw pass, so that its CTAs fill the GPU twice over
int wide_splits(int64_t T, int64_t N) {
  const int64_t strips = (N + 255) / 256, groups = (T + 7) / 8;
  int64_t s = (148 * 8 + strips - 1) / strips;
  s = s < groups ? s : groups;
  return (int)(s < 1 ? 1 : s > kMaxNormPartials ? kMaxNormPartials : s);
}

}  // namespace

int norm_partials_count(int64_t T, int64_t N) { return wide_splits(T, N); }

cudaError_t launch_norm_fwd(const NormFwdArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.y, a.ldy) &&
                   (!a.fused || (vec_ok(a.res, a.ldres) && vec_ok(a.s, a.lds)));
  const FwdParams p = {a.x, a.res, a.ldx, a.ldres, a.T,   a.N,    a.w,    a.b, a.w_f32, a.center,
                       a.eps, a.y, a.s,   a.ldy,   a.lds, a.mean, a.rstd, make_drop(a.drop)};
  return by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto kern = a.fused ? (vec ? norm_fwd_wide_kernel<T, true, true> : norm_fwd_wide_kernel<T, false, true>)
                        : (vec ? norm_fwd_wide_kernel<T, true, false> : norm_fwd_wide_kernel<T, false, false>);
    return launch_pdl(kern, dim3(row_ctas(a.T)), dim3(kWideThreads), 0, st, p);
  });
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.dy, a.lddy) && vec_ok(a.x, a.ldx) &&
                   vec_ok(a.dx, a.lddx) && (!a.ds || vec_ok(a.ds, a.ldds)) &&
                   (!a.fused || vec_ok(a.dres, a.lddres));
  const BwdParams p = {a.dy, a.x, a.ds, a.lddy, a.ldx, a.ldds, a.T, a.N, a.w, a.w_f32, a.center,
                       a.mean, a.rstd, a.dx, a.dres, a.lddx, a.lddres, a.partials,
                       make_drop(a.drop)};
  const int splits = wide_splits(a.T, a.N);
  cudaError_t e = by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    auto kern = a.fused ? (vec ? norm_dx_wide_kernel<T, true, true> : norm_dx_wide_kernel<T, false, true>)
                        : (vec ? norm_dx_wide_kernel<T, true, false> : norm_dx_wide_kernel<T, false, false>);
    // dw first: dx may take the place of dy or x
    auto dwk = vec ? norm_dw_wide_kernel<T, true> : norm_dw_wide_kernel<T, false>;
    const cudaError_t e1 =
        launch_pdl(dwk, dim3((unsigned)((a.N + 255) / 256), (unsigned)splits), dim3(256), 0, st, p);
    if (e1 != cudaSuccess) return e1;
    return launch_pdl(kern, dim3(row_ctas(a.T)), dim3(kWideThreads), 0, st, p);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_colsum_kernel, dim3((unsigned)((a.N + 31) / 32), a.db ? 2u : 1u), dim3(256), 0,
                    st, a.partials, splits, a.N, a.dw, a.db);
}

}  // namespace fa4
