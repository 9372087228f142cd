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

// ------------------------------------------------ rows kept on the chip ---
// How a launch lays rows over threads (host rule: choose_layout).
struct Layout {
  int warps;   // of a team (one row)
  int teams;   // of a CTA
  int stages;  // of the ring
  int words;   // 16-bit rows start on 4-byte boundaries (unaligned kernels)
  int wvec;    // weight and bias start on 16-byte boundaries
};

// Threads a CTA may have for the registers of CH chunks.
constexpr int fwd_threads(int ch) { return ch <= 4 ? 768 : ch == 8 ? 512 : 384; }

// Each team takes every (gridDim.x * teams)-th row, CH chunks per thread; the
// weight and the bias lie in shared memory.
template <typename T, typename W, int CH, bool VEC, bool FUSED>
__global__ void __launch_bounds__(fwd_threads(CH), 1) norm_fwd_kernel(const FwdParams p, const Layout g) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][32];
  constexpr int A = FUSED ? 2 : 1, kStage = A * CH * kTile;
  const int lane = threadIdx.x & 31, cta_warp = threadIdx.x >> 5;
  const int team = cta_warp / g.warps, warp = cta_warp - team * g.warps;
  const int col = warp * CH * kTile, left = (int)p.N - col;  // the warp's columns
  T *const ring = reinterpret_cast<T *>(smem) + (size_t)cta_warp * g.stages * kStage;
  T *const ring_end = ring + g.stages * kStage;
  const int room = g.warps * CH * kTile;
  W *const wsm = reinterpret_cast<W *>(smem + (size_t)g.warps * g.teams * g.stages * kStage * sizeof(T));
  W *const bsm = wsm + room;
  float *red0 = &red[0][team * g.warps], *red1 = &red[1][team * g.warps];
  const int64_t step = (int64_t)gridDim.x * g.teams, row0 = (int64_t)blockIdx.x * g.teams + team;
#pragma unroll
  for (int j = 0; j < CH; ++j)
    if (left - j * kTile < kTile)
      for (int s = 0; s < A * g.stages; ++s) clear_tail(ring + (s * CH + j) * kTile, left - j * kTile, lane);
  __syncwarp();
  grid_dependency_wait();
  grid_dependents_launch();
  stage_vec<T, W>(wsm, static_cast<const W *>(p.w), (int)p.N, room, g.wvec);
  stage_vec<T, W>(bsm, static_cast<const W *>(p.b), p.b ? (int)p.N : 0, room, g.wvec);

  const T *fx = static_cast<const T *>(p.x) + row0 * p.ldx + col;
  const T *fr = FUSED ? static_cast<const T *>(p.res) + row0 * p.ldres + col : nullptr;
  int64_t frow = row0;
  T *ft = ring;
  auto fill = [&]() {  // the next row of the team into the next stage
    if (frow < p.T) {
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        fill_tile<T, VEC>(ft + j * kTile, fx + j * kTile, left - j * kTile, g.words, lane);
        if constexpr (FUSED)
          fill_tile<T, VEC>(ft + (CH + j) * kTile, fr + j * kTile, left - j * kTile, g.words, lane);
      }
      fx += step * p.ldx;
      if constexpr (FUSED) fr += step * p.ldres;
      frow += step;
    }
    ft = ft + kStage == ring_end ? ring : ft + kStage;
    cp_async_commit();
  };
  for (int s = 0; s < g.stages - 1; ++s) fill();
  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  const float inv_n = 1.0f / (float)p.N;
  T *y = static_cast<T *>(p.y) + row0 * p.ldy + col;
  T *sp = FUSED ? static_cast<T *>(p.s) + row0 * p.lds + col : nullptr;

  if (g.stages == 1) cp_async_commit();
  cp_async_wait(g.stages > 1 ? g.stages - 2 : 0);  // the oldest group holds the weights
  __syncthreads();

  T *t = ring;
  for (int64_t row = row0; row < p.T; row += step) {
    __syncwarp();  // the stage filled next was read by the whole warp
    fill();
    cp_async_wait(g.stages - 1);
    __syncwarp();
    uint64_t v[CH][4], acc = 0ull;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      read_tile(t + j * kTile, lane, v[j]);
      if constexpr (FUSED) {
        uint64_t r[4];
        drop_tile<T>(p.drop, key, (uint32_t)row, (uint32_t)(col + j * kTile) / 8, lane, v[j]);
        read_tile(t + (CH + j) * kTile, lane, r);
        Raw8<T> raw;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = f2_add(v[j][i], r[i]);
        pack8(v[j], raw);
        unpack8(raw, v[j]);  // the stored s
        store_tile<T, VEC>(t + j * kTile, sp + j * kTile, left - j * kTile, g.words, lane, v[j]);
      }
      acc = f2_add(acc, f2_add(f2_add(v[j][0], v[j][1]), f2_add(v[j][2], v[j][3])));
    }
    float mean = 0.0f;
    if (p.center) {
      float sum[1] = {f2_sum(acc)};
      team_sum<1>(sum, red0, g.warps, warp, lane, 1 + team);
      mean = sum[0] * inv_n;
    }
    const uint64_t shift = f2_set(-mean);
    float m2[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      // what lies past the row's end is -mean now and does not count
      uint64_t sq = 0ull;
      if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = f2_add(v[j][i], shift);
        uint64_t hi = f2_fma(v[j][2], v[j][2], f2_mul(v[j][3], v[j][3]));
        sq = f2_fma(v[j][0], v[j][0], f2_mul(v[j][1], v[j][1]));
        if (j * kTile + pair_col<T>(lane, 2) >= left) hi = 0ull;
        if (j * kTile + pair_col<T>(lane, 0) >= left) sq = 0ull;
        sq = f2_add(sq, hi);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = j * kTile + pair_col<T>(lane, i);
          v[j][i] = f2_add(v[j][i], shift);
          v[j][i] = f2_pack(c < left ? f2_lo(v[j][i]) : 0.0f, c + 1 < left ? f2_hi(v[j][i]) : 0.0f);
          sq = f2_fma(v[j][i], v[j][i], sq);
        }
      }
      m2[0] += f2_sum(sq);
    }
    team_sum<1>(m2, red1, g.warps, warp, lane, 1 + team);
    const float rstd = rsqrtf(m2[0] * inv_n + p.eps);
    if (warp == 0 && lane == 0) {
      if (p.center) p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    const uint64_t scale = f2_set(rstd);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      uint64_t w[4], b[4];
      read_vec<T, W>(wsm + col + j * kTile, lane, w);
      read_vec<T, W>(bsm + col + j * kTile, lane, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = f2_fma(f2_mul(v[j][i], scale), w[i], b[i]);
      store_tile<T, VEC>(t + j * kTile, y + j * kTile, left - j * kTile, g.words, lane, v[j]);
    }
    // without centring the one barrier of a row does not keep the next row's
    // sums from this row's readers
    if (!p.center) {
      float *q = red0;
      red0 = red1;
      red1 = q;
    }
    y += step * p.ldy;
    if constexpr (FUSED) sp += step * p.lds;
    t = t + kStage == ring_end ? ring : t + kStage;
  }
}

// dx of a team's rows; dw and db of its columns stay in registers over its
// rows, are added up over the CTA's teams in order and go to the CTA's
// partial sums.  Up to two chunks per thread xh and g stay in registers
// between the two passes over a row; with four there is no room, and they are
// computed again.
template <typename T, typename W, int CH, bool VEC, bool FUSED>
__global__ void __launch_bounds__(512, 1) norm_bwd_kernel(const BwdParams p, const Layout g) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float red[2][32];
  constexpr bool KEEP = CH <= 2;
  constexpr int kHead = 16 / (int)sizeof(T);  // a stage starts with the row's mean and rstd
  const int lane = threadIdx.x & 31, cta_warp = threadIdx.x >> 5;
  const int team = cta_warp / g.warps, warp = cta_warp - team * g.warps;
  const int col = warp * CH * kTile, left = (int)p.N - col;  // the warp's columns
  const int arrays = p.ds ? 3 : 2, stage_len = arrays * CH * kTile + kHead;
  T *const ring = reinterpret_cast<T *>(smem) + (size_t)cta_warp * g.stages * stage_len;
  T *const ring_end = ring + g.stages * stage_len;
  float *red0 = &red[0][2 * team * g.warps], *red1 = &red[1][2 * team * g.warps];
  const int64_t step = (int64_t)gridDim.x * g.teams, row0 = (int64_t)blockIdx.x * g.teams + team;
#pragma unroll
  for (int j = 0; j < CH; ++j)
    if (left - j * kTile < kTile)
      for (T *s = ring + kHead; s < ring_end; s += stage_len)
        for (int a = 0; a < arrays; ++a) clear_tail(s + (a * CH + j) * kTile, left - j * kTile, lane);
  __syncwarp();
  grid_dependency_wait();
  grid_dependents_launch();
  const int room = g.warps * CH * kTile;
  W *const wsm = reinterpret_cast<W *>(smem + (size_t)g.warps * g.teams * g.stages * stage_len * sizeof(T));
  stage_vec<T, W>(wsm, static_cast<const W *>(p.w), (int)p.N, room, g.wvec);

  const T *fx = static_cast<const T *>(p.x) + row0 * p.ldx + col;
  const T *fdy = static_cast<const T *>(p.dy) + row0 * p.lddy + col;
  const T *fds = p.ds ? static_cast<const T *>(p.ds) + row0 * p.ldds + col : nullptr;
  int64_t frow = row0;
  T *ft = ring;
  auto fill = [&]() {  // the next row of the team into the next stage
    if (frow < p.T) {
      if (lane == 0) {
        if (p.center) cp_async4(ft, p.mean + frow);
        cp_async4(reinterpret_cast<float *>(ft) + 1, p.rstd + frow);
      }
      T *const t = ft + kHead;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        fill_tile<T, VEC>(t + j * kTile, fx + j * kTile, left - j * kTile, g.words, lane);
        fill_tile<T, VEC>(t + (CH + j) * kTile, fdy + j * kTile, left - j * kTile, g.words, lane);
        if (p.ds)
          fill_tile<T, VEC>(t + (2 * CH + j) * kTile, fds + j * kTile, left - j * kTile, g.words, lane);
      }
      fx += step * p.ldx;
      fdy += step * p.lddy;
      fds += step * p.ldds;
      frow += step;
    }
    ft = ft + stage_len == ring_end ? ring : ft + stage_len;
    cp_async_commit();
  };
  for (int s = 0; s < g.stages - 1; ++s) fill();

  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  uint64_t w[KEEP ? CH : 1][4], dw[CH][4], db[CH][4];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = 0ull;
  if (g.stages == 1) cp_async_commit();
  cp_async_wait(g.stages > 1 ? g.stages - 2 : 0);  // the oldest group holds the weight
  __syncthreads();
  if constexpr (KEEP) {
#pragma unroll
    for (int j = 0; j < CH; ++j) read_vec<T, W>(wsm + col + j * kTile, lane, w[j]);
  }
  const float inv_n = 1.0f / (float)p.N;
  T *dx = static_cast<T *>(p.dx) + row0 * p.lddx + col;
  T *dres = FUSED ? static_cast<T *>(p.dres) + row0 * p.lddres + col : nullptr;

  T *t = ring;
  for (int64_t row = row0; row < p.T; row += step) {
    __syncwarp();  // the stage filled next was read by the whole warp
    fill();
    cp_async_wait(g.stages - 1);
    __syncwarp();
    const float rstd = reinterpret_cast<const float *>(t)[1];
    const uint64_t scale = f2_set(rstd);
    const uint64_t shift = f2_set(p.center ? -reinterpret_cast<const float *>(t)[0] : 0.0f);
    T *const tile = t + kHead;
    uint64_t xh[KEEP ? CH : 1][4], gg[KEEP ? CH : 1][4], s1 = 0ull, s2 = 0ull;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int k = KEEP ? j : 0;
      uint64_t dy[4];
      read_tile(tile + j * kTile, lane, xh[k]);
      read_tile(tile + (CH + j) * kTile, lane, dy);
      if constexpr (!KEEP) read_vec<T, W>(wsm + col + j * kTile, lane, w[0]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        xh[k][i] = f2_mul(f2_add(xh[k][i], shift), scale);
        gg[k][i] = f2_mul(dy[i], w[k][i]);
        dw[j][i] = f2_fma(dy[i], xh[k][i], dw[j][i]);
        db[j][i] = f2_add(db[j][i], dy[i]);
        s1 = f2_add(s1, gg[k][i]);
        s2 = f2_fma(gg[k][i], xh[k][i], s2);
      }
    }
    float c12[2] = {f2_sum(s1), f2_sum(s2)};
    team_sum<2>(c12, red0, g.warps, warp, lane, 1 + team);
    {
      float *q = red0;
      red0 = red1;
      red1 = q;
    }
    const uint64_t c1 = f2_set(p.center ? -c12[0] * inv_n : 0.0f), c2 = f2_set(-c12[1] * inv_n);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      const int k = KEEP ? j : 0;
      uint64_t d[4];
      if constexpr (!KEEP) {
        read_tile(tile + j * kTile, lane, xh[0]);
        read_tile(tile + (CH + j) * kTile, lane, gg[0]);
        read_vec<T, W>(wsm + col + j * kTile, lane, w[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xh[0][i] = f2_mul(f2_add(xh[0][i], shift), scale);
          gg[0][i] = f2_mul(gg[0][i], w[0][i]);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f2_fma(xh[k][i], c2, f2_add(gg[k][i], c1));
      if (p.ds) {
        uint64_t r[4];
        read_tile(tile + (2 * CH + j) * kTile, lane, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = f2_fma(d[i], scale, r[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = f2_mul(d[i], scale);
      }
      if constexpr (FUSED) {
        store_tile<T, VEC>(tile + j * kTile, dres + j * kTile, left - j * kTile, g.words, lane, d);
        drop_tile<T>(p.drop, key, (uint32_t)row, (uint32_t)(col + j * kTile) / 8, lane, d);
      }
      store_tile<T, VEC>(tile + j * kTile, dx + j * kTile, left - j * kTile, g.words, lane, d);
    }
    dx += step * p.lddx;
    if constexpr (FUSED) dres += step * p.lddres;
    t = t + stage_len == ring_end ? ring : t + stage_len;
  }

  // the teams' sums, through the ring's memory
  float *out = p.partials + (int64_t)blockIdx.x * 2 * p.N;
  const int width = g.warps * CH * kTile;
  if (g.teams > 1) {
    cp_async_wait(0);
    __syncthreads();
    float *sums = reinterpret_cast<float *>(smem) + (size_t)2 * team * width + col;
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = j * kTile + pair_col<T>(lane, i);
        *reinterpret_cast<uint64_t *>(sums + c) = dw[j][i];
        *reinterpret_cast<uint64_t *>(sums + width + c) = db[j][i];
      }
    __syncthreads();
    sums = reinterpret_cast<float *>(smem);
    for (int c = threadIdx.x; c < (int)p.N; c += blockDim.x) {
      float a = 0.0f, d = 0.0f;
      for (int k = 0; k < g.teams; ++k) {
        a += sums[2 * k * width + c];
        d += sums[(2 * k + 1) * width + c];
      }
      out[c] = a;
      out[p.N + c] = d;
    }
  } else {
#pragma unroll
    for (int j = 0; j < CH; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int c = j * kTile + pair_col<T>(lane, i / 2) + (i & 1);
        if (c < left) {
          out[col + c] = (i & 1) ? f2_hi(dw[j][i / 2]) : f2_lo(dw[j][i / 2]);
          out[p.N + col + c] = (i & 1) ? f2_hi(db[j][i / 2]) : f2_lo(db[j][i / 2]);
        }
      }
  }
}

constexpr int kSms = 148;
constexpr size_t kMaxSmem = 227 * 1024 - 1024;  // the static arrays' share left out

// Chunks per thread, warps per row, rows per CTA and stages for rows of N
// values whose stage takes `arrays` x N values of `size` bytes, at most
// `threads` threads a CTA; 0 chunks: the row does not fit.
struct Choice {
  int ch = 0;
  Layout g = {};
  size_t smem = 0;
};
Choice choose_layout(int64_t T, int64_t N, int arrays, int size, int head, int threads, size_t budget,
                     int vec_bytes, bool sums) {
  Choice c;
  if (N > 16384) return c;
  const int chunks = (int)((N + 7) / 8);
  c.ch = chunks <= 32 ? 1 : chunks <= 1024 ? 2 : 4;
  c.g.warps = (chunks + 32 * c.ch - 1) / (32 * c.ch);
  c.g.teams = threads / 32 / c.g.warps;
  if (c.g.teams > 8) c.g.teams = 8;
  if (c.g.teams < 1) c.g.teams = 1;
  // few rows: one team per SM first
  while (c.g.teams > 1 && T <= (int64_t)kSms * (c.g.teams - 1)) --c.g.teams;
  const int warps = c.g.warps * c.g.teams;
  const size_t stage = (size_t)warps * ((size_t)arrays * c.ch * kTile * size + head);
  const size_t least = sums && c.g.teams > 1 ? (size_t)warps * c.ch * kTile * 8 : 0;
  const size_t vecs = (size_t)c.g.warps * c.ch * kTile * vec_bytes;
  if (vecs + stage > kMaxSmem) {
    c.ch = 0;
    return c;
  }
  c.g.stages = budget > vecs + stage ? (int)((budget - vecs) / stage) : 1;
  if (c.g.stages > kMaxStages) c.g.stages = kMaxStages;
  c.smem = c.g.stages * stage + vecs;
  if (c.smem < least) c.smem = least;
  return c;
}

template <typename K, typename P>
cudaError_t launch_rows(K kern, const P &p, const Choice &c, int ctas_per_sm, cudaStream_t st) {
  if (c.smem > 40 * 1024) {  // static shared memory counts towards the default 48 KB too
    const cudaError_t e =
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)c.smem);
    if (e != cudaSuccess) return e;
  }
  const int64_t need = (p.T + c.g.teams - 1) / c.g.teams, most = (int64_t)kSms * ctas_per_sm;
  return launch_pdl(kern, dim3((unsigned)(need < most ? need : most)),
                    dim3(32 * c.g.warps * c.g.teams), c.smem, st, p, c.g);
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

unsigned row_ctas(int64_t T) { return (unsigned)(T < kSms * 4 ? T : kSms * 4); }
// row groups of the wide dw pass, so that its CTAs fill the GPU twice over
int wide_splits(int64_t T, int64_t N) {
  const int64_t strips = (N + 255) / 256, groups = (T + 7) / 8;
  int64_t s = (kSms * 8 + strips - 1) / strips;
  s = s < groups ? s : groups;
  return (int)(s < 1 ? 1 : s > kMaxNormPartials ? kMaxNormPartials : s);
}
inline bool word_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 3u) == 0 && ld % 2 == 0;
}

template <typename T, typename W, bool VEC, bool FUSED>
cudaError_t fwd(const FwdParams &p, bool words, cudaStream_t st) {
  if (p.N > 16384)
    return launch_pdl(norm_fwd_wide_kernel<T, VEC, FUSED>, dim3(row_ctas(p.T)), dim3(kWideThreads), 0, st, p);
  const int chunks = (int)((p.N + 7) / 8);
  Choice c;
  const int most = VEC && !FUSED ? 8 : 4;
  c.ch = 1;
  while (c.ch < most && 32 * c.ch < chunks) c.ch *= 2;
  while ((chunks + 32 * c.ch - 1) / (32 * c.ch) * 32 > fwd_threads(c.ch)) c.ch *= 2;
  c.g.warps = (chunks + 32 * c.ch - 1) / (32 * c.ch);
  c.g.teams = fwd_threads(c.ch) / 32 / c.g.warps;
  if (c.g.warps > 1 && c.g.teams > 15) c.g.teams = 15;  // named barriers
  c.g.words = words;
  c.g.wvec = vec_ok(p.w, 8) && vec_ok(p.b, 8);
  const size_t vecs = (size_t)2 * c.g.warps * c.ch * kTile * sizeof(W);
  size_t stage;
  for (;; --c.g.teams) {
    stage = (size_t)c.g.warps * c.g.teams * (FUSED ? 2 : 1) * c.ch * kTile * sizeof(T);
    if (vecs + 3 * stage <= kMaxSmem || c.g.teams == 1) break;
  }
  while (c.g.teams > 1 && p.T <= (int64_t)kSms * (c.g.teams - 1)) --c.g.teams;
  stage = (size_t)c.g.warps * c.g.teams * (FUSED ? 2 : 1) * c.ch * kTile * sizeof(T);
  c.g.stages = (int)((kMaxSmem - vecs) / stage);
  if (c.g.stages > kMaxStages) c.g.stages = kMaxStages;
  if (c.g.stages < 1)
    return launch_pdl(norm_fwd_wide_kernel<T, VEC, FUSED>, dim3(row_ctas(p.T)), dim3(kWideThreads), 0, st, p);
  c.smem = c.g.stages * stage + vecs;
  switch (c.ch) {
    case 1: return launch_rows(norm_fwd_kernel<T, W, 1, VEC, FUSED>, p, c, 1, st);
    case 2: return launch_rows(norm_fwd_kernel<T, W, 2, VEC, FUSED>, p, c, 1, st);
    case 4: return launch_rows(norm_fwd_kernel<T, W, 4, VEC, FUSED>, p, c, 1, st);
    case 8: if constexpr (VEC) return launch_rows(norm_fwd_kernel<T, W, 8, VEC, FUSED>, p, c, 1, st);
    case 16: if constexpr (VEC) return launch_rows(norm_fwd_kernel<T, W, 16, VEC, FUSED>, p, c, 1, st);
  }
  return cudaErrorInvalidValue;
}
// Partial sums of dw and db; *n of them.
template <typename T, typename W, bool VEC, bool FUSED>
cudaError_t bwd(const BwdParams &p, bool words, int *n, cudaStream_t st) {
  Choice c = choose_layout(p.T, p.N, p.ds ? 3 : 2, (int)sizeof(T), 16, 512, kMaxSmem, (int)sizeof(W), true);
  c.g.words = words;
  c.g.wvec = vec_ok(p.w, 8);
  if (c.ch) {
    const int64_t need = (p.T + c.g.teams - 1) / c.g.teams;
    *n = (int)(need < kSms ? need : kSms);
  }
  switch (c.ch) {
    case 1: return launch_rows(norm_bwd_kernel<T, W, 1, VEC, FUSED>, p, c, 1, st);
    case 2: return launch_rows(norm_bwd_kernel<T, W, 2, VEC, FUSED>, p, c, 1, st);
    case 4: return launch_rows(norm_bwd_kernel<T, W, 4, VEC, FUSED>, p, c, 1, st);
  }
  *n = wide_splits(p.T, p.N);
  // dw first: dx may take the place of dy or x
  const cudaError_t e = launch_pdl(norm_dw_wide_kernel<T, VEC>, dim3((unsigned)((p.N + 255) / 256), (unsigned)*n),
                                   dim3(256), 0, st, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_dx_wide_kernel<T, VEC, FUSED>, dim3(row_ctas(p.T)), dim3(kWideThreads), 0, st, p);
}

}  // namespace

int norm_partials_count(int64_t T, int64_t N) {
  const int w = wide_splits(T, N);
  return w > kSms ? w : kSms;
}

cudaError_t launch_norm_fwd(const NormFwdArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.y, a.ldy) &&
                   (!a.fused || (vec_ok(a.res, a.ldres) && vec_ok(a.s, a.lds)));
  const bool words = word_ok(a.x, a.ldx) && word_ok(a.y, a.ldy) &&
                     (!a.fused || (word_ok(a.res, a.ldres) && word_ok(a.s, a.lds)));
  const FwdParams p = {a.x, a.res, a.ldx, a.ldres, a.T,   a.N,    a.w,    a.b, a.w_f32, a.center,
                       a.eps, a.y, a.s,   a.ldy,   a.lds, a.mean, a.rstd, make_drop(a.drop)};
  return by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return a.w_f32 ? (a.fused ? (vec ? fwd<T, float, true, true>(p, words, st) : fwd<T, float, false, true>(p, words, st))
                   : (vec ? fwd<T, float, true, false>(p, words, st) : fwd<T, float, false, false>(p, words, st))) : 
       (a.fused ? (vec ? fwd<T, T, true, true>(p, words, st) : fwd<T, T, false, true>(p, words, st))
                   : (vec ? fwd<T, T, true, false>(p, words, st) : fwd<T, T, false, false>(p, words, st)));
  });
}

cudaError_t launch_norm_bwd(const NormBwdArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.dy, a.lddy) && vec_ok(a.x, a.ldx) &&
                   vec_ok(a.dx, a.lddx) && (!a.ds || vec_ok(a.ds, a.ldds)) &&
                   (!a.fused || vec_ok(a.dres, a.lddres));
  const bool words = word_ok(a.dy, a.lddy) && word_ok(a.x, a.ldx) && word_ok(a.dx, a.lddx) &&
                     (!a.ds || word_ok(a.ds, a.ldds)) && (!a.fused || word_ok(a.dres, a.lddres));
  const BwdParams p = {a.dy, a.x, a.ds, a.lddy, a.ldx, a.ldds, a.T, a.N, a.w, a.w_f32, a.center,
                       a.mean, a.rstd, a.dx, a.dres, a.lddx, a.lddres, a.partials,
                       make_drop(a.drop)};
  int n = 0;
  const cudaError_t e = by_type(a.dtype, [&](auto t) {
    using T = decltype(t);
    return a.w_f32 ? (a.fused ? (vec ? bwd<T, float, true, true>(p, words, &n, st) : bwd<T, float, false, true>(p, words, &n, st))
                   : (vec ? bwd<T, float, true, false>(p, words, &n, st) : bwd<T, float, false, false>(p, words, &n, st))) :
      (a.fused ? (vec ? bwd<T, T, true, true>(p, words, &n, st) : bwd<T, T, false, true>(p, words, &n, st))
                   : (vec ? bwd<T, T, true, false>(p, words, &n, st) : bwd<T, T, false, false>(p, words, &n, st)));
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(norm_colsum_kernel, dim3((unsigned)((a.N + 31) / 32), a.db ? 2u : 1u),
                    dim3(kSumThreads), 0, st, a.partials, n, a.N, a.dw, a.db);
}

}  // namespace fa4
