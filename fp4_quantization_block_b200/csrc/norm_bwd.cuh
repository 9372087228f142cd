// norm_bwd.cuh -- layer norm backward, alone or fused (norm.cuh).
#pragma once

#include "norm.cuh"

namespace fa4 {
namespace norm {

struct BwdParams {
  const void *dy, *x, *ds;
  int64_t lddy, ldx, ldds, T, N;
  const void *w;
  int w_f32, center;
  const float *mean, *rstd;
  void *dx, *dres;
  int64_t lddx, lddres;
  float *partials;  // [cluster][2][N]
  float *dw, *db;   // where there is one cluster only
  uint32_t *status;  // set when a wait within a cluster gives up
  uint64_t timeout_ns;  // the limit of such a wait
  uint32_t withheld;    // a row whose sums a cluster's first CTA does not send; no row is ~0
  int one;
  Drop drop;
  int64_t step_x, step_dy, step_ds, step_dx, step_dres;  // elements between a team's rows
};

// Rows too long for the chip: dx of one row per CTA.
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

// The columns col .. end - 1 of dx (and dres) of n of a warp's rows, all NaN.
// Out of line: inside the kernel its loops cost registers of the loop over the
// rows (fused 2000 x 24576 bf16: 180 us against 133).
template <typename T, bool FUSED>
__device__ __noinline__ void leave_nan(void *dx, int64_t lddx, void *dres, int64_t lddres, int64_t row,
                                       uint32_t step, int n, int col, int end) {
  const T nan = from_float<T>(__int_as_float(0x7FC00000));
  for (; n > 0; --n, row += step)
    for (int c = col + (threadIdx.x & 31); c < end; c += 32) {
      static_cast<T *>(dx)[row * lddx + c] = nan;
      if constexpr (FUSED) static_cast<T *>(dres)[row * lddres + c] = nan;
    }
}

// dx of a team's rows; dw and db of its columns stay in registers over its
// rows, are added up over the CTA's teams in order and go to the CTA's partial
// sums.  A row takes two passes over its columns, with mean(g) and mean(g xh)
// of the whole row between them; xh and g stay in registers.  CLUSTER: rows
// too wide for a CTA are shared by a cluster of CTAs, each with some of the
// columns (and fewer partial sums to write): every warp sends its part of the
// two sums to all of them, and each team waits at a barrier of its own for the
// parts of its row, not for another team or for a fence over its stores.  Two
// barriers and two buffers take turns: a part of the row after the next one is
// sent only when all parts of the next one have come, and a warp sends its own
// only after it has read this row's.  A wait that gives up ends its
// warp's rows: the status word is set, and what the warp leaves undone is NaN,
// its columns of dx (and dres) from that row on, and of dw and db.
//
// 8192 x 4096 bf16 with ds takes 47.8 us (5.6 TB/s; 65536 rows 7.0 TB/s):
// nearly 10 us are a launch's own, the first row's latency, the last row's,
// the sums at the end and the second launch.  Fused with dropout 68.8 us:
// half of all issue slots are used, by 16 warps of 128 registers (the sums of
// dw and db are 32 of them).  Wide rows: 1000 x 14336 fp16 34.9 us, 2.5 TB/s;
// 2000 x 24576 bf16 90 us (115 with a barrier of the whole cluster at each
// row, which also waits for the stores of dx).  Tried and slower: clusters of
// two for rows that fit a CTA (50 us at 4096 x 8192 against 45), the second
// pass computing xh and g again (67 us at 8192 x 4096), four chunks a thread
// (53 us at 4096 x 8192), the dropout's bits before the data (fused 85 us).
template <typename T, typename W, int CH, bool VEC, bool FUSED, bool DS, bool CLUSTER>
__global__ void __launch_bounds__(32 * kBwdWarps, 1) norm_bwd_kernel(const BwdParams p, const Layout g) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int kParts = CLUSTER ? 8 * kBwdWarps : kBwdWarps;
  __shared__ float2 red[2][kParts];  // [row buffer][team][CTA][warp]
  __shared__ uint64_t arrived[2][CLUSTER ? kBwdWarps : 1];  // [row buffer][team]
  constexpr int A = DS ? 3 : 2, kLen = kTileLen<T, VEC>, kStage = A * CH * kLen;
  const int lane = threadIdx.x & 31, cta_warp = threadIdx.x >> 5;
  const int team = cta_warp / g.warps, warp = cta_warp - team * g.warps;
  const int rank = CLUSTER ? blockIdx.x % g.cluster : 0, cid = CLUSTER ? blockIdx.x / g.cluster : blockIdx.x;
  const int room = g.warps * CH * kTile;  // the CTA's share of a row
  const int col = rank * room + warp * CH * kTile, left = (int)p.N - col;  // the warp's columns
  T *const ring = reinterpret_cast<T *>(smem) + (size_t)cta_warp * g.stages * kStage;
  const int ring_len = g.stages * kStage;
  W *const wsm = reinterpret_cast<W *>(smem + (size_t)g.warps * g.teams * g.stages * kStage * sizeof(T));
  const uint32_t q = cid * g.teams + team;
  const int n = g.rows(q);
  if constexpr (VEC) {  // (tiles past the row's end too: they are read)
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (left - j * kTile < kTile)
        for (int s = 0; s < A * g.stages; ++s)
          clear_tail(ring + (s * CH + j) * kLen, left - j * kTile, kLen, lane);
    __syncwarp();
  }
  if constexpr (CLUSTER) {  // all CTAs and their barriers are there before anything is sent to them
    if (threadIdx.x < 2 * kBwdWarps) barrier_init(&arrived[0][0] + threadIdx.x);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncwarp();
    cluster_sync();
  }
  grid_dependency_wait();
  grid_dependents_launch();
  const int cols = (int)p.N - rank * room;
  stage_vec<T, W>(wsm, static_cast<const W *>(p.w) + rank * room, cols < 0 ? 0 : cols < room ? cols : room, room,
                  g.wvec);

  const T *fx = static_cast<const T *>(p.x) + q * p.ldx + col;
  const T *fdy = static_cast<const T *>(p.dy) + q * p.lddy + col;
  const T *fds = DS ? static_cast<const T *>(p.ds) + q * p.ldds + col : nullptr;
  int ahead = n;  // rows not yet asked for
  int fs = 0;     // the stage that the next one goes to
  auto fill = [&]() {
    if (ahead > 0) {
      T *const t = ring + fs;
      const bool head = !VEC && q == 0 && col == 0 && ahead == n;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!VEC && left - j * kTile <= 0) break;
        const bool h = head && j == 0;
        fill_tile<T, VEC>(t + j * kLen, fx + j * kTile, left - j * kTile, h, lane);
        fill_tile<T, VEC>(t + (CH + j) * kLen, fdy + j * kTile, left - j * kTile, h, lane);
        if constexpr (DS) fill_tile<T, VEC>(t + (2 * CH + j) * kLen, fds + j * kTile, left - j * kTile, h, lane);
      }
      fx += p.step_x;
      fdy += p.step_dy;
      if constexpr (DS) fds += p.step_ds;
      --ahead;
    }
    fs = fs + kStage == ring_len ? 0 : fs + kStage;
    cp_async_commit();
  };
  for (int s = 0; s < g.stages - 1; ++s) fill();

  // the next row's statistics, a row ahead
  const float *mean_p = p.center ? p.mean + q : nullptr, *rstd_p = p.rstd + q;
  float mean_next = 0.0f, rstd_next = 0.0f;
  if (n > 0) {
    if (mean_p) mean_next = *mean_p;
    rstd_next = *rstd_p;
  }
  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  uint64_t w[CH][4], dw[CH][4], db[CH][4];
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = 0ull;
  const float inv_n = 1.0f / (float)p.N;
  T *dx = static_cast<T *>(p.dx) + q * p.lddx + col;
  T *dres = FUSED ? static_cast<T *>(p.dres) + q * p.lddres + col : nullptr;

  const int parts = CLUSTER ? g.cluster * g.warps : g.warps;  // of a row's sums
  if (g.stages == 1) cp_async_commit();            // no row has been asked for: the weight's copies alone
  cp_async_wait(g.stages > 1 ? g.stages - 2 : 0);  // the oldest group holds the weight
  __syncthreads();
#pragma unroll
  for (int j = 0; j < CH; ++j) read_vec<T, W>(wsm + warp * CH * kTile + j * kTile, lane, w[j]);
  float2 *red0 = &red[0][team * parts], *red1 = &red[1][team * parts];
  const bool upper = lane >= 16;  // the lanes that add up the second sum
  int ts = 0, stop = n;  // the row whose wait gave up
  uint32_t row = q;
  for (int k = 0; k < n; ++k) {
    __syncwarp();  // the stage filled next was read by the whole warp
    fill();
    const float rstd = rstd_next, mean = mean_next;
    if (k + 1 < n) {
      rstd_p += g.step;
      rstd_next = *rstd_p;
      if (mean_p) {
        mean_p += g.step;
        mean_next = *mean_p;
      }
    }
    cp_async_wait(g.stages - 1);
    __syncwarp();
    T *const t = ring + ts;
    const uint64_t scale = f2_set(rstd);
    uint64_t xh[CH][4], gg[CH][4], s1 = 0ull, s2 = 0ull;
    {
      const uint64_t shift = f2_set(-mean);
      const int mx = VEC ? 0 : misaligned(static_cast<const T *>(p.x) + row * p.ldx);
      const int md = VEC ? 0 : misaligned(static_cast<const T *>(p.dy) + row * p.lddy);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        uint64_t dy[4];
        if (!VEC && left - j * kTile <= 0) {  // past the row's end
#pragma unroll
          for (int i = 0; i < 4; ++i) xh[j][i] = gg[j][i] = 0ull;
          continue;
        }
        read_tile<T, VEC>(t + j * kLen, mx, lane, xh[j]);
        read_tile<T, VEC>(t + (CH + j) * kLen, md, lane, dy);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          xh[j][i] = f2_mul(f2_add(xh[j][i], shift), scale);
          gg[j][i] = f2_mul(dy[i], w[j][i]);
          dw[j][i] = f2_fma(dy[i], xh[j][i], dw[j][i]);
          db[j][i] = f2_add(db[j][i], dy[i]);
          s1 = f2_add(s1, gg[j][i]);
          s2 = f2_fma(gg[j][i], xh[j][i], s2);
        }
      }
    }
    // both sums in one butterfly: the lower lanes take the first, the upper
    // ones the second
    float v = f2_sum(s1), u = f2_sum(s2);
    {
      const float keep = upper ? u : v;
      v = keep + __shfl_xor_sync(0xFFFFFFFFu, upper ? v : u, 16);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    }
    if (parts > 1) {
      const int l = lane & 15;
      if constexpr (CLUSTER) {
        uint64_t *const barrier = &arrived[k & 1][team];
        const float2 both = make_float2(__shfl_sync(0xFFFFFFFFu, v, 0), __shfl_sync(0xFFFFFFFFu, v, 16));
        if (warp == 0 && lane == 0) barrier_expect(barrier, 8 * parts);
        if (lane < g.cluster && !(row == p.withheld && rank == 0))
          cluster_send(&red0[rank * g.warps + warp], barrier, lane, both);
        // (a wait ends by itself; what a lane saw decides for the warp)
        if (!__all_sync(0xFFFFFFFFu, barrier_wait(barrier, (k >> 1) & 1, p.timeout_ns))) {
          stop = k;
          break;
        }
        v = 0.0f;
        for (int i = l; i < parts; i += 16) v += upper ? red0[i].y : red0[i].x;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      } else {
        if (l == 0) reinterpret_cast<float *>(red0 + warp)[upper] = v;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * g.warps) : "memory");
        const int peer = l & (parts > 8 ? 15 : parts > 4 ? 7 : parts > 2 ? 3 : 1);
        v = peer < parts ? reinterpret_cast<const float *>(red0 + peer)[upper] : 0.0f;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1)
          if (o < parts) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
      }
      float2 *const next = red0;  // the row after the next one's
      red0 = red1;
      red1 = next;
    }
    v *= -inv_n;
    const float m1 = __shfl_sync(0xFFFFFFFFu, v, 0), m2 = __shfl_sync(0xFFFFFFFFu, v, 16);
    {
      const uint64_t c1 = f2_set(p.center ? m1 : 0.0f), c2 = f2_set(m2);
#pragma unroll
      for (int j = 0; j < CH; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) gg[j][i] = f2_fma(xh[j][i], c2, f2_add(gg[j][i], c1));
        if constexpr (DS) {
          uint64_t r[4] = {};
          const int mr = VEC ? 0 : misaligned(static_cast<const T *>(p.ds) + row * p.ldds);
          if (VEC || left - j * kTile > 0) read_tile<T, VEC>(t + (2 * CH + j) * kLen, mr, lane, r);
#pragma unroll
          for (int i = 0; i < 4; ++i) gg[j][i] = f2_fma(gg[j][i], scale, r[i]);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) gg[j][i] = f2_mul(gg[j][i], scale);
        }
      }
      if constexpr (FUSED) {
        store_tiles<T, CH, VEC>(t, dres, left, lane, gg);
#pragma unroll
        for (int j = 0; j < CH; ++j)
          drop_tile<T>(p.drop, key, row, (uint32_t)(col + j * kTile) / 8, lane, gg[j]);
      }
      store_tiles<T, CH, VEC>(t, dx, left, lane, gg);
      dx += p.step_dx;
      if constexpr (FUSED) dres += p.step_dres;
    }
    row += g.step;
    ts = ts + kStage == ring_len ? 0 : ts + kStage;
  }

  if constexpr (CLUSTER) {
    if (stop < n) {
      if (lane == 0) *p.status = 7u;
      leave_nan<T, FUSED>(p.dx, p.lddx, p.dres, p.lddres, row, g.step, n - stop, col,
                          (int)p.N - col < CH * kTile ? (int)p.N : col + CH * kTile);
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) dw[j][i] = db[j][i] = f2_set(__int_as_float(0x7FC00000));
    }
    // nobody leaves while something may still be sent to them, or (where a
    // wait gave up) may be on its way
    __syncwarp();
    cluster_sync();
    if (stop < n)
      for (const uint64_t begin = globaltimer(); globaltimer() - begin < 100000ull;) __nanosleep(1000);
    __syncwarp();
  }
  // the teams' sums, through the ring's memory, in the teams' order
  float *const out_w = p.one ? p.dw : p.partials + (int64_t)cid * 2 * p.N;
  float *const out_b = p.one ? p.db : out_w + p.N;
  cp_async_wait(0);
  __syncthreads();
  float *sums = reinterpret_cast<float *>(smem) + (size_t)2 * team * room + warp * CH * kTile;
#pragma unroll
  for (int j = 0; j < CH; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = j * kTile + pair_col<T>(lane, i);
      *reinterpret_cast<uint64_t *>(sums + c) = dw[j][i];
      *reinterpret_cast<uint64_t *>(sums + room + c) = db[j][i];
    }
  __syncthreads();
  sums = reinterpret_cast<float *>(smem);
  for (int c = threadIdx.x; c < room && c < cols; c += blockDim.x) {
    float a = 0.0f, d = 0.0f;
    for (int k = 0; k < g.teams; ++k) {
      a += sums[2 * k * room + c];
      d += sums[(2 * k + 1) * room + c];
    }
    out_w[rank * room + c] = a;
    if (out_b) out_b[rank * room + c] = d;
  }
}

// dx, and dw and db or *n partial sums of them (0: dw and db are done).
template <typename T, typename W, bool VEC, bool FUSED, bool DS>
cudaError_t launch_bwd(BwdParams p, int *n, cudaStream_t st) {
  const int ch = p.N <= 256 ? 1 : 2, warps = ceil_div(p.N < (1 << 17) ? p.N : (1 << 17), kTile * ch);
  Layout g = {};
  g.wvec = vec_ok(p.w, 8);
  // As few CTAs to a row as its columns need; but where a cluster of eight
  // takes all rows in two rounds, that one cluster, which needs no partial sums
  // and no second launch (8 x 4096 bf16: 3.3 us against 5.8; at four rounds
  // the second launch is cheaper: 64 x 4096 6.8 us against 9.7).
  int log = 0;
  while (log < 3 && ceil_div(warps, 1 << log) > kBwdWarps) ++log;
  const int eighth = ceil_div(warps, 8), at_once = eighth <= kBwdWarps ? kBwdWarps / eighth : 0;
  const bool few = ch == 2 && p.T <= 2 * at_once;
  if (few)
    while (log < 3 && (1 << log) < warps) ++log;
  g.cluster = 1 << log;
  g.warps = ceil_div(warps, g.cluster);
  const size_t vecs = (size_t)g.warps * ch * kTile * sizeof(W);
  // rows at a time as if ds were there, so that dw and db do not depend on it
  const size_t tile = (size_t)ch * kTileLen<T, VEC> * sizeof(T), most_team = 3 * g.warps * tile;
  const size_t team = (DS ? 3 : 2) * g.warps * tile;
  if (g.warps > kBwdWarps || vecs + most_team > kMaxSmem) {
    *n = wide_splits(p.T, p.N);
    // dw first: dx may take the place of dy or x
    const cudaError_t e = launch_pdl(norm_dw_wide_kernel<T, VEC>, dim3((unsigned)ceil_div(p.N, 256), (unsigned)*n),
                                     dim3(256), 0, st, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_dx_wide_kernel<T, VEC, FUSED>, dim3(row_ctas(p.T)), dim3(kWideThreads), 0, st, p);
  }
  const int most = few ? 1 : kMaxClusters[log];
  g.teams = kBwdWarps / g.warps;
  if (g.warps > 1 && g.teams > 15) g.teams = 15;  // named barriers
  while (g.teams > 1 && (vecs + 3 * g.teams * most_team > kMaxSmem || p.T <= (int64_t)most * (g.teams - 1)))
    --g.teams;
  g.stages = (int)((kMaxSmem - vecs) / (g.teams * team));
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  size_t smem = vecs + g.stages * g.teams * team;
  const size_t sums = (size_t)g.teams * g.warps * ch * kTile * 8;
  if (smem < sums) smem = sums;
  const int64_t need = (p.T + g.teams - 1) / g.teams;
  const int clusters = need < most ? (int)need : most;
  g.share(p.T, (int64_t)clusters * g.teams);
  p.step_x = g.step * p.ldx;
  p.step_dy = g.step * p.lddy;
  p.step_ds = g.step * p.ldds;
  p.step_dx = g.step * p.lddx;
  p.step_dres = g.step * p.lddres;
  p.one = clusters == 1;
  *n = p.one ? 0 : clusters;
  const int ctas = clusters * g.cluster;
  if (ch == 1) return launch_rows(norm_bwd_kernel<T, W, 1, VEC, FUSED, DS, false>, p, g, smem, ctas, st);
  if (g.cluster == 1) return launch_rows(norm_bwd_kernel<T, W, 2, VEC, FUSED, DS, false>, p, g, smem, ctas, st);
  return launch_rows(norm_bwd_kernel<T, W, 2, VEC, FUSED, DS, true>, p, g, smem, ctas, st);
}
template <typename T, typename W>
cudaError_t backward_w(const NormBwdArgs &a, int *n, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.dy, a.lddy) && vec_ok(a.x, a.ldx) && vec_ok(a.dx, a.lddx) &&
                   (!a.ds || vec_ok(a.ds, a.ldds)) && (!a.fused || vec_ok(a.dres, a.lddres));
  BwdParams p = {};
  p.dy = a.dy;
  p.x = a.x;
  p.ds = a.ds;
  p.lddy = a.lddy;
  p.ldx = a.ldx;
  p.ldds = a.ldds;
  p.T = a.T;
  p.N = a.N;
  p.w = a.w;
  p.w_f32 = a.w_f32;
  p.center = a.center;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.dx = a.dx;
  p.dres = a.dres;
  p.lddx = a.lddx;
  p.lddres = a.lddres;
  p.partials = a.partials;
  p.dw = a.dw;
  p.status = a.status;
  p.timeout_ns = a.timeout_ns;
  p.withheld = a.withheld < 0 ? ~0u : (uint32_t)a.withheld;
  p.db = a.db;
  p.drop = make_drop(a.drop);
  auto go = [&](auto v, auto f) {
    constexpr bool V = decltype(v)::value, F = decltype(f)::value;
    return a.ds ? launch_bwd<T, W, V, F, true>(p, n, st) : launch_bwd<T, W, V, F, false>(p, n, st);
  };
  using std::false_type;
  using std::true_type;
  if (a.fused) return vec ? go(true_type(), true_type()) : go(false_type(), true_type());
  return vec ? go(true_type(), false_type()) : go(false_type(), false_type());
}
template <typename T>
cudaError_t backward(const NormBwdArgs &a, int *n, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (!a.w_f32) return backward_w<T, T>(a, n, st);
  return backward_w<T, float>(a, n, st);
}

}  // namespace norm
}  // namespace fa4
