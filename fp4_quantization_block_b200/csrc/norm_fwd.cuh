// norm_fwd.cuh -- layer norm forward, alone or fused (norm.cuh).
#pragma once

#include "norm.cuh"

namespace fa4 {
namespace norm {

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
  int64_t step_x, step_res, step_y, step_s;  // elements between a team's rows
};

// Rows too long for the chip: one CTA per row, the row read again for each
// pass, the weight and the bias by element.  2000 x 20000 fp32 takes 140 us,
// 2.3 TB/s of what a single pass moves (off 16-byte boundaries 264 us).
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

// Threads a CTA may have for the registers of CH chunks (128 each for 512
// threads, 80 for 768).
constexpr int fwd_threads(int ch, bool fused) { return ch <= 4 && !fused ? 768 : 512; }

// Each team takes every (gridDim.x * teams)-th row, CH chunks per thread; the
// weight and the bias lie in shared memory.  A warp finds the mean of its own
// columns and the squares about it; the team's are put together from the
// warps' with one barrier (Chan, Golub and LeVeque, "Updating formulae and a
// pairwise algorithm for computing sample variances", 1979): with n_w, m_w and
// q_w a warp's count, mean and squares, mean = sum n_w m_w / N and the row's
// squares are sum q_w + n_w (m_w - mean)^2.
//
// Bound by memory once enough rows are in flight and few enough instructions
// are spent on each: 8192 x 4096 bf16 takes 22.9 us, 5.85 TB/s (fused with
// dropout and the residual 47.5 us, 5.65 TB/s).  The same row in registers
// only, a team per row without a ring, took 45 us (latency); two chunks a
// thread 28 us, four 24 (the sums' instructions are per warp and row); a
// second barrier for the variance 1 us more.
template <typename T, typename W, int CH, bool VEC, bool FUSED>
__global__ void __launch_bounds__(fwd_threads(CH, FUSED), 1) norm_fwd_kernel(const FwdParams p, const Layout g) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float2 red[2][24];
  constexpr int A = FUSED ? 2 : 1, kLen = kTileLen<T, VEC>, kStage = A * CH * kLen;
  const int lane = threadIdx.x & 31, cta_warp = threadIdx.x >> 5;
  const int team = cta_warp / g.warps, warp = cta_warp - team * g.warps;
  const int col = warp * CH * kTile, left = (int)p.N - col;  // the warp's columns
  T *const ring = reinterpret_cast<T *>(smem) + (size_t)cta_warp * g.stages * kStage;
  const int ring_len = g.stages * kStage;
  const int room = g.warps * CH * kTile;
  W *const wsm = reinterpret_cast<W *>(smem + (size_t)g.warps * g.teams * g.stages * kStage * sizeof(T));
  W *const bsm = wsm + room;
  float2 *red0 = &red[0][team * g.warps], *red1 = &red[1][team * g.warps];
  const uint32_t q = blockIdx.x * g.teams + team;
  const int n = g.rows(q);
  if constexpr (VEC) {  // (tiles past the row's end too: they are read)
#pragma unroll
    for (int j = 0; j < CH; ++j)
      if (left - j * kTile < kTile)
        for (int s = 0; s < A * g.stages; ++s)
          clear_tail(ring + (s * CH + j) * kLen, left - j * kTile, kLen, lane);
    __syncwarp();
  }
  grid_dependency_wait();
  grid_dependents_launch();
  stage_vec<T, W>(wsm, static_cast<const W *>(p.w), (int)p.N, room, g.wvec);
  stage_vec<T, W>(bsm, static_cast<const W *>(p.b), p.b ? (int)p.N : 0, room, g.wvec);

  const T *fx = static_cast<const T *>(p.x) + q * p.ldx + col;
  const T *fr = FUSED ? static_cast<const T *>(p.res) + q * p.ldres + col : nullptr;
  int ahead = n;  // rows not yet asked for
  int fs = 0;     // the stage that the next one goes to
  auto fill = [&]() {
    if (ahead > 0) {
      T *const ft = ring + fs;
      const bool head = !VEC && q == 0 && col == 0 && ahead == n;
#pragma unroll
      for (int j = 0; j < CH; ++j) {
        if (!VEC && left - j * kTile <= 0) break;
        fill_tile<T, VEC>(ft + j * kLen, fx + j * kTile, left - j * kTile, head && j == 0, lane);
        if constexpr (FUSED)
          fill_tile<T, VEC>(ft + (CH + j) * kLen, fr + j * kTile, left - j * kTile, head && j == 0, lane);
      }
      fx += p.step_x;
      if constexpr (FUSED) fr += p.step_res;
      --ahead;
    }
    fs = fs + kStage == ring_len ? 0 : fs + kStage;
    cp_async_commit();
  };
  for (int s = 0; s < g.stages - 1; ++s) fill();
  const uint64_t key = FUSED ? p.drop.key() : 0ull;
  const float inv_n = 1.0f / (float)p.N;
  const float own_n = (float)(left < CH * kTile ? left : CH * kTile), inv_own = 1.0f / own_n;
  // of the warp whose sums this lane puts together
  const int peer = lane & (g.warps > 8 ? 15 : g.warps > 4 ? 7 : g.warps > 2 ? 3 : 1);
  const int peer_left = (int)p.N - peer * CH * kTile;
  const float peer_n = (float)(peer_left < 0 ? 0 : peer_left < CH * kTile ? peer_left : CH * kTile);
  T *y = static_cast<T *>(p.y) + q * p.ldy + col;
  T *sp = FUSED ? static_cast<T *>(p.s) + q * p.lds + col : nullptr;
  if (g.stages == 1) cp_async_commit();
  cp_async_wait(g.stages > 1 ? g.stages - 2 : 0);  // the oldest group holds the weights
  __syncthreads();

  int ts = 0;
  uint32_t row = q;
  for (int k = 0; k < n; ++k) {
    __syncwarp();  // the stage filled next was read by the whole warp
    fill();
    cp_async_wait(g.stages - 1);
    __syncwarp();
    T *const t = ring + ts;
    const int mx = VEC ? 0 : misaligned(static_cast<const T *>(p.x) + row * p.ldx);
    uint64_t v[CH][4], acc = 0ull;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      if (!VEC && left - j * kTile <= 0) {
        v[j][0] = v[j][1] = v[j][2] = v[j][3] = 0ull;
        continue;
      }
      read_tile<T, VEC>(t + j * kLen, mx, lane, v[j]);
      if constexpr (FUSED) {
        const int mr = VEC ? 0 : misaligned(static_cast<const T *>(p.res) + row * p.ldres);
        uint64_t r[4];
        drop_tile<T>(p.drop, key, row, (uint32_t)(col + j * kTile) / 8, lane, v[j]);
        read_tile<T, VEC>(t + (CH + j) * kLen, mr, lane, r);
        Raw8<T> raw;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = f2_add(v[j][i], r[i]);
        pack8(v[j], raw);
        unpack8(raw, v[j]);  // the stored s
      }
      acc = f2_add(acc, f2_add(f2_add(v[j][0], v[j][1]), f2_add(v[j][2], v[j][3])));
    }
    if constexpr (FUSED) store_tiles<T, CH, VEC>(t, sp, left, lane, v);
    float mean = p.center ? warp_sum(f2_sum(acc)) * inv_own : 0.0f;
    const uint64_t own = f2_set(-mean);
    acc = 0ull;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      // what lies past the row's end does not count
      uint64_t d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) d[i] = f2_add(v[j][i], own);
      if constexpr (VEC) {
        uint64_t lo = f2_fma(d[0], d[0], f2_mul(d[1], d[1])), hi = f2_fma(d[2], d[2], f2_mul(d[3], d[3]));
        if (j * kTile + pair_col<T>(lane, 0) >= left) lo = 0ull;
        if (j * kTile + pair_col<T>(lane, 2) >= left) hi = 0ull;
        acc = f2_add(acc, f2_add(lo, hi));
      } else if ((j + 1) * kTile <= left) {
#pragma unroll
        for (int i = 0; i < 4; ++i) acc = f2_fma(d[i], d[i], acc);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = j * kTile + pair_col<T>(lane, i);
          d[i] = f2_pack(c < left ? f2_lo(d[i]) : 0.0f, c + 1 < left ? f2_hi(d[i]) : 0.0f);
          acc = f2_fma(d[i], d[i], acc);
        }
      }
    }
    float m2 = warp_sum(f2_sum(acc));
    if (g.warps > 1) {
      if (lane == 0) red0[warp] = make_float2(mean, m2);
      asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * g.warps) : "memory");
      const float2 q = peer < g.warps ? red0[peer] : make_float2(0.0f, 0.0f);
      mean = peer_n * q.x;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        if (o < g.warps) mean += __shfl_xor_sync(0xFFFFFFFFu, mean, o);
      mean *= inv_n;
      const float d = q.x - mean;
      m2 = fmaf(peer_n * d, d, q.y);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1)
        if (o < g.warps) m2 += __shfl_xor_sync(0xFFFFFFFFu, m2, o);
      float2 *const next = red0;  // the row after the next one's
      red0 = red1;
      red1 = next;
    }
    const float rstd = rsqrtf(m2 * inv_n + p.eps);
    if (warp == 0 && lane == 0) {
      if (p.center) p.mean[row] = mean;
      p.rstd[row] = rstd;
    }
    const uint64_t scale = f2_set(rstd), shift = f2_set(-mean);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      uint64_t w[4], b[4];
      read_vec<T, W>(wsm + col + j * kTile, lane, w);
      read_vec<T, W>(bsm + col + j * kTile, lane, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] = f2_fma(f2_mul(f2_add(v[j][i], shift), scale), w[i], b[i]);
    }
    store_tiles<T, CH, VEC>(t, y, left, lane, v);
    y += p.step_y;
    if constexpr (FUSED) sp += p.step_s;
    row += g.step;
    ts = ts + kStage == ring_len ? 0 : ts + kStage;
  }
}

template <typename T, typename W, bool VEC, bool FUSED>
cudaError_t launch_fwd(FwdParams p, cudaStream_t st) {
  const int chunks = ceil_div(p.N < 32768 ? p.N : 32768, 8);
  // Eight chunks a thread save instructions per row (8192 x 4096: 22.9 us
  // against 25.5 with four).  With dropout they need registers that the
  // generator's work has use for (46.7 us with four against 49.6), and off
  // 16-byte boundaries for the shifted words (4096 x 4099: 26.9 against 30.9).
  const int most = VEC && !FUSED ? 8 : 4;
  int ch = 1;
  while (ch < most && 32 * ch < chunks) ch *= 2;
  while (ceil_div(chunks, 32 * ch) > 16 && ch < 8) ch *= 2;
  Layout g = {};
  g.cluster = 1;
  g.wvec = vec_ok(p.w, 8) && vec_ok(p.b, 8);
  g.warps = ceil_div(chunks, 32 * ch);
  const size_t vecs = (size_t)2 * g.warps * ch * kTile * sizeof(W);
  const size_t team = (size_t)g.warps * (FUSED ? 2 : 1) * ch * kTileLen<T, VEC> * sizeof(T);
  // from 18433 columns of fp32 on, 22529 of 16-bit rows with fp32 weights, 32769
  // with 16-bit ones; fused, 14337 (unaligned 13313), 18433 and 28673 (26625)
  if (p.N > 32768 || vecs + team > kMaxSmem)
    return launch_pdl(norm_fwd_wide_kernel<T, VEC, FUSED>, dim3(row_ctas(p.T)), dim3(kWideThreads), 0, st, p);
  g.teams = fwd_threads(ch, FUSED) / 32 / g.warps;
  if (g.warps > 1 && g.teams > 15) g.teams = 15;  // named barriers
  // at least three stages (binary32 4096 x 4096: 23.6 us against 31.5 with
  // two and more teams); few rows are spread over the SMs first
  while (g.teams > 1 && (vecs + 3 * g.teams * team > kMaxSmem || p.T <= (int64_t)kSms * (g.teams - 1))) --g.teams;
  g.stages = (int)((kMaxSmem - vecs) / (g.teams * team));
  if (g.stages > kMaxStages) g.stages = kMaxStages;
  const size_t smem = vecs + g.stages * g.teams * team;
  const int64_t need = (p.T + g.teams - 1) / g.teams;
  const int ctas = need < kSms ? (int)need : kSms;
  g.share(p.T, (int64_t)ctas * g.teams);
  p.step_x = g.step * p.ldx;
  p.step_res = g.step * p.ldres;
  p.step_y = g.step * p.ldy;
  p.step_s = g.step * p.lds;
  switch (ch) {
    case 1: return launch_rows(norm_fwd_kernel<T, W, 1, VEC, FUSED>, p, g, smem, ctas, st);
    case 2: return launch_rows(norm_fwd_kernel<T, W, 2, VEC, FUSED>, p, g, smem, ctas, st);
    case 4: return launch_rows(norm_fwd_kernel<T, W, 4, VEC, FUSED>, p, g, smem, ctas, st);
  }
  return launch_rows(norm_fwd_kernel<T, W, 8, VEC, FUSED>, p, g, smem, ctas, st);
}
template <typename T, typename W>
cudaError_t forward_w(const NormFwdArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.y, a.ldy) &&
                   (!a.fused || (vec_ok(a.res, a.ldres) && vec_ok(a.s, a.lds)));
  FwdParams p = {};
  p.x = a.x;
  p.res = a.res;
  p.ldx = a.ldx;
  p.ldres = a.ldres;
  p.T = a.T;
  p.N = a.N;
  p.w = a.w;
  p.b = a.b;
  p.w_f32 = a.w_f32;
  p.center = a.center;
  p.eps = a.eps;
  p.y = a.y;
  p.s = a.s;
  p.ldy = a.ldy;
  p.lds = a.lds;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.drop = make_drop(a.drop);
  if (a.fused) return vec ? launch_fwd<T, W, true, true>(p, st) : launch_fwd<T, W, false, true>(p, st);
  return vec ? launch_fwd<T, W, true, false>(p, st) : launch_fwd<T, W, false, false>(p, st);
}
template <typename T>
cudaError_t forward(const NormFwdArgs &a, cudaStream_t st) {
  if constexpr (sizeof(T) == 2)
    if (!a.w_f32) return forward_w<T, T>(a, st);
  return forward_w<T, float>(a, st);
}

}  // namespace norm
}  // namespace fa4
