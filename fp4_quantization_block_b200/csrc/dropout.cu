// dropout.cu -- dropout from the counter-based generator, with or without the
// residual addition: y = [res +] (kept ? x * scale : 0), the mask computed
// from (key, row, column) where it is needed (rows.cuh) and never stored.
// The backward pass is the same map of dy under the same key.
//
// Two or three accesses of an element against some twenty instructions, most
// of them the generator's: with a residual bound by memory (16384 x 4096 bf16
// 61.2 us, 6.6 TB/s), without one as much by instructions (8192 x 4096 25.2
// us, 5.3 TB/s).  Each thread has all its loads in flight before it computes,
// and the grid covers the matrix once.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace {

using namespace rows;

constexpr int kThreads = 256;
// Rows of a thread where there are enough for every SM: 8192 x 4096 bf16 takes
// 30.0, 27.9 and 25.2 us with one, two and four.  Few rows are spread over the
// SMs instead.
constexpr int kRows = 4;
// Tiles of a warp of 16-bit rows off 16-byte boundaries: four rows, or two and
// their residuals (8192 x 4099 bf16 41.4 us, with one row 46.5, element by
// element 46.5; with residual 53.3).
constexpr int kTiles = 4;

struct DropoutParams {
  const void *x, *res;
  void *y;
  int64_t ldx, ldres, ldy, T, N;
  int64_t units;  // of the matrix: chunks of eight columns of a group of rows, or warps' tiles
  Divisor per_row;
  Drop drop;
};

// Row and unit in its row of the n-th unit of the CTA's, which start at
// `first` = (row0, unit0).
__device__ __forceinline__ void place(const DropoutParams &p, int64_t row0, uint32_t unit0, uint32_t n,
                                      int64_t &row, uint32_t &unit) {
  const uint32_t u = unit0 + n, q = p.per_row.quotient(u);
  row = row0 + q;
  unit = u - q * p.per_row.d;
}

// Rows on 16-byte boundaries, N a multiple of eight.  A thread takes the same
// chunk of ROWS consecutive rows (one division, one key schedule and the first
// half of the generator's first round for all of them); a unit is a chunk of
// such a group of rows.  Consecutive lanes have consecutive units; binary32
// lanes have the even or odd halves of two of them, so that their 16-byte
// accesses are consecutive.  y may be x or res itself: a thread reads its
// elements before it writes them.
template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const DropoutParams p) {
  constexpr int H = sizeof(T) / 2;  // 16-byte pieces of a lane in a row
  constexpr int kPer16 = 16 / (int)sizeof(T);
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const uint64_t key = p.drop.key();
  const int64_t first = (int64_t)blockIdx.x * kThreads;
  const int64_t group0 = p.units < (int64_t(1) << 31) ? p.per_row.quotient((uint32_t)first) : first / p.per_row.d;
  const uint32_t unit0 = (uint32_t)(first - group0 * p.per_row.d);
  const uint32_t warp0 = threadIdx.x & ~31u;
  int64_t row[H];
  uint32_t unit[H], c[H];
  bool in[H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const uint32_t k = H == 1 ? threadIdx.x : warp0 + 16 * h + (lane >> 1);
    place(p, group0, unit0, k, row[h], unit[h]);
    row[h] *= ROWS;
    c[h] = 8 * unit[h] + (H == 2 ? kPer16 * (lane & 1) : 0);
    in[h] = first + k < p.units;
  }
  uint4 x[ROWS][H], r[ROWS][H];
#pragma unroll
  for (int h = 0; h < H; ++h) {
    const T *px = static_cast<const T *>(p.x) + row[h] * p.ldx + c[h];
    const T *pr = static_cast<const T *>(p.res) + row[h] * p.ldres + c[h];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      if (in[h] && (ROWS == 1 || row[h] + k < p.T)) {
        x[k][h] = __ldcs(reinterpret_cast<const uint4 *>(px));
        if (p.res) r[k][h] = __ldcs(reinterpret_cast<const uint4 *>(pr));
      }
      px += p.ldx;
      pr += p.ldres;
    }
  }
  // the block whose bits this lane computes: its chunk, or (binary32) the
  // first or the second of the two that it shares with its neighbour
  const int mine = H == 1 ? 0 : lane & 1;
  const uint32_t block = mine ? unit[H - 1] : unit[0];
  const int64_t brow = mine ? row[H - 1] : row[0];
  T *py[H];
#pragma unroll
  for (int h = 0; h < H; ++h) py[h] = static_cast<T *>(p.y) + row[h] * p.ldy + c[h];
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    Raw8<T> raw;
    uint64_t f[4];
#pragma unroll
    for (int h = 0; h < H; ++h) raw.v[h] = x[k][h];
    unpack8(raw, f);
    if (p.drop.threshold) {
      const u32x4 b = philox(block, (uint32_t)brow + k, 0u, kDropTag, (uint32_t)key, (uint32_t)(key >> 32));
      uint32_t w[4] = {b.x, b.y, b.z, b.w};
      if constexpr (H == 2) share_bits(b, lane, w);
      drop_pairs(p.drop, w, f);
    }
    if (p.res) {
      uint64_t g[4];
#pragma unroll
      for (int h = 0; h < H; ++h) raw.v[h] = r[k][h];
      unpack8(raw, g);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = f2_add(f[i], g[i]);
    }
    pack8(f, raw);
#pragma unroll
    for (int h = 0; h < H; ++h) {
      if (in[h] && (ROWS == 1 || row[h] + k < p.T)) *reinterpret_cast<uint4 *>(py[h]) = raw.v[h];
      py[h] += p.ldy;
    }
  }
}

// 16-bit rows off 16-byte boundaries: a warp takes 256 columns of ROWS
// consecutive rows, by the aligned words that they lie in (rows.cuh), so that a
// lane has a whole block of the generator.  The words of all rows are on their
// way together; each row's bits are computed before its words are waited for.
template <typename T, int ROWS, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_shifted_kernel(const DropoutParams p) {
  static_assert(sizeof(T) == 2, "");
  __shared__ __align__(16) T tiles[kThreads / 32][ROWS][RES ? 2 : 1][kTileLen<T, false>];
  const int lane = threadIdx.x & 31;
  const uint32_t warp = threadIdx.x >> 5;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 32);
  const int64_t group0 = p.units < (int64_t(1) << 31) ? p.per_row.quotient((uint32_t)first) : first / p.per_row.d;
  if (first + warp >= p.units) return;
  int64_t row;
  uint32_t unit;
  place(p, group0, (uint32_t)(first - group0 * p.per_row.d), warp, row, unit);
  row *= ROWS;
  const int64_t col = (int64_t)unit * kTile;
  const int left = (int)(p.N - col), rows = p.T - row < ROWS ? (int)(p.T - row) : ROWS;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx + col;
  const T *res = static_cast<const T *>(p.res) + (RES ? row * p.ldres + col : 0);
  T *y = static_cast<T *>(p.y) + row * p.ldy + col;
  const bool head = row == 0 && col == 0;
#pragma unroll
  for (int k = 0; k < ROWS; ++k) {
    if (k < rows) {
      fill_tile<T, false>(tiles[warp][k][0], x + k * p.ldx, left, head && k == 0, lane);
      if constexpr (RES) fill_tile<T, false>(tiles[warp][k][RES], res + k * p.ldres, left, head && k == 0, lane);
    }
    cp_async_commit();
  }
  const uint64_t key = p.drop.key();
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if (k < rows) {
      uint32_t w[4];
      if (p.drop.threshold) {
        const u32x4 b = philox(unit * (kTile / 8) + lane, (uint32_t)row + k, 0u, kDropTag, (uint32_t)key,
                               (uint32_t)(key >> 32));
        w[0] = b.x, w[1] = b.y, w[2] = b.z, w[3] = b.w;
      }
      cp_async_wait(ROWS - 1 - k);
      __syncwarp();
      uint64_t f[1][4];
      read_tile<T, false>(tiles[warp][k][0], misaligned(x + k * p.ldx), lane, f[0]);
      if (p.drop.threshold) drop_pairs(p.drop, w, f[0]);
      if constexpr (RES) {
        uint64_t g[4];
        read_tile<T, false>(tiles[warp][k][RES], misaligned(res + k * p.ldres), lane, g);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[0][i] = f2_add(f[0][i], g[i]);
      }
      store_tiles<T, 1, false>(tiles[warp][k][0], y + k * p.ldy, left, lane, f);
    }
}

// Other binary32 rows: a warp takes 256 columns of a row, element by element in
// column order (lane l the columns l, 32 + l, ...), so that its accesses are
// consecutive; lane l computes the bits of block l of the tile, and each
// element takes its bit from the lane that has it.
template <typename T>
__global__ void __launch_bounds__(kThreads) dropout_elements_kernel(const DropoutParams p) {
  const int lane = threadIdx.x & 31;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = (int64_t)blockIdx.x * (kThreads / 32);
  const int64_t row0 = p.units < (int64_t(1) << 31) ? p.per_row.quotient((uint32_t)first) : first / p.per_row.d;
  const uint32_t warp = threadIdx.x >> 5;
  if (first + warp >= p.units) return;
  int64_t row;
  uint32_t unit;
  place(p, row0, (uint32_t)(first - row0 * p.per_row.d), warp, row, unit);
  const int64_t col = (int64_t)unit * kTile + lane;
  const T *x = static_cast<const T *>(p.x) + row * p.ldx + col;
  const T *res = static_cast<const T *>(p.res) + row * p.ldres + col;
  T *y = static_cast<T *>(p.y) + row * p.ldy + col;
  T v[8], r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (col + 32 * i < p.N) {
      v[i] = x[32 * i];
      if (p.res) r[i] = res[32 * i];
    }
  uint32_t bits = 0xFFu;  // which of the block's eight are kept
  if (p.drop.threshold) {
    const uint64_t key = p.drop.key();
    const u32x4 b = philox(unit * (kTile / 8) + lane, (uint32_t)row, 0u, kDropTag, (uint32_t)key,
                           (uint32_t)(key >> 32));
    const uint32_t w[4] = {b.x, b.y, b.z, b.w}, t = p.drop.threshold << 16;
    bits = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      bits |= ((w[i] << 16) >= t ? 1u << (2 * i) : 0u) | (w[i] >= t ? 2u << (2 * i) : 0u);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t block = __shfl_sync(0xFFFFFFFFu, bits, 4 * i + (lane >> 3));
    if (col + 32 * i < p.N) {
      float f = (block >> (lane & 7)) & 1u ? to_float(v[i]) * p.drop.scale : 0.0f;
      if (p.res) f += to_float(r[i]);
      y[32 * i] = from_float<T>(f);
    }
  }
}

inline bool vec_ok(const void *p, int64_t ld) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

template <typename T>
cudaError_t launch(const DropoutArgs &a, cudaStream_t st) {
  const bool vec = a.N % 8 == 0 && vec_ok(a.x, a.ldx) && vec_ok(a.y, a.ldy) &&
                   (!a.res || vec_ok(a.res, a.ldres));
  const int64_t per_row = vec ? a.N / 8 : (a.N + kTile - 1) / kTile;
  const int64_t per_cta = vec ? kThreads : kThreads / 32;
  const bool many = a.T * per_row > 148 * 8 * per_cta;
  // rows of a thread
  const int rows = !many || (!vec && sizeof(T) == 4) ? 1 : vec ? kRows : a.res ? kTiles / 2 : kTiles;
  const int64_t units = (a.T + rows - 1) / rows * per_row;
  const int64_t ctas = (units + per_cta - 1) / per_cta;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;  // 2^31 x 4 KB is no GPU's memory
  const DropoutParams p = {a.x, a.res, a.y, a.ldx, a.ldres, a.ldy, a.T, a.N, units,
                           Divisor((uint32_t)per_row),
                           {a.drop.seed, a.drop.step, a.drop.threshold, a.drop.scale}};
  void (*kern)(DropoutParams) = many ? dropout_kernel<T, kRows> : dropout_kernel<T, 1>;
  if (!vec) {
    if constexpr (sizeof(T) == 2)
      kern = a.res ? (many ? dropout_shifted_kernel<T, kTiles / 2, true> : dropout_shifted_kernel<T, 1, true>)
                   : (many ? dropout_shifted_kernel<T, kTiles, false> : dropout_shifted_kernel<T, 1, false>);
    else
      kern = dropout_elements_kernel<T>;
  }
  return launch_pdl(kern, dim3((unsigned)ctas), dim3(kThreads), 0, st, p);
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
