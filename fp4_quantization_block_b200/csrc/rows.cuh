// rows.cuh -- device helpers of the row-wise training operators (norm.cu,
// dropout.cu): element types, chunks of eight columns, sums over a row's
// threads, and the dropout mask.
//
// A thread's unit is a chunk: eight consecutive columns of one row, which is
// one 16-byte access of a 16-bit type (two of binary32) and one block of the
// mask's generator.  Arithmetic is binary32 whatever the element type; a
// value is rounded once, where it is stored.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "fa4_device.cuh"

namespace fa4 {
namespace rows {

// ------------------------------------------------------------ elements ---
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_float<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_float<float>(float v) {
  return v;
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw8 {
  uint4 v[sizeof(T) / 2];
};
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo(w[i]);
    f[2 * i + 1] = bf16hi(w[i]);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__half> &r, float (&f)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float> &r, float (&f)[8]) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w,
                         r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
__device__ __forceinline__ void pack8(const float (&f)[8], Raw8<__nv_bfloat16> &r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack8(const float (&f)[8], Raw8<__half> &r) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 b = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&b);
  }
  r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void pack8(const float (&f)[8], Raw8<float> &r) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(f[i]);
  r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  r.v[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

// Columns c .. c+7 of a row of `cols`, zeros past its end.  VEC: the row
// starts on a 16-byte boundary and cols is a multiple of eight, so a chunk is
// wholly inside or wholly outside.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *row, int64_t c, int64_t cols, float (&f)[8]) {
  if constexpr (VEC) {
    Raw8<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i)
      r.v[i] = c < cols ? reinterpret_cast<const uint4 *>(row + c)[i] : make_uint4(0u, 0u, 0u, 0u);
    unpack8(r, f);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? to_float(row[c + i]) : 0.0f;
  }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store8(T *row, int64_t c, int64_t cols, const float (&f)[8]) {
  if constexpr (VEC) {
    if (c < cols) {
      Raw8<T> r;
      pack8(f, r);
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(row + c)[i] = r.v[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < cols) row[c + i] = from_float<T>(f[i]);
  }
}
// The same eight values as they read back from memory.
template <typename T>
__device__ __forceinline__ void round8(float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_float(from_float<T>(f[i]));
}

// A weight or bias vector: binary32 or the activations' type.
template <typename T>
struct Vec {
  const void *p;
  int f32;
  __device__ __forceinline__ float at(int64_t c) const {
    return f32 ? static_cast<const float *>(p)[c] : to_float(static_cast<const T *>(p)[c]);
  }
};

// -------------------------------------------------------------- dropout ---
// The mask is a function of (key, row, column) and is never stored: element
// (r, c) has 16 random bits u, the half c & 1 of word (c >> 1) & 3 of
// Philox4x32-7 (fa4_device.cuh) on the counter (c >> 3, r, 0, kDropTag) under
// the 64-bit key seed + *step, and is kept iff u >= threshold.  The tag keeps
// these counters apart from the stochastic-rounding ones, whose words 2 and 3
// are zero, under any key.  A kept value is multiplied by 65536 / (65536 -
// threshold), the reciprocal of the exact probability of being kept.
constexpr uint32_t kDropTag = 0x44524F50u;
struct Drop {
  uint64_t seed;
  const uint64_t *step;  // device scalar added to seed; may be null
  uint32_t threshold;    // in [0, 65535]: the probability of being dropped x 65536
  float scale;           // 65536 / (65536 - threshold)
  __device__ __forceinline__ uint64_t key() const { return seed + (step ? *step : 0ull); }
};
// Eight columns from c (a multiple of eight): kept values scaled, dropped
// ones zero whatever they were (a dropped infinity or NaN leaves no trace).
__device__ __forceinline__ void drop8(const Drop &d, uint64_t key, uint32_t row, uint32_t c,
                                      float (&f)[8]) {
  if (d.threshold == 0u) return;
  const u32x4 b = philox(c >> 3, row, 0u, kDropTag, (uint32_t)key, (uint32_t)(key >> 32));
  const uint32_t w[4] = {b.x, b.y, b.z, b.w}, t = d.threshold << 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = (w[i] << 16) >= t ? f[2 * i] * d.scale : 0.0f;
    f[2 * i + 1] = w[i] >= t ? f[2 * i + 1] * d.scale : 0.0f;
  }
}

// ----------------------------------------------------------------- sums ---
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// ----------------------------------------------- rows kept on the chip ---
// A team of W warps holds one row: warp w's j-th tile is the 256 columns from
// 256 (j W + w), lane l's chunk the eight from 8 l in it.  Tiles come through
// a ring of stages in shared memory, private to the warp, filled by
// asynchronous copies several rows ahead, so that what is in flight does not
// depend on registers; a warp waits only for its own copies.
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest n groups of this thread have arrived.
__device__ __forceinline__ void cp_async_wait(int n) {
  if (n >= 3)
    asm volatile("cp.async.wait_group 3;" ::: "memory");
  else if (n == 2)
    asm volatile("cp.async.wait_group 2;" ::: "memory");
  else if (n == 1)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}
constexpr int kMaxStages = 4;

// A warp's copy of columns cb .. cb+255 (those below cols) of a row into a
// tile.  VEC: 16-byte copies.  Otherwise 4-byte ones where the row allows
// them (`words`: binary32, or 16-bit rows that start on 4-byte boundaries),
// and plain loads for 16-bit rows that do not.  Visible to the warp after
// cp_async_wait and __syncwarp.
template <typename T, bool VEC>
__device__ __forceinline__ void fill_tile(T *tile, const T *row, int cb, int cols, bool words, int lane) {
  constexpr int kPer16 = 16 / (int)sizeof(T), kPer4 = 4 / (int)sizeof(T);
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 256 / (32 * kPer16); ++i) {
      const int e = (32 * i + lane) * kPer16;
      if (cb + e < cols) cp_async16(tile + e, row + cb + e);
    }
  } else if (sizeof(T) == 4 || words) {
#pragma unroll
    for (int i = 0; i < 256 / (32 * kPer4); ++i) {
      const int e = (32 * i + lane) * kPer4;
      if (cb + e + kPer4 <= cols)
        cp_async4(tile + e, row + cb + e);
      else if (cb + e < cols)
        tile[e] = row[cb + e];
    }
  } else {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (cb + 32 * i + lane < cols) v[i] = row[cb + 32 * i + lane];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (cb + 32 * i + lane < cols) tile[32 * i + lane] = v[i];
  }
}
// A lane's chunk of a tile at column c = cb + 8 lane, zeros from cols on.
template <typename T, bool VEC>
__device__ __forceinline__ void read_tile(const T *tile, int c, int cols, int lane, float (&f)[8]) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = reinterpret_cast<const uint4 *>(tile + 8 * lane)[i];
  unpack8(r, f);
  if (VEC) {
    if (c >= cols)
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = c + i < cols ? f[i] : 0.0f;
  }
}
// Stores the warp's 256 columns from cb, lane l holding the eight from 8 l:
// 16-bit chunks directly, the others through `tile` (which the warp has
// finished reading), so that neighbouring lanes write neighbouring bytes.
template <typename T, bool VEC>
__device__ __forceinline__ void store_tile(T *tile, T *row, int cb, int cols, bool words, int lane,
                                           const float (&f)[8]) {
  constexpr int kPer16 = 16 / (int)sizeof(T), kPer4 = 4 / (int)sizeof(T);
  Raw8<T> r;
  pack8(f, r);
  if constexpr (VEC && sizeof(T) == 2) {
    if (cb + 8 * lane < cols) *reinterpret_cast<uint4 *>(row + cb + 8 * lane) = r.v[0];
    return;
  }
  __syncwarp();  // the tile's last readers
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<uint4 *>(tile + 8 * lane)[i] = r.v[i];
  __syncwarp();
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < 256 / (32 * kPer16); ++i) {
      const int e = (32 * i + lane) * kPer16;
      if (cb + e < cols) *reinterpret_cast<uint4 *>(row + cb + e) = *reinterpret_cast<const uint4 *>(tile + e);
    }
  } else if (sizeof(T) == 4 || words) {
#pragma unroll
    for (int i = 0; i < 256 / (32 * kPer4); ++i) {
      const int e = (32 * i + lane) * kPer4;
      if (cb + e + kPer4 <= cols)
        *reinterpret_cast<uint32_t *>(row + cb + e) = *reinterpret_cast<const uint32_t *>(tile + e);
      else if (cb + e < cols)
        row[cb + e] = tile[e];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = 32 * i + lane;
      if (cb + e < cols) row[cb + e] = tile[e];
    }
  }
}

// Sums of K values over a team of W warps, the same bits in every thread: a
// butterfly in the warp, then over the warps' sums.  `red` holds W x K floats;
// two uses of one buffer need a barrier of the team between them.
template <int K>
__device__ __forceinline__ void team_sum(float (&v)[K], float *red, int W, int warp, int lane, int bar) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (W == 1) return;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[warp * K + k] = v[k];
  asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(32 * W) : "memory");
  const int pow2 = W > 8 ? (W > 16 ? 32 : 16) : (W > 4 ? 8 : (W > 2 ? 4 : 2)), l = lane & (pow2 - 1);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = l < W ? red[l * K + k] : 0.0f;
  for (int o = pow2 >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], o);
}

}  // namespace rows
}  // namespace fa4
