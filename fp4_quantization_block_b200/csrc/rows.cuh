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

}  // namespace rows
}  // namespace fa4
