// rows.cuh -- device helpers of the row-wise training operators (norm_fwd.cuh,
// norm_bwd.cuh, dropout.cu, swiglu_bwd.cu): element types, chunks of eight
// columns, sums over a row's threads, the dropout mask, rows kept on the chip,
// and the exchange between the CTAs of a cluster.
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

// ------------------------------------------------------------- division ---
// Quotients by a divisor d < 2^31 known on the host, for n < 2^31: with s =
// ceil(log2 d) and m = ceil(2^(32 + s) / d) - 2^32, n / d = (hi(m n) + n) >> s
// exactly (Granlund and Montgomery, "Division by invariant integers using
// multiplication", PLDI 1994; the sum stays below 2^32 for these n).
struct Divisor {
  uint32_t d, m, s;
  Divisor() = default;
  explicit Divisor(uint32_t v) : d(v), m(0), s(0) {
    while ((uint64_t(1) << s) < v) ++s;
    m = (uint32_t)(((uint64_t(1) << 32) * ((uint64_t(1) << s) - v)) / v + 1);
  }
  __device__ __forceinline__ uint32_t quotient(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

// ---------------------------------------------------------------- pairs ---
// A chunk as four packed binary32 pairs, for arithmetic at two values an
// instruction (fa4_device.cuh): pair i holds columns 2i and 2i + 1.
__device__ __forceinline__ uint64_t f2_set(float v) { return f2_pack(v, v); }
__device__ __forceinline__ float f2_lo(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return a;
}
__device__ __forceinline__ float f2_hi(uint64_t v) {
  float a, b;
  f2_unpack(v, a, b);
  return b;
}
__device__ __forceinline__ float f2_sum(uint64_t v) { return f2_lo(v) + f2_hi(v); }
template <typename T>
__device__ __forceinline__ void unpack8(const Raw8<T> &r, uint64_t (&f)[4]) {
  float v[8];
  unpack8(r, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_pack(v[2 * i], v[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ void pack8(const uint64_t (&f)[4], Raw8<T> &r) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(f[i], v[2 * i], v[2 * i + 1]);
  pack8(v, r);
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
// A team of warps holds one row: a warp has CH tiles of 256 columns each, one
// after the other; a lane has eight values of a tile as four pairs, for 16-bit
// types the columns from 8 l, for binary32 four from 4 l and four from 128 +
// 4 l, so that a warp's 16-byte accesses to memory and to shared memory are
// consecutive.  Tiles come through a ring of stages in shared memory, private
// to the warp, filled by asynchronous copies several rows ahead, so that what
// is in flight does not depend on registers; a warp waits only for its own
// copies.
__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
__device__ __forceinline__ void cp_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// Only the first `bytes` are read; the rest of the 16 are zeros.
__device__ __forceinline__ void cp_async16(void *dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes)
               : "memory");
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
constexpr int kTile = 256;

// The tile column of a lane's pair i (its first value).
template <typename T>
__device__ __forceinline__ int pair_col(int lane, int i) {
  return sizeof(T) == 2 ? 8 * lane + 2 * i : (i < 2 ? 0 : 124) + 4 * lane + 2 * i;
}
// Dropout of a lane's pairs with the bits of its two half blocks.
__device__ __forceinline__ void drop_pairs(const Drop &d, const uint32_t (&w)[4], uint64_t (&f)[4]) {
  const uint32_t t = d.threshold << 16;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    f2_unpack(f2_mul(f[i], f2_set(d.scale)), lo, hi);
    f[i] = f2_pack((w[i] << 16) >= t ? lo : 0.0f, w[i] >= t ? hi : 0.0f);
  }
}
// The bits of a binary32 lane, which has four columns of each of two blocks:
// of a pair of lanes the even one has the first halves and computed the first
// block's bits b, the odd one the second halves and the second block's; they
// exchange the words that the other needs.
__device__ __forceinline__ void share_bits(const u32x4 &b, int lane, uint32_t (&w)[4]) {
  const bool odd = lane & 1;
  const uint32_t g0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? b.x : b.z, 1);
  const uint32_t g1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? b.y : b.w, 1);
  w[0] = odd ? g0 : b.x;
  w[1] = odd ? g1 : b.y;
  w[2] = odd ? b.z : g0;
  w[3] = odd ? b.w : g1;
}
// Dropout of a lane's values of the tile whose first generator block is
// `group`.
template <typename T>
__device__ __forceinline__ void drop_tile(const Drop &d, uint64_t key, uint32_t row, uint32_t group, int lane,
                                          uint64_t (&f)[4]) {
  if (d.threshold == 0u) return;
  const uint32_t mine = sizeof(T) == 2 ? lane : (lane >> 1) + 16 * (lane & 1);
  const u32x4 b = philox(group + mine, row, 0u, kDropTag, (uint32_t)key, (uint32_t)(key >> 32));
  uint32_t w[4] = {b.x, b.y, b.z, b.w};
  if constexpr (sizeof(T) == 4) share_bits(b, lane, w);
  drop_pairs(d, w, f);
}

// A tile of a ring.  VEC: rows on 16-byte boundaries.  Otherwise a row starts
// `mis` bytes past one, and the tile holds the aligned 16-byte words that the
// columns lie in, one word more.
template <typename T, bool VEC>
constexpr int kTileLen = VEC ? kTile : kTile + 16 / (int)sizeof(T);
__device__ __forceinline__ int misaligned(const void *p) { return (int)(reinterpret_cast<uintptr_t>(p) & 15u); }

// A warp's copy of the first `left` of 256 columns from src into a tile, zeros
// after them (VEC: what lies after them is not touched).  Visible to the warp
// after cp_async_wait and __syncwarp.  Unless VEC the first word may begin
// before src, in the row before or its padding; `head` says that there is no
// such row, and the word is copied by elements.
template <typename T, bool VEC>
__device__ __forceinline__ void fill_tile(T *tile, const T *src, int left, bool head, int lane) {
  constexpr int kPer16 = 16 / (int)sizeof(T), kWords = kTile / kPer16;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < kWords / 32; ++i) {
      const int e = (32 * i + lane) * kPer16;
      if (e < left) cp_async16(tile + e, src + e);
    }
  } else {
    if (left <= 0) return;  // a tile past the row's end
    const int mis = misaligned(src);
    const char *word0 = reinterpret_cast<const char *>(src) - mis;
    if (left >= kTile + kPer16 && !(head && mis)) {  // every word whole, and the one after them
#pragma unroll
      for (int i = 0; i < kWords; i += 32) cp_async16(tile + (i + lane) * kPer16, word0 + 16 * (i + lane));
      if (lane == 0) cp_async16(tile + kTile, word0 + 16 * kWords);
      return;
    }
    const int total = (left < kTile ? left : kTile) * (int)sizeof(T) + mis;
#pragma unroll
    for (int i = 0; i < kWords + 1; i += 32) {
      const int w = i + lane;
      if (w > kWords) break;
      const int bytes = total - 16 * w;
      if (w == 0 && head && mis) {
        const int off = mis / (int)sizeof(T);
        for (int e = 0; e < kPer16 - off; ++e) tile[off + e] = e < left ? src[e] : from_float<T>(0.0f);
      } else {
        cp_async16(tile + w * kPer16, bytes > 0 ? word0 + 16 * w : word0, bytes < 0 ? 0 : bytes > 16 ? 16 : bytes);
      }
    }
  }
}
// Zeros a tile of `len` elements from `left` on, which no copy touches
// afterwards: those columns read as zeros in every row.
template <typename T>
__device__ __forceinline__ void clear_tail(T *tile, int left, int len, int lane) {
  for (int e = (left > 0 ? left : 0) + lane; e < len; e += 32) tile[e] = from_float<T>(0.0f);
}
// The 16 bytes that start `mis` (even, the same in the whole warp) bytes into
// two neighbouring words.
__device__ __forceinline__ uint4 shifted(const uint4 &a, const uint4 &b, int mis) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (mis & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (mis & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  if (mis & 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// A lane's values of a tile (mis: of the row's start, unless VEC).
template <typename T, bool VEC>
__device__ __forceinline__ void read_tile(const T *tile, int mis, int lane, uint64_t (&f)[4]) {
  constexpr int kLane = sizeof(T) == 2 ? 8 : 4;
  Raw8<T> r;
#pragma unroll
  for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
    const uint4 *w = reinterpret_cast<const uint4 *>(tile + 128 * h + kLane * lane);
    r.v[h] = VEC ? w[0] : shifted(w[0], w[1], mis);
  }
  unpack8(r, f);
}
// Stores the first `left` of the warp's CH x 256 columns at dst.  VEC: each
// lane its 16-byte words.  Otherwise through `stage` (CH tiles that the warp
// has finished reading): the columns in order, then the aligned words of dst
// out of them, and the elements before the first and after the last of these.
template <typename T, int CH, bool VEC>
__device__ __forceinline__ void store_tiles(T *stage, T *dst, int left, int lane, const uint64_t (&f)[CH][4]) {
  constexpr int kLane = sizeof(T) == 2 ? 8 : 4, P = 16 / (int)sizeof(T);
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      Raw8<T> r;
      pack8(f[j], r);
#pragma unroll
      for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
        const int c = j * kTile + 128 * h + kLane * lane;
        if (c < left) *reinterpret_cast<uint4 *>(dst + c) = r.v[h];
      }
    }
  } else {
    if (left <= 0) return;  // a warp past the row's end
    __syncwarp();  // the stage's last readers
#pragma unroll
    for (int j = 0; j < CH; ++j) {
      Raw8<T> r;
      pack8(f[j], r);
#pragma unroll
      for (int h = 0; h < (int)sizeof(T) / 2; ++h)
        *reinterpret_cast<uint4 *>(stage + j * kTile + 128 * h + kLane * lane) = r.v[h];
    }
    __syncwarp();
    const int n = left < CH * kTile ? left : CH * kTile;
    const int mis = misaligned(dst), off = mis / (int)sizeof(T);
    // word k of dst's has the columns from k P - off
#pragma unroll
    for (int i = 0; i <= CH * kTile / P; i += 32) {
      const int k = i + lane, c = k * P - off;
      if (c >= 0 && c + P <= n) {
        const uint4 *w = reinterpret_cast<const uint4 *>(stage) + k;
        *reinterpret_cast<uint4 *>(dst + c) = mis ? shifted(w[-1], w[0], 16 - mis) : w[0];
      }
    }
    const int head = !mis ? 0 : P - off < n ? P - off : n;
    const int last = (n + off) / P * P - off, tail = last > head ? last : head;
    const int c = lane < 16 ? lane : tail + lane - 16;
    if (lane < 16 ? c < head : c < n) dst[c] = stage[c];
  }
}

// Weights in shared memory as a lane reads them: those of binary32 beside
// 16-bit rows as two planes per tile, the lanes' first four columns and their
// last four; the others as they lie.
template <typename T, typename W>
__device__ __forceinline__ int vec_slot(int c) {
  if (sizeof(T) == 2 && sizeof(W) == 4)
    return (c & ~(kTile - 1)) + 128 * ((c >> 2) & 1) + 4 * ((c >> 3) & 31) + (c & 3);
  return c;
}
// The CTA's copy of `cols` weights, zeros up to `room` (complete after
// cp_async_wait and a barrier).  vec: they start on a 16-byte boundary.
template <typename T, typename W>
__device__ __forceinline__ void stage_vec(W *dst, const W *src, int cols, int room, bool vec) {
  constexpr int kPer16 = 16 / (int)sizeof(W);
  const int whole = vec ? cols / kPer16 * kPer16 : 0;
  for (int c = kPer16 * threadIdx.x; c < whole; c += kPer16 * blockDim.x)
    cp_async16(dst + vec_slot<T, W>(c), src + c);
  for (int c = whole + threadIdx.x; c < room; c += blockDim.x)
    dst[vec_slot<T, W>(c)] = c < cols ? src[c] : from_float<W>(0.0f);
}
// A lane's staged weights of a tile.
template <typename T, typename W>
__device__ __forceinline__ void read_vec(const W *tile, int lane, uint64_t (&f)[4]) {
  static_assert(sizeof(W) == 4 || sizeof(T) == sizeof(W), "weights of the rows' type or binary32");
  read_tile<W, true>(tile, 0, lane, f);
}

// ------------------------------------------------------------- clusters ---
// The CTAs of a cluster exchange small sums by asynchronous stores that count
// their bytes at a barrier beside the place they go to: the receivers wait for
// exactly these, and no fence waits for the senders' stores to memory.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
// Sends v to the same place of the CTA `rank`, eight bytes at its barrier.
__device__ __forceinline__ void cluster_send(float2 *place, uint64_t *barrier, int rank, float2 v) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(
                   cluster_addr(smem_addr(place), rank)),
               "f"(v.x), "f"(v.y), "r"(cluster_addr(smem_addr(barrier), rank))
               : "memory");
}
__device__ __forceinline__ void barrier_init(uint64_t *barrier) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(smem_addr(barrier)) : "memory");
}
// The one arrival of a phase, and the bytes that the phase waits for.
__device__ __forceinline__ void barrier_expect(uint64_t *barrier, int bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(barrier)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ uint64_t globaltimer() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
// Waits for a phase; false if it did not complete within timeout_ns.
__device__ __forceinline__ bool barrier_wait(uint64_t *barrier, uint32_t parity, uint64_t timeout_ns) {
  const uint32_t addr = smem_addr(barrier);
  uint64_t begin = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(addr), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 15u) == 15u) {
      const uint64_t now = globaltimer();
      if (begin == 0) begin = now;
      if (now - begin > timeout_ns) return false;
    }
  }
}
// A barrier of all threads of the cluster.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace rows
}  // namespace fa4
