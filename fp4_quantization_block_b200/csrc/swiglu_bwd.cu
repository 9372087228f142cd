// swiglu_bwd.cu -- backward pass of the SwiGLU activation whose forward pass
// is the producer of the down projection's input (quantize.cu).
//
// h = silu(g) u, silu(g) = g sg, sg = 1 / (1 + exp(-g)):
//   du = dh silu(g),   dg = dh u sg (1 + g (1 - sg)),
// in binary32, each rounded once to bf16.  The reciprocal is the hardware's
// estimate (one unit in the last place, far inside bf16's step).  For gates
// below -87 1 + exp(-g) leaves the range that it takes and sg would be zero, so
// a thread that has one takes a form of its own, out of line, which leaves the
// others their 32 registers (8192 x 14336 in a stream of calls 175.5 us, 173.2
// without the question; one form for all, from exp(-|g|), 179, and on packed
// pairs, with 38 registers, 183).
//
// Bound by memory: 10 bytes per element of h.  8192 x 14336 takes 171 us, 6.85
// TB/s.  One chunk of eight channels per thread (two or four are as fast there
// and slower for few rows: 96 x 14336 3.9, 4.3 and 4.9 us); the grid covers dh
// once.
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa4_kernels.h"
#include "launch.cuh"
#include "rows.cuh"

namespace fa4 {
namespace {

using namespace rows;

constexpr int kThreads = 256;

__device__ __forceinline__ float reciprocal(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Whether one of eight gates is below -87: as unsigned 16-bit numbers, the
// negative ones of larger magnitude (NaN among them) are above -87's.
__device__ __forceinline__ bool any_far(const uint4 &g) {
  const uint32_t m = __vimax3_u16x2(__vimax3_u16x2(g.x, g.y, g.z), g.w, 0u);
  return m > 0xC2AEFFFFu || (m << 16) > 0xC2AEFFFFu;
}
// A thread's eight channels where any_far, from memory again: below -87 sg is
// exp(g) to binary32's last bit, the other gates' is what it is beside others.
__device__ __noinline__ void far_gates(const uint16_t *z, int64_t F, const uint16_t *dh, uint16_t *dz) {
  using T = __nv_bfloat16;
  for (int j = 0; j < 8; ++j) {
    const float g = to_float(reinterpret_cast<const T *>(z)[j]), u = to_float(reinterpret_cast<const T *>(z)[F + j]);
    const float d = to_float(reinterpret_cast<const T *>(dh)[j]);
    const float e = expf(g < -87.0f ? g : -g), sg = g < -87.0f ? e : reciprocal(1.0f + e);
    reinterpret_cast<T *>(dz)[j] = from_float<T>(d * u * (sg * fmaf(g, 1.0f - sg, 1.0f)));
    reinterpret_cast<T *>(dz)[F + j] = from_float<T>(d * (g * sg));
  }
}

// dz may be z itself: a thread reads its elements before it writes them.
__global__ void __launch_bounds__(kThreads) swiglu_bwd_kernel(const SwigluBwdArgs p, const int64_t units,
                                                              const Divisor per_row) {
  using T = __nv_bfloat16;
  grid_dependency_wait();
  grid_dependents_launch();
  const int64_t first = (int64_t)blockIdx.x * kThreads;
  if (first + threadIdx.x >= units) return;
  const int64_t row0 = units < (int64_t(1) << 31) ? per_row.quotient((uint32_t)first) : first / per_row.d;
  const uint32_t n = (uint32_t)(first - row0 * per_row.d) + threadIdx.x, q = per_row.quotient(n);
  const int64_t row = row0 + q, c = 8 * (int64_t)(n - q * per_row.d);
  const uint16_t *z = p.z + row * p.ldz + c;
  Raw8<T> g, u, d;
  g.v[0] = __ldcs(reinterpret_cast<const uint4 *>(z));
  u.v[0] = __ldcs(reinterpret_cast<const uint4 *>(z + p.F));
  d.v[0] = __ldcs(reinterpret_cast<const uint4 *>(p.dh + row * p.lddh + c));
  const bool far = any_far(g.v[0]);
  float gf[8], uf[8], df[8];
  unpack8(g, gf);
  unpack8(u, uf);
  unpack8(d, df);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float sg = reciprocal(1.0f + expf(-gf[j]));
    const float du = df[j] * (gf[j] * sg);
    gf[j] = df[j] * uf[j] * (sg * fmaf(gf[j], 1.0f - sg, 1.0f));
    uf[j] = du;
  }
  pack8(gf, g);
  pack8(uf, u);
  uint16_t *dz = p.dz + row * p.lddz + c;
  if (far) {  // (nothing of it is stored yet)
    far_gates(z, p.F, p.dh + row * p.lddh + c, dz);
    return;
  }
  *reinterpret_cast<uint4 *>(dz) = g.v[0];
  *reinterpret_cast<uint4 *>(dz + p.F) = u.v[0];
}

}  // namespace

cudaError_t launch_swiglu_bwd(const SwigluBwdArgs &a, cudaStream_t st) {
  const int64_t per_row = a.F / 8, units = a.T * per_row;
  const int64_t ctas = (units + kThreads - 1) / kThreads;
  if (ctas >= (int64_t(1) << 31)) return cudaErrorInvalidValue;  // 2^31 x 4 KB is no GPU's memory
  return launch_pdl(swiglu_bwd_kernel, dim3((unsigned)ctas), dim3(kThreads), 0, st, a, units,
                    Divisor((uint32_t)per_row));
}

}  // namespace fa4
