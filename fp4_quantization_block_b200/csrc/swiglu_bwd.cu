// swiglu_bwd.cu -- backward pass of the SwiGLU activation whose forward pass
// is the producer of the down projection's input (quantize.cu).
//
// h = silu(g) u, silu(g) = g sg, sg = 1 / (1 + exp(-g)):
//   du = dh silu(g),   dg = dh u sg (1 + g (1 - sg)),
// in binary32, each rounded once to bf16.  With e = exp(-|g|) <= 1 the sigmoid
// and 1 - sg are 1 / (1 + e) and e / (1 + e) in the order of g's sign: neither
// overflows or cancels, and sg keeps its value for g below -87, where exp(-g)
// leaves the range that the reciprocal takes.  The reciprocal, of a value
// between one and two, is the hardware's estimate (one unit in the last place,
// far inside bf16's step).
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
  uint64_t gf[4], uf[4], df[4];
  unpack8(g, gf);
  unpack8(u, uf);
  unpack8(d, df);
  const uint64_t one = f2_set(1.0f);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = f2_lo(gf[j]), hi = f2_hi(gf[j]);
    const uint64_t e = f2_pack(expf(-fabsf(lo)), expf(-fabsf(hi))), sum = f2_add(one, e);
    const float rl = reciprocal(f2_lo(sum)), rh = reciprocal(f2_hi(sum));
    const uint64_t s = f2_mul(e, f2_pack(rl, rh));
    const float sl = f2_lo(s), sh = f2_hi(s);
    const uint64_t sg = f2_pack(lo < 0.0f ? sl : rl, hi < 0.0f ? sh : rh);
    const uint64_t rest = f2_pack(lo < 0.0f ? rl : sl, hi < 0.0f ? rh : sh);  // 1 - sg
    const uint64_t du = f2_mul(df[j], f2_mul(gf[j], sg));
    gf[j] = f2_mul(f2_mul(df[j], uf[j]), f2_mul(sg, f2_fma(gf[j], rest, one)));
    uf[j] = du;
  }
  pack8(gf, g);
  pack8(uf, u);
  uint16_t *dz = p.dz + row * p.lddz + c;
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
