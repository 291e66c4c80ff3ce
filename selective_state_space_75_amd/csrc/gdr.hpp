// gdr.hpp -- device helpers shared by the gated delta rule's kernels (gfx950).
#pragma once

#include "device_math.hpp"
#include "kernels.hpp"

namespace mamba {

__device__ __forceinline__ float gdr_load(const float* p) { return *p; }
__device__ __forceinline__ float gdr_load(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void gdr_store(float* p, float x) { *p = x; }
__device__ __forceinline__ void gdr_store(uint16_t* p, float x) { *p = f32_to_bf16(x); }

// Sum over the 16 lanes of a lane group, in every lane (rotations inside the group:
// four vector adds, no LDS).
__device__ __forceinline__ float gdr_sum16(float x) {
#define GDR_ROR(n) \
  x += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + n, 0xf, 0xf, true))
  GDR_ROR(8);
  GDR_ROR(4);
  GDR_ROR(2);
  GDR_ROR(1);
#undef GDR_ROR
  return x;
}

// Tokens of batch row b that count: all L, or lengths[b] held to 0 .. L.
__device__ __forceinline__ int64_t gdr_length(const GdrParams& p, int64_t b) {
  if (!p.lengths) return p.L;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

__device__ __forceinline__ float gdr_sigmoid(float x) { return hw_rcp(1.0f + hw_exp2(-x * kLog2e)); }

// a = exp(A softplus(x))
__device__ __forceinline__ float gdr_decay(float x, float A) { return hw_exp2(softplus(x) * A * kLog2e); }

// 1 / |x| of a key or query from its sum of squares.  One Newton step on the
// hardware's reciprocal root (1 ulp) leaves about half an ulp: the factor goes
// into every number of the row.
__device__ __forceinline__ float gdr_rnorm(float ss) {
  const float s = ss + kGdrNormEps;
  const float r = __builtin_amdgcn_rsqf(s);
  return r * __builtin_fmaf(-0.5f * s * r, r, 1.5f);
}

}  // namespace mamba
