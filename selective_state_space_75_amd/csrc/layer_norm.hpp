// layer_norm.hpp -- device helpers shared by the layer norm's kernels (gfx950).
#pragma once

#include <type_traits>

#include "glr.hpp"

namespace mamba {

// 1 / sqrt(v), the hardware's root with one Newton step (about half an ulp): it goes into every
// number of the token.
__device__ __forceinline__ float norm_root(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float h = __builtin_fmaf(-0.5f * v * r, r, 1.5f);
  return r * (v < 1e37f && v > 1e-37f ? h : 1.0f);
}

// Halves a wave's numbers over its halves: a becomes the sum over lane ^ 32 of a in the lower 32
// lanes, and of b in the upper.
__device__ __forceinline__ float fold32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false,
                                                  false);
  const uint32_t x = r[0], y = r[1];
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}
// The same over lane ^ 16: a in even rows of 16 lanes, b in odd ones.
__device__ __forceinline__ float fold16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false,
                                                  false);
  const uint32_t x = r[0], y = r[1];
  return __builtin_bit_cast(float, x) + __builtin_bit_cast(float, y);
}

// Sum over the lanes of a row of 16 that share lane % kT, in all of them.
template <int kT>
__device__ __forceinline__ float row_sum(float x) {
  if constexpr (kT <= 8) x += dpp<0x128, 0xf>(0.0f, x);
  if constexpr (kT <= 4) x += dpp<0x124, 0xf>(0.0f, x);
  if constexpr (kT <= 2) x += dpp<0x122, 0xf>(0.0f, x);
  if constexpr (kT <= 1) x += dpp<0x121, 0xf>(0.0f, x);
  return x;
}

// Sums of kN numbers (a multiple of 4) over the lanes of a workgroup that share threadIdx.x % kT
// (kT <= 8), in every lane.  Inside a wave the numbers are folded over its halves and rows, so that each
// exchange halves how many there are; a quarter of them per row of 16 lanes is then left in LDS,
// summed over the waves by one lane per sum, and read back.
// lds: (waves + 1) * kT * kN floats.
template <int kT, int kN, int kThreads>
__device__ __forceinline__ void group_sum(float (&v)[kN], float* lds) {
  static_assert(kN % 4 == 0 && kT <= 8, "four quarters");
  constexpr int kWaves = kThreads / 64, kQ = kN / 4;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float h[kN / 2], q[kQ];
#pragma unroll
  for (int j = 0; j < kN / 2; ++j) h[j] = fold32(v[j], v[j + kN / 2]);
#pragma unroll
  for (int j = 0; j < kQ; ++j) q[j] = row_sum<kT>(fold16(h[j], h[j + kQ]));
  // row 0 holds numbers 0 .., row 1 those from kQ, row 2 from 2 kQ, row 3 from 3 kQ
  float* total = lds + kWaves * kT * kN;
  __syncthreads();                       // an earlier sum may still be read
  if ((lane & 15) < kT) {
    float* at = (kWaves > 1 ? lds + wave * kT * kN : total) + (lane & 15) * kN + (lane >> 4) * kQ;
#pragma unroll
    for (int j = 0; j < kQ; ++j) at[j] = q[j];
  }
  __syncthreads();
  if constexpr (kWaves > 1) {
    if (threadIdx.x < kT * kN) {
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) s += lds[w * kT * kN + threadIdx.x];
      total[threadIdx.x] = s;
    }
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = total[(lane % kT) * kN + j];
}

// Sum of kN numbers over a team of 2^k <= 64 neighbouring lanes, or (kWaves) of team / 64 <= 16 whole waves, in every lane
// of it.  Lane l of a row of 16 reads wave l's sum, so that all waves' come in one round trip to LDS (read one after
// the other they took a tenth of a token's time with ten waves, and a fifth with 14; for two waves it is the other
// way round, 1000 channels 18.9 us, 19.8.  kMany: there are more than two).  lds: waves * kN floats.
template <int kN, bool kWaves, bool kMany = false>
__device__ __forceinline__ void team_sum(float (&v)[kN], int team, float* lds) {
  if constexpr (!kWaves) {
    for (int m = 1; m < team; m *= 2) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] += __shfl_xor(v[j], m);
    }
  } else {
    const int lane = threadIdx.x & 63, w = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int of = team >> 6, first = wave - wave % of;
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] = wave_sum63(v[j]);
    __syncthreads();                     // an earlier sum may still be read
    if (lane == 63) {
#pragma unroll
      for (int j = 0; j < kN; ++j) lds[wave * kN + j] = v[j];
    }
    __syncthreads();
    if (!kMany && of <= 2) {
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = lds[first * kN + j] + (of == 2 ? lds[(first + of - 1) * kN + j] : 0.0f);
    } else {
      const float* at = lds + (first + (w < of ? w : 0)) * kN;
#pragma unroll
      for (int j = 0; j < kN; ++j) v[j] = lane_of(row_sum<1>(w < of ? at[j] : 0.0f), 0);
    }
  }
}

// Workgroups go to the eight XCDs in turn.  Work is renumbered so that each XCD has a contiguous
// range of it: neighbouring tiles share cache lines, and those then meet in one L2.
__device__ __forceinline__ int64_t by_xcd(int64_t i, int64_t n) {
  const int64_t xcd = i & 7, q = n >> 3, r = n & 7;
  return xcd * q + (xcd < r ? xcd : r) + (i >> 3);
}

template <typename T>
__device__ __forceinline__ Raw8<T> load_all8(const T* p) {
  Raw8<T> o;
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k) o.w[k] = *(reinterpret_cast<const u32x4_u*>(p) + k);
  return o;
}
// base[v]: a base that the workgroup shares and a lane's 32-bit offset (v * sizeof(T) < 2^32), one register for
// all the channels of a lane.
template <typename T>
__device__ __forceinline__ T* lane_at(T* base, uint32_t v) {
  using Byte = std::conditional_t<std::is_const_v<T>, const char, char>;
  return reinterpret_cast<T*>(reinterpret_cast<Byte*>(base) + (uint32_t)(v * sizeof(T)));
}

// Whether a tile's results go past the caches.  They do where they are whole cache lines, rows being `row` bytes apart.
// Parts of a line are left to meet the neighbouring tile's in L2 (4 x 5120 channels in 40 groups, L = 1003, fp32: forward
// 81 us past the caches, 43 through them, backward 92, 64, gated 182, 105), unless a call's results, `all` bytes
// of them, fit into the 32 MB of the L2s and `few` says that this is faster: 2-byte numbers (8 x 500 channels,
// L = 2045, gated: 20.0, 24.4, backward 33.0, 35.5) and the gated backward pass (12 heads of 80, 3 x 1003 tokens, fp32:
// 22.9, 24.8), not ungated fp32 (8 x 200 channels, L = 2045: 12.6, 10.6, backward 20.0, 17.4).
__device__ __forceinline__ bool past_caches(const void* base, int64_t row, int64_t all, bool few) {
  return (reinterpret_cast<uintptr_t>(base) | (uint64_t)row) % 128 == 0 || (few && all < (int64_t(32) << 20));
}
template <typename O>
__device__ __forceinline__ void store_all8(O* p, const float (&v)[8], bool past) {
  if (past) {
    asm volatile("");                    // without these the compiler makes one plain store of the two
    store8<O, true>(p, v, 8, 8);
    asm volatile("");
  } else {
    store8<O, false>(p, v, 8, 8);
  }
}

// Statistics of one token per lane over the group's channels, fewer than 8 tokens, a workgroup of 256: 32
// channel lanes of 8 token lanes, in two sweeps.  lds: 5 * 8 * 4 floats.
template <typename T>
__device__ __forceinline__ void norm_short_stats(const NormParams& p, const T* x, bool on, float& mu, float& k, float* lds) {
  float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (!p.rms) {
    for (int64_t c = threadIdx.x / 8; c < p.Dg && on; c += 32) v[0] += get1(x + c * p.L);
    group_sum<8, 4, 256>(v, lds);
    v[0] *= p.inv_dg;
  }
  mu = v[0];
  v[0] = 0.0f;
  for (int64_t c = threadIdx.x / 8; c < p.Dg && on; c += 32) {
    const float d = get1(x + c * p.L) - mu;
    v[0] = __builtin_fmaf(d, d, v[0]);
  }
  v[1] = v[2] = v[3] = 0.0f;
  group_sum<8, 4, 256>(v, lds);
  k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
}

// Statistics of one token-major row, a workgroup of 256.
template <typename T>
__device__ __forceinline__ void norm_row_stats(const NormParams& p, const T* x, float& mu, float& k, float* lds) {
  float v[1] = {0.0f};
  if (!p.rms) {
    for (int64_t c = threadIdx.x; c < p.Dg; c += 256) v[0] += get1(x + c);
    team_sum<1, true, true>(v, 256, lds);
    v[0] *= p.inv_dg;
  }
  mu = v[0];
  v[0] = 0.0f;
  for (int64_t c = threadIdx.x; c < p.Dg; c += 256) {
    const float d = get1(x + c) - mu;
    v[0] = __builtin_fmaf(d, d, v[0]);
  }
  team_sum<1, true, true>(v, 256, lds);
  k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
}

}  // namespace mamba
