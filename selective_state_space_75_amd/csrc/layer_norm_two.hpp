// layer_norm_two.hpp -- the layer norm of channel-major groups in two launches (gfx950): statistics of every
// token, then results.  Both go through the activations in whole cache lines (64 tokens, or 512) with every
// CU at work, whatever the group's size; what the second reads again comes from the last-level cache while the
// activations fit there.  (A tile held on the chip between the sweeps is read once, but a group of 5120
// channels leaves room for 16 tokens backward, 32 bytes of a line: 134 us at 4 x 2048 tokens, bf16, where the two
// launches and the sum of the weight's parts take 81, 33 + 44 + 4.)
#pragma once

#include "layer_norm.hpp"

namespace mamba {
namespace {

// Sum over the kT lanes of a token team, in its first lane.
template <int kT>
__device__ __forceinline__ float lane_sum(float x) {
  if constexpr (kT >= 8) x += dpp<0x104, 0xf>(0.0f, x);
  if constexpr (kT >= 4) x += dpp<0x102, 0xf>(0.0f, x);
  if constexpr (kT >= 2) x += dpp<0x101, 0xf>(0.0f, x);
  return x;
}

// Statistics of kNormColTwo: a workgroup takes 64 tokens of `chunk` channels of the group, one read of x (and,
// backward, dy and z).  A thread sums around its first channel's value, which is one of the numbers summed, so that
// the difference of squares loses at most its count of channels (40) in units of 2^-24; threads
// are then brought to the workgroup's mean.
template <typename T, typename Gr, bool kBwd, bool kGate>
__global__ __launch_bounds__(kNormStatThreads) void norm_stat_kernel(NormParams p) {
  constexpr int kT = kNormStatLanes, kCL = kNormStatThreads / kT, kBatch = kBwd ? 2 : 4, kSums = kBwd ? 24 : 8;
  __shared__ float lds[(kNormStatThreads / 64 + 1) * kT * kSums];
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int64_t piece = id / p.tiles, tile = id - piece * p.tiles;        // piece: (b, group, chunk)
  const int64_t bg = piece / p.chunks, c_lo = (piece - bg * p.chunks) * p.chunk;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int64_t c_hi = c_lo + p.chunk < p.Dg ? c_lo + p.chunk : p.Dg;
  const int64_t t0 = tile * (8 * kT) + (threadIdx.x % kT) * 8;
  const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  const Gr* dy = kBwd ? static_cast<const Gr*>(p.dy) + (b * p.D + ch) * p.L + t : nullptr;
  float s[8], s1[8], v[kSums];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = s1[j] = 0.0f;
#pragma unroll
  for (int j = 0; j < kSums; ++j) v[j] = 0.0f;
  int n = 0;
  for (int64_t c = c_lo + threadIdx.x / kT; c < c_hi; c += kBatch * kCL) {
    Raw8<T> r[kBatch], zr[kBatch];
    Raw8<Gr> dr[kBatch];
    float w[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t cq = c + q * kCL < c_hi ? c + q * kCL : c;            // a channel that is there, not counted below
      r[q] = load_all8(x + cq * p.L);
      if constexpr (kBwd) {
        dr[q] = load_all8(dy + cq * p.L);
        w[q] = p.weight ? p.weight[ch + cq] : 1.0f;
      }
      if constexpr (kGate) zr[q] = load_all8(z + cq * p.L);
    }
    if (n == 0 && !p.rms) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = get8(r[0], j);
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      if (c + q * kCL < c_hi) {
        ++n;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float d = get8(r[q], j) - s[j];
          s1[j] += d;
          v[j] = __builtin_fmaf(d, d, v[j]);
          if constexpr (kBwd) {
            float g = get8(dr[q], j) * w[q];
            if constexpr (kGate) g *= silu(get8(zr[q], j));
            v[8 + j] += g;
            v[16 + j] = __builtin_fmaf(g, d, v[16 + j]);
          }
        }
      }
    }
  }
  float mean[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mean[j] = 0.0f;
  if (!p.rms) {
    // The mean is summed from the first channel's value on, so that an offset of all channels costs it nothing.
    const Raw8<T> from = load_all8(x + c_lo * p.L);
    const float count = (float)n, inv = n ? 1.0f / count : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mean[j] = __builtin_fmaf(count, n ? s[j] - get8(from, j) : 0.0f, s1[j]);
    group_sum<kT, 8, kNormStatThreads>(mean, lds);
    const float all = 1.0f / (float)(c_hi - c_lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mean[j] = __builtin_fmaf(mean[j], all, get8(from, j));
      const float m = s1[j] * inv, d = (s[j] - mean[j]) + m;              // the thread's mean around s, and around the mean
      v[j] = __builtin_fmaf(count * d, d, __builtin_fmaf(-s1[j], m, v[j]));
      if constexpr (kBwd) v[16 + j] = __builtin_fmaf(v[8 + j], s[j] - mean[j], v[16 + j]);
    }
  }
  group_sum<kT, kSums, kNormStatThreads>(v, lds);
  if (threadIdx.x >= kT || t0 >= p.L) return;
  float* o = p.stat + piece * (1 + kSums / 8) * p.L + t;
  float part[8];
  store8<float, false>(o, mean, 8, 8);
#pragma unroll
  for (int q = 0; q < kSums / 8; ++q) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = v[8 * q + j];
    store8<float, false>(o + (q + 1) * p.L, part, 8, 8);
  }
}

// Results of kNormColTwo: 8 kT tokens of apply_chans channels.  The group's statistics come together from
// its pieces once per workgroup; a lane then holds those of its 8 tokens and goes through channels.
template <typename T, typename Gr, bool kBwd, bool kGate, int kT>
__global__ __launch_bounds__(kNormApplyThreads) void norm_apply_kernel(NormParams p) {
  constexpr int kCL = kNormApplyThreads / kT, kQ = kBwd ? 4 : 2;      // numbers of a piece's statistics
  __shared__ float lds[kBwd ? 4 : 2][8 * kT];
  const int64_t slabs = (p.Dg + p.apply_chans - 1) / p.apply_chans, tiles = (p.L + 8 * kT - 1) / (8 * kT);
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int64_t cols = id / tiles, tile = id - cols * tiles;              // cols: (b, group, slab)
  const int64_t bg = cols / slabs, c_lo = (cols - bg * slabs) * p.apply_chans;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int64_t c_hi = c_lo + p.apply_chans < p.Dg ? c_lo + p.apply_chans : p.Dg;
  const int64_t base = tile * (8 * kT) < p.L - 8 ? tile * (8 * kT) : p.L - 8;
  const int64_t t0 = tile * (8 * kT) + (threadIdx.x % kT) * 8;
  // The last lane takes the row's last 8 tokens whole; the first `dup` of them are the lane's before it.
  const bool on = t0 < p.L;
  const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
  const int dup = on ? (int)(t0 - t) : 8;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  const int64_t row = (b * p.D + ch) * p.L + t;
  const Gr* dy = kBwd ? static_cast<const Gr*>(p.dy) + row : nullptr;
  Gr* out = static_cast<Gr*>(kBwd ? p.dx : p.y) + row;
  Gr* dz = kBwd && kGate ? static_cast<Gr*>(p.dz) + row : nullptr;
  float* sums = kBwd ? p.part + (b * tiles + tile) * 2 * p.D + ch : nullptr;
  // The channel to come is loaded while the one at hand is worked on, the first of them before the statistics.
  Raw8<T> rn, zn;
  Raw8<Gr> dn;
  float wn, bn = 0.0f;
  auto load = [&](int64_t c) {
    const int64_t cq = c < c_hi ? c : c_hi - 1;
    rn = load_all8(x + cq * p.L);
    if constexpr (kBwd) dn = load_all8(dy + cq * p.L);
    if constexpr (kGate) zn = load_all8(z + cq * p.L);
    if constexpr (kGate || !kBwd) bn = p.bias ? p.bias[ch + cq] : 0.0f;
    wn = p.weight ? p.weight[ch + cq] : 1.0f;
  };
  load(c_lo + threadIdx.x / kT);
  if (threadIdx.x < 8 * kT && base + threadIdx.x < p.L) {
    const float* st = p.stat + bg * p.chunks * kQ * p.L + base + threadIdx.x;
    float mu = 0.0f, m2 = 0.0f, sg = 0.0f, sx = 0.0f;
    if (!p.rms) {
      const float from = st[0];
#pragma unroll 4
      for (int64_t k = 1; k < p.chunks; ++k) {
        const int64_t n = p.chunk * (k + 1) < p.Dg ? p.chunk : p.Dg - p.chunk * k;
        mu = __builtin_fmaf((float)n, st[k * kQ * p.L] - from, mu);
      }
      mu = __builtin_fmaf(mu, p.inv_dg, from);
    }
#pragma unroll 4
    for (int64_t k = 0; k < p.chunks; ++k) {
      const int64_t n = p.chunk * (k + 1) < p.Dg ? p.chunk : p.Dg - p.chunk * k;
      const float d = st[k * kQ * p.L] - mu;
      m2 += __builtin_fmaf((float)n * d, d, st[(k * kQ + 1) * p.L]);
      if constexpr (kBwd) {
        const float g = st[(k * kQ + 2) * p.L];
        sg += g;
        sx += __builtin_fmaf(g, d, st[(k * kQ + 3) * p.L]);
      }
    }
    const float k = norm_root(__builtin_fmaf(m2, p.inv_dg, p.eps));
    lds[0][threadIdx.x] = mu;
    lds[1][threadIdx.x] = k;
    if constexpr (kBwd) {
      lds[2][threadIdx.x] = p.rms ? 0.0f : sg * p.inv_dg;
      lds[3][threadIdx.x] = sx * k * p.inv_dg;
    }
  }
  __syncthreads();
  float mu[8], k[8], mg[8], mx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = (int)(t - base) + j;
    mu[j] = lds[0][at];
    k[j] = lds[1][at];
    if constexpr (kBwd) {
      mg[j] = lds[2][at];
      mx[j] = lds[3][at];
    }
  }
  for (int64_t c = c_lo + threadIdx.x / kT; c < c_hi; c += kCL) {
    const Raw8<T> r = rn, zr = zn;
    const Raw8<Gr> dr = dn;
    const float w = wn, bias = bn;
    load(c + kCL);
    float o[8];
    if constexpr (!kBwd) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = __builtin_fmaf((get8(r, j) - mu[j]) * k[j], w, bias);
        if constexpr (kGate) o[j] *= silu(get8(zr, j));
      }
      if (on) store8(out + c * p.L, o, 8, 8);
    } else {
      float dm[8], sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dm[j] = get8(dr, j);
      if constexpr (kGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float zj = get8(zr, j), s = sigmoid(zj), xh = (get8(r, j) - mu[j]) * k[j];
          o[j] = dm[j] * __builtin_fmaf(xh, w, bias) * s * __builtin_fmaf(zj, 1.0f - s, 1.0f);
          dm[j] *= zj * s;
        }
        if (on) store8(dz + c * p.L, o, 8, 8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (get8(r, j) - mu[j]) * k[j];
        o[j] = k[j] * (__builtin_fmaf(dm[j], w, -mg[j]) - xh * mx[j]);
        const float one = j < dup ? 0.0f : dm[j];
        sw = __builtin_fmaf(one, j < dup ? 0.0f : xh, sw);
        sb += one;
      }
      if (on) store8(out + c * p.L, o, 8, 8);
      sw = kT == 64 ? wave_sum63(sw) : lane_sum<kT>(sw);
      sb = kT == 64 ? wave_sum63(sb) : lane_sum<kT>(sb);
      if (threadIdx.x % kT == (kT == 64 ? 63 : 0)) {
        sums[c] = sw;
        sums[p.D + c] = sb;
      }
    }
  }
}

// The forward statistics do not know the output's type.
template <bool kBwd, typename T, typename Gr>
struct NormStatType { using type = Gr; };
template <typename T, typename Gr>
struct NormStatType<false, T, Gr> { using type = T; };

template <typename T, typename Gr, bool kBwd, bool kGate>
hipError_t norm_two(const NormParams& p, const NormPlan& q, hipStream_t s) {
  hipLaunchKernelGGL((norm_stat_kernel<T, typename NormStatType<kBwd, T, Gr>::type, kBwd, kBwd && kGate>), dim3((unsigned)(p.B * p.G * q.chunks * q.tiles)),
                     dim3(kNormStatThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t tiles = (p.L + 8 * q.apply_lanes - 1) / (8 * q.apply_lanes);
  const dim3 grid((unsigned)(p.B * tiles * p.G * ((p.Dg + q.apply_chans - 1) / q.apply_chans)));
  if (q.apply_lanes == 64)
    hipLaunchKernelGGL((norm_apply_kernel<T, Gr, kBwd, kGate, 64>), grid, dim3(kNormApplyThreads), 0, s, p);
  else
    hipLaunchKernelGGL((norm_apply_kernel<T, Gr, kBwd, kGate, 8>), grid, dim3(kNormApplyThreads), 0, s, p);
  return hipGetLastError();
}

}  // namespace
}  // namespace mamba
