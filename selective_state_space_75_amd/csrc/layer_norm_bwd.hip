// layer_norm_bwd.hip -- gradients of the layer norm over channels (gfx950).
//
// With xh = (x - mean) k, m = xh w + b, y = m silu(z), dm = dy silu(z) and g = dm w, per token:
//     dx = k (g - mean(g) - xh mean(g xh))   (rms: without mean(g)),   dz = dy m sigma (1 + z (1 - sigma))
// and over tokens dw = sum dm xh, db = sum dm.  The sums of g, g (x - mean) and (x - mean)^2 are taken in one
// sweep once the mean is known.  The tile of x and dy stays in registers (z is read again from the caches);
// the layouts are those of layer_norm.hip.  A workgroup takes every parts-th tile and keeps its channels' sums
// of dw and db on the chip, so that one partial sum per workgroup and channel is written, and one
// small launch adds those up in a fixed order.
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

template <typename T, typename Gr, bool kGate, int kThreads, int kT, int kC>
__global__ __launch_bounds__(kThreads) void norm_col_bwd_kernel(NormParams p) {
  constexpr int kCL = kThreads / kT;
  __shared__ float lds[(kThreads / 64 + 1) * kT * 24];
  extern __shared__ float channel[];                     // weight, sums of dw and db, (gate) bias of the group
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int64_t g = id / p.parts, part = id - g * p.parts, ch = g * p.Dg;
  const int Dg = (int)p.Dg, c0 = threadIdx.x / kT;
  for (int c = threadIdx.x; c < Dg; c += kThreads) {
    channel[c] = p.weight ? p.weight[ch + c] : 1.0f;
    channel[Dg + c] = channel[2 * Dg + c] = 0.0f;
    if constexpr (kGate) channel[3 * Dg + c] = p.bias ? p.bias[ch + c] : 0.0f;
  }
  __syncthreads();
  for (int64_t i = part; i < p.B * p.tiles; i += p.parts) {
    const int64_t b = i / p.tiles, t0 = (i - b * p.tiles) * (8 * kT) + (threadIdx.x % kT) * 8;
    // The last lane takes the row's last 8 tokens whole; the first `dup` of them are the lane's before it.
    const bool on = t0 < p.L;
    const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
    const int dup = on ? (int)(t0 - t) : 8;
    const uint32_t at = (uint32_t)(c0 * p.L + t);
    int64_t step = kCL * p.L;
    asm("" : "+s"(step));                                // its multiples are not worth registers across sweeps
    const int64_t row = (b * p.D + ch) * p.L;
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L;
    const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L : nullptr;
    const Gr* dy = static_cast<const Gr*>(p.dy) + row;
    Gr* dx = static_cast<Gr*>(p.dx) + row;
    Gr* dz = kGate ? static_cast<Gr*>(p.dz) + row : nullptr;
    Raw8<T> r[kC];
    Raw8<Gr> dr[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      if (c0 + k * kCL < Dg) {
        r[k] = load_all8(lane_at(x + k * step, at));
        dr[k] = load_all8(lane_at(dy + k * step, at));
      }
    }
    float mu[8], v[24];
#pragma unroll
    for (int j = 0; j < 8; ++j) mu[j] = 0.0f;
#pragma unroll
    for (int j = 0; j < 24; ++j) v[j] = 0.0f;
    if (!p.rms) {
#pragma unroll
      for (int k = 0; k < kC; ++k) {
        if (c0 + k * kCL < Dg) {
#pragma unroll
          for (int j = 0; j < 8; ++j) mu[j] += get8(r[k], j);
        }
      }
      group_sum<kT, 8, kThreads>(mu, lds);
#pragma unroll
      for (int j = 0; j < 8; ++j) mu[j] *= p.inv_dg;
    }
#pragma unroll
    for (int k = 0; k < kC; ++k)
      if (k * kCL < Dg) keep(r[k]);
    asm("" : "+s"(step));
    constexpr int kBatch = kGate ? 2 : 4;                // loads of z under way at a time
#pragma unroll
    for (int kk = 0; kk < kC; kk += kBatch) {
      if (kk * kCL >= Dg) continue;
      Raw8<T> zr[kBatch];
      if constexpr (kGate) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
          if (c0 + (kk + q) * kCL < Dg) zr[q] = load_all8(lane_at(z + (kk + q) * step, at));
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        if (c0 + (kk + q) * kCL < Dg) {
          const float w = channel[c0 + (kk + q) * kCL];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float d = get8(r[kk + q], j) - mu[j];
            float gj = get8(dr[kk + q], j) * w;
            if constexpr (kGate) gj *= silu(get8(zr[q], j));
            v[j] = __builtin_fmaf(d, d, v[j]);
            v[8 + j] += gj;
            v[16 + j] = __builtin_fmaf(gj, d, v[16 + j]);
          }
        }
      }
    }
    group_sum<kT, 24, kThreads>(v, lds);
    // v[j] becomes k, v[8 + j] mean(g), v[16 + j] mean(g xh)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = norm_root(__builtin_fmaf(v[j], p.inv_dg, p.eps));
      v[8 + j] = p.rms ? 0.0f : v[8 + j] * p.inv_dg;
      v[16 + j] *= v[j] * p.inv_dg;
    }
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      if (k * kCL < Dg) {
        keep(r[k]);
        keep(dr[k]);
      }
    }
    asm("" : "+s"(step));
#pragma unroll
    for (int kk = 0; kk < kC; kk += kBatch) {
      if (kk * kCL >= Dg) continue;
      Raw8<T> zr[kBatch];
      if constexpr (kGate) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q)
          if (c0 + (kk + q) * kCL < Dg) zr[q] = load_all8(lane_at(z + (kk + q) * step, at));
      }
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const int c = c0 + (kk + q) * kCL;
        if (c < Dg) {
          const float w = channel[c];
          float o[8], dm[8], sw = 0.0f, sb = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) dm[j] = get8(dr[kk + q], j);
          if constexpr (kGate) {
            const float bias = channel[3 * Dg + c];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float zj = get8(zr[q], j), s = sigmoid(zj), xh = (get8(r[kk + q], j) - mu[j]) * v[j];
              o[j] = dm[j] * __builtin_fmaf(xh, w, bias) * s * __builtin_fmaf(zj, 1.0f - s, 1.0f);
              dm[j] *= zj * s;
            }
            if (on) store8(lane_at(dz + (kk + q) * step, at), o, 8, 8);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (get8(r[kk + q], j) - mu[j]) * v[j];
            o[j] = v[j] * (__builtin_fmaf(dm[j], w, -v[8 + j]) - xh * v[16 + j]);
            const float one = j < dup ? 0.0f : dm[j];
            sw = __builtin_fmaf(one, j < dup ? 0.0f : xh, sw);
            sb += one;
          }
          if (on) store8(lane_at(dx + (kk + q) * step, at), o, 8, 8);
          sw = lane_sum<kT>(sw);
          sb = lane_sum<kT>(sb);
          if (threadIdx.x % kT == 0) {                   // this lane's alone
            channel[Dg + c] += sw;
            channel[2 * Dg + c] += sb;
          }
        }
      }
    }
  }
  float* sums = p.part + part * 2 * p.D + ch;
  __syncthreads();
  for (int c = threadIdx.x; c < Dg; c += kThreads) {
    sums[c] = channel[Dg + c];
    sums[p.D + c] = channel[2 * Dg + c];
  }
}

// Statistics of kNormColTwo: a workgroup takes 64 tokens of `chunk` channels of the group, one read of x, dy
// and z.  A thread sums around its first channel's value, which is one of the numbers summed, so that
// the difference of squares loses at most its count of channels (32) in units of 2^-24; threads
// are then brought to the workgroup's mean.
template <typename T, typename Gr, bool kGate>
__global__ __launch_bounds__(kNormStatThreads) void norm_stat_kernel(NormParams p) {
  constexpr int kT = kNormStatLanes, kCL = kNormStatThreads / kT, kBatch = kGate ? 2 : 4;
  __shared__ float lds[(kNormStatThreads / 64 + 1) * kT * 24];
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int64_t piece = id / p.tiles, tile = id - piece * p.tiles;        // piece: (b, group, chunk)
  const int64_t bg = piece / p.chunks, c_lo = (piece - bg * p.chunks) * p.chunk;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int64_t c_hi = c_lo + p.chunk < p.Dg ? c_lo + p.chunk : p.Dg;
  const int64_t t0 = tile * (8 * kT) + (threadIdx.x % kT) * 8;
  const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  const Gr* dy = static_cast<const Gr*>(p.dy) + (b * p.D + ch) * p.L + t;
  float s[8], s1[8], v[24];
#pragma unroll
  for (int j = 0; j < 8; ++j) s[j] = s1[j] = 0.0f;
#pragma unroll
  for (int j = 0; j < 24; ++j) v[j] = 0.0f;
  int n = 0;
  for (int64_t c = c_lo + threadIdx.x / kT; c < c_hi; c += kBatch * kCL) {
    Raw8<T> r[kBatch], zr[kBatch];
    Raw8<Gr> dr[kBatch];
    float w[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t cq = c + q * kCL < c_hi ? c + q * kCL : c;            // a channel that is there, not counted below
      r[q] = load_all8(x + cq * p.L);
      dr[q] = load_all8(dy + cq * p.L);
      if constexpr (kGate) zr[q] = load_all8(z + cq * p.L);
      w[q] = p.weight ? p.weight[ch + cq] : 1.0f;
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
          float g = get8(dr[q], j) * w[q];
          if constexpr (kGate) g *= silu(get8(zr[q], j));
          s1[j] += d;
          v[j] = __builtin_fmaf(d, d, v[j]);
          v[8 + j] += g;
          v[16 + j] = __builtin_fmaf(g, d, v[16 + j]);
        }
      }
    }
  }
  float mean[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mean[j] = 0.0f;
  if (!p.rms) {
    const float count = (float)n, inv = n ? 1.0f / count : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) mean[j] = __builtin_fmaf(count, s[j], s1[j]);
    group_sum<kT, 8, kNormStatThreads>(mean, lds);
    const float all = 1.0f / (float)(c_hi - c_lo);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      mean[j] *= all;
      const float m = s1[j] * inv, d = (s[j] - mean[j]) + m;              // the thread's mean around s, and around the mean
      v[j] = __builtin_fmaf(count * d, d, __builtin_fmaf(-s1[j], m, v[j]));
      v[16 + j] = __builtin_fmaf(v[8 + j], s[j] - mean[j], v[16 + j]);
    }
  }
  group_sum<kT, 24, kNormStatThreads>(v, lds);
  if (threadIdx.x >= kT || t0 >= p.L) return;
  float* o = p.stat + piece * 4 * p.L + t;
  float part[8];
  store8<float, false>(o, mean, 8, 8);
#pragma unroll
  for (int q = 0; q < 3; ++q) {
#pragma unroll
    for (int j = 0; j < 8; ++j) part[j] = v[8 * q + j];
    store8<float, false>(o + (q + 1) * p.L, part, 8, 8);
  }
}

// Results of kNormColTwo: 8 kT tokens of apply_chans channels.  The group's statistics come together from
// its pieces once per workgroup; a lane then holds those of its 8 tokens and goes through channels.
template <typename T, typename Gr, bool kGate, int kT>
__global__ __launch_bounds__(kNormApplyThreads) void norm_apply_kernel(NormParams p) {
  constexpr int kCL = kNormApplyThreads / kT, kBatch = 2;
  __shared__ float lds[4][8 * kT];
  const int64_t slabs = (p.Dg + p.apply_chans - 1) / p.apply_chans, tiles = (p.L + 8 * kT - 1) / (8 * kT);
  // Backwards through what norm_stat_kernel read last, which the caches still hold.
  const int64_t id = gridDim.x - 1 - (int64_t)blockIdx.x;
  const int64_t cols = id / tiles, tile = id - cols * tiles;              // cols: (b, group, slab)
  const int64_t bg = cols / slabs, c_lo = (cols - bg * slabs) * p.apply_chans;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int64_t c_hi = c_lo + p.apply_chans < p.Dg ? c_lo + p.apply_chans : p.Dg;
  const int64_t base = tile * (8 * kT) < p.L - 8 ? tile * (8 * kT) : p.L - 8;
  if (threadIdx.x < 8 * kT && base + threadIdx.x < p.L) {
    const float* st = p.stat + bg * p.chunks * 4 * p.L + base + threadIdx.x;
    float mu = 0.0f, m2 = 0.0f, sg = 0.0f, sx = 0.0f;
    if (!p.rms) {
      for (int64_t k = 0; k < p.chunks; ++k) {
        const int64_t n = p.chunk * (k + 1) < p.Dg ? p.chunk : p.Dg - p.chunk * k;
        mu = __builtin_fmaf((float)n, st[k * 4 * p.L], mu);
      }
      mu *= p.inv_dg;
    }
    for (int64_t k = 0; k < p.chunks; ++k) {
      const int64_t n = p.chunk * (k + 1) < p.Dg ? p.chunk : p.Dg - p.chunk * k;
      const float d = st[k * 4 * p.L] - mu, g = st[(k * 4 + 2) * p.L];
      m2 += __builtin_fmaf((float)n * d, d, st[(k * 4 + 1) * p.L]);
      sg += g;
      sx += __builtin_fmaf(g, d, st[(k * 4 + 3) * p.L]);
    }
    const float k = norm_root(__builtin_fmaf(m2, p.inv_dg, p.eps));
    lds[0][threadIdx.x] = mu;
    lds[1][threadIdx.x] = k;
    lds[2][threadIdx.x] = p.rms ? 0.0f : sg * p.inv_dg;
    lds[3][threadIdx.x] = sx * k * p.inv_dg;
  }
  __syncthreads();
  const int64_t t0 = tile * (8 * kT) + (threadIdx.x % kT) * 8;
  // The last lane takes the row's last 8 tokens whole; the first `dup` of them are the lane's before it.
  const bool on = t0 < p.L;
  const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
  const int dup = on ? (int)(t0 - t) : 8;
  float mu[8], k[8], mg[8], mx[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int at = (int)(t - base) + j;
    mu[j] = lds[0][at];
    k[j] = lds[1][at];
    mg[j] = lds[2][at];
    mx[j] = lds[3][at];
  }
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  const int64_t row = (b * p.D + ch) * p.L + t;
  const Gr* dy = static_cast<const Gr*>(p.dy) + row;
  Gr* dx = static_cast<Gr*>(p.dx) + row;
  Gr* dz = kGate ? static_cast<Gr*>(p.dz) + row : nullptr;
  float* sums = p.part + (b * tiles + tile) * 2 * p.D + ch;
  for (int64_t c = c_lo + threadIdx.x / kT; c < c_hi; c += kBatch * kCL) {
    Raw8<T> r[kBatch], zr[kBatch];
    Raw8<Gr> dr[kBatch];
    float w[kBatch], bias[kBatch];
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t cq = c + q * kCL < c_hi ? c + q * kCL : c;
      r[q] = load_all8(x + cq * p.L);
      dr[q] = load_all8(dy + cq * p.L);
      if constexpr (kGate) {
        zr[q] = load_all8(z + cq * p.L);
        bias[q] = p.bias ? p.bias[ch + cq] : 0.0f;
      }
      w[q] = p.weight ? p.weight[ch + cq] : 1.0f;
    }
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int64_t cq = c + q * kCL;
      if (cq >= c_hi) continue;
      float o[8], dm[8], sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dm[j] = get8(dr[q], j);
      if constexpr (kGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float zj = get8(zr[q], j), s = sigmoid(zj), xh = (get8(r[q], j) - mu[j]) * k[j];
          o[j] = dm[j] * __builtin_fmaf(xh, w[q], bias[q]) * s * __builtin_fmaf(zj, 1.0f - s, 1.0f);
          dm[j] *= zj * s;
        }
        if (on) store8(dz + cq * p.L, o, 8, 8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (get8(r[q], j) - mu[j]) * k[j];
        o[j] = k[j] * (__builtin_fmaf(dm[j], w[q], -mg[j]) - xh * mx[j]);
        const float one = j < dup ? 0.0f : dm[j];
        sw = __builtin_fmaf(one, j < dup ? 0.0f : xh, sw);
        sb += one;
      }
      if (on) store8(dx + cq * p.L, o, 8, 8);
      if constexpr (kT == 64) {
        sw = wave_sum63(sw);
        sb = wave_sum63(sb);
        if (threadIdx.x % 64 == 63) {
          sums[cq] = sw;
          sums[p.D + cq] = sb;
        }
      } else {
        sw = lane_sum<kT>(sw);
        sb = lane_sum<kT>(sb);
        if (threadIdx.x % kT == 0) {
          sums[cq] = sw;
          sums[p.D + cq] = sb;
        }
      }
    }
  }
}

// Any group, fewer than 8 tokens: four sweeps over every tile; the sums of dw and db live in their part in memory.
template <typename T, typename Gr, int kTok>
__global__ __launch_bounds__(256) void norm_col_long_bwd_kernel(NormParams p) {
  __shared__ float lds[5 * 8 * 16];
  const int64_t g = blockIdx.x / p.parts, part = blockIdx.x - g * p.parts, ch = g * p.Dg;
  float* sums = p.part + part * 2 * p.D + ch;
  bool first = true;
  for (int64_t i = part; i < p.B * p.tiles; i += p.parts, first = false) {
    const int64_t b = i / p.tiles, t = ((i - b * p.tiles) * 8 + threadIdx.x % 8) * kTok;
    const int live = kTok == 8 ? clamp8(p.L - t) : t < p.L ? 1 : 0;
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
    const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
    const int64_t at = (b * p.D + ch) * p.L + t;
    const Gr* dy = static_cast<const Gr*>(p.dy) + at;
    float mu[8], k[8], sg[16];
    norm_col_stats<T, kTok>(p, x, live, mu, k, lds);
#pragma unroll
    for (int j = 0; j < 16; ++j) sg[j] = 0.0f;
    for (int64_t c = threadIdx.x / 8; c < p.Dg; c += 32) {
      const float w = p.weight ? p.weight[ch + c] : 1.0f;
      float xv[kTok], gv[kTok];
      load_tok<T, kTok>(x + c * p.L, live, xv);
      load_tok<Gr, kTok>(dy + c * p.L, live, gv);
      if (z) {
        float zv[kTok];
        load_tok<T, kTok>(z + c * p.L, live, zv);
#pragma unroll
        for (int j = 0; j < kTok; ++j) gv[j] *= silu(zv[j]);
      }
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        sg[j] = __builtin_fmaf(gv[j], w, sg[j]);
        sg[8 + j] = __builtin_fmaf(gv[j] * w, (xv[j] - mu[j]) * k[j], sg[8 + j]);
      }
    }
    group_sum<8, 16, 256>(sg, lds);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sg[j] = p.rms ? 0.0f : sg[j] * p.inv_dg;
      sg[8 + j] *= p.inv_dg;
    }
    for (int64_t c = threadIdx.x / 8; c < p.Dg; c += 32) {
      const float w = p.weight ? p.weight[ch + c] : 1.0f, bias = p.bias ? p.bias[ch + c] : 0.0f;
      float xv[kTok], dm[kTok], o[8], sw = 0.0f, sb = 0.0f;
      load_tok<T, kTok>(x + c * p.L, live, xv);
      load_tok<Gr, kTok>(dy + c * p.L, live, dm);
#pragma unroll
      for (int j = 0; j < kTok; ++j) xv[j] = (xv[j] - mu[j]) * k[j];
      if (z) {
        float zv[kTok];
        load_tok<T, kTok>(z + c * p.L, live, zv);
#pragma unroll
        for (int j = 0; j < kTok; ++j) {
          const float s = sigmoid(zv[j]);
          o[j] = dm[j] * __builtin_fmaf(xv[j], w, bias) * s * __builtin_fmaf(zv[j], 1.0f - s, 1.0f);
          dm[j] *= zv[j] * s;
        }
        store_tok<Gr, kTok>(static_cast<Gr*>(p.dz) + at + c * p.L, live, o);
      }
#pragma unroll
      for (int j = 0; j < kTok; ++j) {
        o[j] = k[j] * (__builtin_fmaf(dm[j], w, -sg[j]) - xv[j] * sg[8 + j]);
        if (j < live) {
          sw = __builtin_fmaf(dm[j], xv[j], sw);
          sb += dm[j];
        }
      }
      store_tok<Gr, kTok>(static_cast<Gr*>(p.dx) + at + c * p.L, live, o);
#pragma unroll
      for (int m = 1; m < 8; m *= 2) {
        sw += __shfl_xor(sw, m);
        sb += __shfl_xor(sb, m);
      }
      if (threadIdx.x % 8 == 0) {
        sums[c] = first ? sw : sums[c] + sw;
        sums[p.D + c] = first ? sb : sums[p.D + c] + sb;
      }
    }
  }
}

// Token-major: a team of lanes, or a workgroup, takes every parts-th token of a group; 8 channels a thread,
// the last thread the group's last 8 whole (see norm_row_fwd_kernel).
template <typename T, typename Gr, bool kBlock>
__global__ __launch_bounds__(kBlock ? 1024 : 256) void norm_row_bwd_kernel(NormParams p) {
  __shared__ float lds[3 * 16];
  const int team = p.team;
  const int64_t id = kBlock ? blockIdx.x : (int64_t)blockIdx.x * (256 / team) + threadIdx.x / team;
  const int at = (kBlock ? threadIdx.x : threadIdx.x % team) * 8, Dg = (int)p.Dg;
  const int64_t part = id / p.G, ch = (id - part * p.G) * p.Dg;
  const bool on = at < Dg && part < p.parts;
  const int c = at < Dg - 8 ? at : Dg - 8, dup = on ? at - c : 8;
  Raw8<float> wr, br;
  if (p.weight) wr = load_all8(p.weight + ch + c);
  if (p.bias) br = load_all8(p.bias + ch + c);
  float sw[8], sb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sw[j] = sb[j] = 0.0f;
  for (int64_t b = part; b < p.B; b += p.parts) {
    const Raw8<T> r = load_all8(static_cast<const T*>(p.x) + b * p.x_stride + ch + c);
    const Raw8<Gr> dr = load_all8(static_cast<const Gr*>(p.dy) + b * p.D + ch + c);
    Raw8<T> zr;
    if (p.z) zr = load_all8(static_cast<const T*>(p.z) + b * p.z_stride + ch + c);
    float mu[1] = {0.0f}, v[3] = {0.0f, 0.0f, 0.0f};
    if (!p.rms) {
#pragma unroll
      for (int j = 0; j < 8; ++j) mu[0] += j < dup ? 0.0f : get8(r, j);
      team_sum<1, kBlock>(mu, team, lds);
      mu[0] *= p.inv_dg;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = get8(r, j) - mu[0];
      float g = get8(dr, j) * (p.weight ? get8(wr, j) : 1.0f);
      if (p.z) g *= silu(get8(zr, j));
      if (j >= dup) {
        v[0] = __builtin_fmaf(d, d, v[0]);
        v[1] += g;
        v[2] = __builtin_fmaf(g, d, v[2]);
      }
    }
    team_sum<3, kBlock>(v, team, lds);
    const float k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
    const float mg = p.rms ? 0.0f : v[1] * p.inv_dg, mx = v[2] * k * p.inv_dg;
    float o[8], dm[8], xh[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dm[j] = get8(dr, j);
      xh[j] = (get8(r, j) - mu[0]) * k;
    }
    const int64_t out = b * p.D + ch + c;
    if (p.z) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float zj = get8(zr, j), s = sigmoid(zj);
        o[j] = dm[j] * __builtin_fmaf(xh[j], p.weight ? get8(wr, j) : 1.0f, p.bias ? get8(br, j) : 0.0f) * s *
               __builtin_fmaf(zj, 1.0f - s, 1.0f);
        dm[j] *= zj * s;
      }
      if (on) store8(static_cast<Gr*>(p.dz) + out, o, 8, 8);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j] = k * (__builtin_fmaf(dm[j], p.weight ? get8(wr, j) : 1.0f, -mg) - xh[j] * mx);
      sw[j] = __builtin_fmaf(dm[j], xh[j], sw[j]);
      sb[j] += dm[j];
    }
    if (on) store8(static_cast<Gr*>(p.dx) + out, o, 8, 8);
  }
  if (!on) return;
  // channels that two threads have: both hold the same sums
  float* sums = p.part + part * 2 * p.D + ch + c;
  store8<float, false>(sums, sw, 8, 8);
  store8<float, false>(sums + p.D, sb, 8, 8);
}

// Token-major, any group.
template <typename T, typename Gr>
__global__ __launch_bounds__(256) void norm_row_long_bwd_kernel(NormParams p) {
  __shared__ float lds[8];
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  float* sums = p.part + part * 2 * p.D + ch;
  bool first = true;
  for (int64_t b = part; b < p.B; b += p.parts, first = false) {
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch;
    const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch : nullptr;
    const int64_t at = b * p.D + ch;
    const Gr* dy = static_cast<const Gr*>(p.dy) + at;
    float mu, k, sg[2] = {0.0f, 0.0f};
    norm_row_stats(p, x, mu, k, lds);
    for (int64_t c = threadIdx.x; c < p.Dg; c += 256) {
      float g = get1(dy + c) * (p.weight ? p.weight[ch + c] : 1.0f);
      if (z) g *= silu(get1(z + c));
      sg[0] += g;
      sg[1] = __builtin_fmaf(g, (get1(x + c) - mu) * k, sg[1]);
    }
    team_sum<2, true>(sg, 256, lds);
    sg[0] = p.rms ? 0.0f : sg[0] * p.inv_dg;
    sg[1] *= p.inv_dg;
    for (int64_t c = threadIdx.x; c < p.Dg; c += 256) {
      const float w = p.weight ? p.weight[ch + c] : 1.0f, xh = (get1(x + c) - mu) * k;
      float dm = get1(dy + c);
      if (z) {
        const float zj = get1(z + c), s = sigmoid(zj);
        put1(static_cast<Gr*>(p.dz) + at + c, dm * __builtin_fmaf(xh, w, p.bias ? p.bias[ch + c] : 0.0f) * s *
                                                   __builtin_fmaf(zj, 1.0f - s, 1.0f));
        dm *= zj * s;
      }
      put1(static_cast<Gr*>(p.dx) + at + c, k * (__builtin_fmaf(dm, w, -sg[0]) - xh * sg[1]));
      sums[c] = first ? dm * xh : __builtin_fmaf(dm, xh, sums[c]);
      sums[p.D + c] = first ? dm : sums[p.D + c] + dm;
    }
  }
}

// dweight and dbias from their parts: 32 channels x 8 parts at a time per workgroup.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormParams p) {
  __shared__ float half[8][32];
  const int64_t n = 2 * p.D, c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const int y = threadIdx.x >> 5;
  float o = 0.0f;
  if (c < n)
    for (int64_t i = y; i < p.parts; i += 8) o += p.part[i * n + c];
  half[y][threadIdx.x & 31] = o;
  __syncthreads();
  if (y || c >= n) return;
  for (int w = 1; w < 8; ++w) o += half[w][threadIdx.x];
  if (c < p.D) p.dweight[c] = o;
  else p.dbias[c - p.D] = o;
}

template <typename T, typename Gr, int kI>
hipError_t col_t(const NormParams& p, unsigned grid, hipStream_t s) {
  constexpr NormShape q = kNormBwd[kI];
  const unsigned lds = (unsigned)((p.z ? 4 : 3) * p.Dg * sizeof(float));
  if (p.z)
    hipLaunchKernelGGL((norm_col_bwd_kernel<T, Gr, true, q.threads, q.lanes, q.chans>), dim3(grid), dim3(q.threads), lds, s, p);
  else
    hipLaunchKernelGGL((norm_col_bwd_kernel<T, Gr, false, q.threads, q.lanes, q.chans>), dim3(grid), dim3(q.threads), lds, s, p);
  return hipGetLastError();
}

template <typename T, typename Gr, bool kGate>
hipError_t two_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  hipLaunchKernelGGL((norm_stat_kernel<T, Gr, kGate>), dim3((unsigned)(p.B * p.G * q.chunks * q.tiles)),
                     dim3(kNormStatThreads), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)(q.parts * p.G * ((p.Dg + q.apply_chans - 1) / q.apply_chans)));
  if (q.apply_lanes == 64)
    hipLaunchKernelGGL((norm_apply_kernel<T, Gr, kGate, 64>), grid, dim3(kNormApplyThreads), 0, s, p);
  else
    hipLaunchKernelGGL((norm_apply_kernel<T, Gr, kGate, 8>), grid, dim3(kNormApplyThreads), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename Gr>
hipError_t main_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const unsigned grid = (unsigned)(p.parts * p.G);
  switch (q.kind) {
    case 0: return col_t<T, Gr, 0>(p, grid, s);
    case 1: return col_t<T, Gr, 1>(p, grid, s);
    case kNormColTwo: return p.z ? two_t<T, Gr, true>(p, q, s) : two_t<T, Gr, false>(p, q, s);
    case kNormColLong:
      hipLaunchKernelGGL((norm_col_long_bwd_kernel<T, Gr, 1>), dim3(grid), dim3(256), 0, s, p);
      break;
    case kNormRowTeam:
      hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, false>), dim3((grid + 256 / p.team - 1) / (256 / p.team)), dim3(256),
                         0, s, p);
      break;
    case kNormRowBlock:
      hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, true>), dim3(grid), dim3(q.threads), 0, s, p);
      break;
    default:
      hipLaunchKernelGGL((norm_row_long_bwd_kernel<T, Gr>), dim3(grid), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <typename T, typename Gr>
hipError_t bwd_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const hipError_t e = main_t<T, Gr>(p, q, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((2 * p.D + 31) / 32)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormParams& p, const NormPlan& q, Dt in, Dt grad, hipStream_t s) {
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, q, s) : bwd_t<uint16_t, float>(p, q, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, q, s) : bwd_t<float, float>(p, q, s);
}

}  // namespace mamba
