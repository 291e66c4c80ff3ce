// layer_norm.hip -- the layer norm over channels and its gradients (gfx950).
//
// Per token and group of Dg channels: xh = (x - mean) k, k = 1 / sqrt(var + eps) (rms: mean = 0 and the
// mean of x^2), m = xh w + b, y = m silu(z).  With dm = dy silu(z) and g = dm w:
//     dx = k (g - mean(g) - xh mean(g xh))  (rms: without mean(g)),  dz = dy m sigma (1 + z (1 - sigma)),
//     dw = sum over tokens of dm xh,  db = sum of dm.
//
// Two forms.  Channel-major (L > 1): channels are L apart, so a thread takes 8 consecutive tokens
// of a channel (one load) and neighbouring lanes the tokens after them; the sums run over the channel
// lanes of a workgroup.  Token-major (L = 1): a row's channels lie together, and a thread takes 8 of
// them.  One read of each input and one write of each output is what HBM has to carry.
#include "glr.hpp"

namespace mamba {
namespace {

// Sums of kN numbers over the lanes of a workgroup that share threadIdx.x % kT, in every lane.
// lds: waves * kT * kN floats.
template <int kT, int kN>
__device__ __forceinline__ void group_sum(float (&v)[kN], float* lds) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int m = kT; m < 64; m *= 2) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] += __shfl_xor(v[j], m);
  }
  if (waves == 1) return;
  __syncthreads();                       // an earlier sum may still be read
  if (lane < kT) {
#pragma unroll
    for (int j = 0; j < kN; ++j) lds[(wave * kT + lane) * kN + j] = v[j];
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kN; ++j) v[j] = 0.0f;
  for (int w = 0; w < waves; ++w) {
#pragma unroll
    for (int j = 0; j < kN; ++j) v[j] += lds[(w * kT + lane % kT) * kN + j];
  }
}

// 1 / sqrt(v), the hardware's root with one Newton step (about half an ulp): it goes into every
// number of the token.
__device__ __forceinline__ float norm_root(float v) {
  const float r = __builtin_amdgcn_rsqf(v);
  const float h = __builtin_fmaf(-0.5f * v * r, r, 1.5f);
  return r * (v < 1e37f && v > 1e-37f ? h : 1.0f);
}

constexpr int kLanes = 8;                // token lanes: 64 tokens, 128 bytes of bf16

// Statistics of 8 tokens over the group's channels, in two sweeps.
template <typename T>
__device__ __forceinline__ void col_stats(const NormParams& p, const T* x, int live, float (&mu)[8], float (&k)[8],
                                          float* lds) {
  const int64_t c0 = threadIdx.x / kLanes, step = blockDim.x / kLanes;
#pragma unroll
  for (int j = 0; j < 8; ++j) mu[j] = k[j] = 0.0f;
  if (!p.rms) {
    for (int64_t c = c0; c < p.Dg; c += step) {
      const Raw8<T> r = load_raw8(x + c * p.L, live);
#pragma unroll
      for (int j = 0; j < 8; ++j) mu[j] += get8(r, j);
    }
    group_sum<kLanes, 8>(mu, lds);
#pragma unroll
    for (int j = 0; j < 8; ++j) mu[j] *= p.inv_dg;
  }
  for (int64_t c = c0; c < p.Dg; c += step) {
    const Raw8<T> r = load_raw8(x + c * p.L, live);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = get8(r, j) - mu[j];
      k[j] = __builtin_fmaf(v, v, k[j]);
    }
  }
  group_sum<kLanes, 8>(k, lds);
#pragma unroll
  for (int j = 0; j < 8; ++j) k[j] = norm_root(__builtin_fmaf(k[j], p.inv_dg, p.eps));
}

template <typename T, typename O>
__global__ __launch_bounds__(256) void norm_col_fwd_kernel(NormParams p) {
  __shared__ float lds[4 * kLanes * 8];
  const int64_t tiles = (p.L + 8 * kLanes - 1) / (8 * kLanes);
  const int64_t bg = blockIdx.x / tiles, tile = blockIdx.x - bg * tiles;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int64_t t = tile * (8 * kLanes) + (threadIdx.x % kLanes) * 8;
  const int live = clamp8(p.L - t);
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  O* y = static_cast<O*>(p.y) + (b * p.D + ch) * p.L + t;
  float mu[8], k[8];
  col_stats(p, x, live, mu, k, lds);
  for (int64_t c = threadIdx.x / kLanes; c < p.Dg; c += blockDim.x / kLanes) {
    const Raw8<T> r = load_raw8(x + c * p.L, live);
    const float w = p.weight ? p.weight[ch + c] : 1.0f, bias = p.bias ? p.bias[ch + c] : 0.0f;
    float o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf((get8(r, j) - mu[j]) * k[j], w, bias);
    if (z) {
      const Raw8<T> zr = load_raw8(z + c * p.L, live);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr, j));
    }
    store8(y + c * p.L, o, live, live);
  }
}

// A workgroup takes every parts-th tile and keeps its sums of dweight and dbias in its part of p.part.
template <typename T, typename Gr>
__global__ __launch_bounds__(256) void norm_col_bwd_kernel(NormParams p) {
  __shared__ float lds[4 * kLanes * 16];
  const int64_t tiles = (p.L + 8 * kLanes - 1) / (8 * kLanes);
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  float* sums = p.part + part * 2 * p.D + ch;
  bool first = true;
  for (int64_t i = part; i < p.B * tiles; i += p.parts, first = false) {
    const int64_t b = i / tiles, t = (i - b * tiles) * (8 * kLanes) + (threadIdx.x % kLanes) * 8;
    const int live = clamp8(p.L - t);
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
    const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
    const int64_t at = (b * p.D + ch) * p.L + t;
    const Gr* dy = static_cast<const Gr*>(p.dy) + at;
    float mu[8], k[8], sg[16];
    col_stats(p, x, live, mu, k, lds);
#pragma unroll
    for (int j = 0; j < 16; ++j) sg[j] = 0.0f;
    for (int64_t c = threadIdx.x / kLanes; c < p.Dg; c += blockDim.x / kLanes) {
      const Raw8<T> r = load_raw8(x + c * p.L, live);
      const Raw8<Gr> dr = load_raw8(dy + c * p.L, live);
      const float w = p.weight ? p.weight[ch + c] : 1.0f;
      float g[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = get8(dr, j) * w;
      if (z) {
        const Raw8<T> zr = load_raw8(z + c * p.L, live);
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= silu(get8(zr, j));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sg[j] += g[j];
        sg[8 + j] = __builtin_fmaf(g[j], (get8(r, j) - mu[j]) * k[j], sg[8 + j]);
      }
    }
    group_sum<kLanes, 16>(sg, lds);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sg[j] = p.rms ? 0.0f : sg[j] * p.inv_dg;
      sg[8 + j] *= p.inv_dg;
    }
    for (int64_t c = threadIdx.x / kLanes; c < p.Dg; c += blockDim.x / kLanes) {
      const Raw8<T> r = load_raw8(x + c * p.L, live);
      const Raw8<Gr> dr = load_raw8(dy + c * p.L, live);
      const float w = p.weight ? p.weight[ch + c] : 1.0f, bias = p.bias ? p.bias[ch + c] : 0.0f;
      float dm[8], o[8], sw = 0.0f, sb = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) dm[j] = get8(dr, j);
      if (z) {
        const Raw8<T> zr = load_raw8(z + c * p.L, live);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float zj = get8(zr, j), s = sigmoid(zj);
          o[j] = dm[j] * __builtin_fmaf((get8(r, j) - mu[j]) * k[j], w, bias) * s * __builtin_fmaf(zj, 1.0f - s, 1.0f);
          dm[j] *= zj * s;
        }
        store8(static_cast<Gr*>(p.dz) + at + c * p.L, o, live, live);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float xh = (get8(r, j) - mu[j]) * k[j];
        o[j] = k[j] * (dm[j] * w - sg[j] - xh * sg[8 + j]);
        if (j < live) {
          sw = __builtin_fmaf(dm[j], xh, sw);
          sb += dm[j];
        }
      }
      store8(static_cast<Gr*>(p.dx) + at + c * p.L, o, live, live);
#pragma unroll
      for (int m = 1; m < kLanes; m *= 2) {
        sw += __shfl_xor(sw, m);
        sb += __shfl_xor(sb, m);
      }
      if (threadIdx.x % kLanes == 0) {
        sums[c] = first ? sw : sums[c] + sw;
        sums[p.D + c] = first ? sb : sums[p.D + c] + sb;
      }
    }
  }
}

// Token-major: a workgroup per row and group.
template <typename T>
__device__ __forceinline__ void row_stats(const NormParams& p, const T* x, float& mu, float& k, float* lds) {
  float v[1] = {0.0f};
  if (!p.rms) {
    for (int64_t c = threadIdx.x; c < p.Dg; c += blockDim.x) v[0] += get1(x + c);
    group_sum<1, 1>(v, lds);
    v[0] *= p.inv_dg;
  }
  mu = v[0];
  v[0] = 0.0f;
  for (int64_t c = threadIdx.x; c < p.Dg; c += blockDim.x) {
    const float d = get1(x + c) - mu;
    v[0] = __builtin_fmaf(d, d, v[0]);
  }
  group_sum<1, 1>(v, lds);
  k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
}

template <typename T, typename O>
__global__ __launch_bounds__(256) void norm_row_fwd_kernel(NormParams p) {
  __shared__ float lds[4];
  const int64_t b = blockIdx.x / p.G, ch = (blockIdx.x - b * p.G) * p.Dg;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch : nullptr;
  O* y = static_cast<O*>(p.y) + b * p.D + ch;
  float mu, k;
  row_stats(p, x, mu, k, lds);
  for (int64_t c = threadIdx.x; c < p.Dg; c += blockDim.x) {
    float o = __builtin_fmaf((get1(x + c) - mu) * k, p.weight ? p.weight[ch + c] : 1.0f, p.bias ? p.bias[ch + c] : 0.0f);
    if (z) o *= silu(get1(z + c));
    put1(y + c, o);
  }
}

template <typename T, typename Gr>
__global__ __launch_bounds__(256) void norm_row_bwd_kernel(NormParams p) {
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
    row_stats(p, x, mu, k, lds);
    for (int64_t c = threadIdx.x; c < p.Dg; c += blockDim.x) {
      float g = get1(dy + c) * (p.weight ? p.weight[ch + c] : 1.0f);
      if (z) g *= silu(get1(z + c));
      sg[0] += g;
      sg[1] = __builtin_fmaf(g, (get1(x + c) - mu) * k, sg[1]);
    }
    group_sum<1, 2>(sg, lds);
    sg[0] = p.rms ? 0.0f : sg[0] * p.inv_dg;
    sg[1] *= p.inv_dg;
    for (int64_t c = threadIdx.x; c < p.Dg; c += blockDim.x) {
      const float w = p.weight ? p.weight[ch + c] : 1.0f, xh = (get1(x + c) - mu) * k;
      float dm = get1(dy + c);
      if (z) {
        const float zj = get1(z + c), s = sigmoid(zj);
        put1(static_cast<Gr*>(p.dz) + at + c, dm * __builtin_fmaf(xh, w, p.bias ? p.bias[ch + c] : 0.0f) * s *
                                                   __builtin_fmaf(zj, 1.0f - s, 1.0f));
        dm *= zj * s;
      }
      put1(static_cast<Gr*>(p.dx) + at + c, k * (dm * w - sg[0] - xh * sg[1]));
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

template <typename T, typename O>
hipError_t fwd_t(const NormParams& p, hipStream_t s) {
  if (p.L == 1) {
    hipLaunchKernelGGL((norm_row_fwd_kernel<T, O>), dim3((unsigned)(p.B * p.G)), dim3(256), 0, s, p);
  } else {
    const int64_t tiles = (p.L + 8 * kLanes - 1) / (8 * kLanes);
    hipLaunchKernelGGL((norm_col_fwd_kernel<T, O>), dim3((unsigned)(p.B * p.G * tiles)), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

template <typename T, typename Gr>
hipError_t bwd_t(const NormParams& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.parts * p.G));
  if (p.L == 1) hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr>), grid, dim3(256), 0, s, p);
  else hipLaunchKernelGGL((norm_col_bwd_kernel<T, Gr>), grid, dim3(256), 0, s, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((2 * p.D + 31) / 32)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_fwd(const NormParams& p, Dt in, Dt out, hipStream_t s) {
  if (in == Dt::BF16) return out == Dt::BF16 ? fwd_t<uint16_t, uint16_t>(p, s) : fwd_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? fwd_t<float, uint16_t>(p, s) : fwd_t<float, float>(p, s);
}

hipError_t launch_norm_bwd(const NormParams& p, Dt in, Dt grad, hipStream_t s) {
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, s) : bwd_t<uint16_t, float>(p, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, s) : bwd_t<float, float>(p, s);
}

}  // namespace mamba
