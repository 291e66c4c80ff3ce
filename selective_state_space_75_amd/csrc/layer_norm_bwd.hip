// layer_norm_bwd.hip -- gradients of the layer norm over channels (gfx950).
//
// With xh = (x - mean) k, m = xh w + b, y = m silu(z), dm = dy silu(z) and g = dm w, per token:
//     dx = k (g - mean(g) - xh mean(g xh))   (rms: without mean(g)),   dz = dy m sigma (1 + z (1 - sigma))
// and over tokens dw = sum dm xh, db = sum dm.  The sums of g, g (x - mean) and (x - mean)^2 are taken in one
// sweep once the mean is known.  The tile of x and dy stays in registers (z is read again from the caches);
// the layouts are those of layer_norm.hip.  A workgroup takes every parts-th tile and keeps its channels' sums
// of dw and db on the chip, so that one partial sum per workgroup and channel is written, and one
// small launch adds those up in a fixed order.
#include "layer_norm_two.hpp"

namespace mamba {
namespace {

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
    constexpr bool kHold = kGate && kC <= 4;             // z stays too
    Raw8<T> r[kC], zh[kHold ? kC : 1];
    Raw8<Gr> dr[kC];
#pragma unroll
    for (int k = 0; k < kC; ++k) {
      if (c0 + k * kCL < Dg) {
        r[k] = load_all8(lane_at(x + k * step, at));
        dr[k] = load_all8(lane_at(dy + k * step, at));
        if constexpr (kHold) zh[k] = load_all8(lane_at(z + k * step, at));
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
    constexpr int kBatch = kGate || kC < 4 ? 2 : 4;      // loads of z under way at a time
#pragma unroll
    for (int kk = 0; kk < kC; kk += kBatch) {
      if (kk * kCL >= Dg) continue;
      Raw8<T> zr[kBatch];
      if constexpr (kGate) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if constexpr (kHold) zr[q] = zh[kk + q];
          else if (c0 + (kk + q) * kCL < Dg) zr[q] = load_all8(lane_at(z + (kk + q) * step, at));
        }
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
        if constexpr (kHold) keep(zh[k]);
      }
    }
    asm("" : "+s"(step));
#pragma unroll
    for (int kk = 0; kk < kC; kk += kBatch) {
      if (kk * kCL >= Dg) continue;
      Raw8<T> zr[kBatch];
      if constexpr (kGate) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
          if constexpr (kHold) zr[q] = zh[kk + q];
          else if (c0 + (kk + q) * kCL < Dg) zr[q] = load_all8(lane_at(z + (kk + q) * step, at));
        }
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

// Fewer than 8 tokens: a token a lane, 8 token lanes, four sweeps over the group; the sums of dw and db live in
// their part in memory.
template <typename T, typename Gr>
__global__ __launch_bounds__(256) void norm_col_long_bwd_kernel(NormParams p) {
  __shared__ float lds[5 * 8 * 4];
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  const int t = threadIdx.x % 8;
  const bool on = t < p.L;
  float* sums = p.part + part * 2 * p.D + ch;
  bool first = true;
  for (int64_t b = part; b < p.B; b += p.parts, first = false) {
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
    const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
    const int64_t at = (b * p.D + ch) * p.L + t;
    const Gr* dy = static_cast<const Gr*>(p.dy) + at;
    float mu, k, sg[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    norm_short_stats(p, x, on, mu, k, lds);
    for (int64_t c = threadIdx.x / 8; c < p.Dg && on; c += 32) {
      float g = get1(dy + c * p.L) * (p.weight ? p.weight[ch + c] : 1.0f);
      if (z) g *= silu(get1(z + c * p.L));
      sg[0] += g;
      sg[1] = __builtin_fmaf(g, (get1(x + c * p.L) - mu) * k, sg[1]);
    }
    group_sum<8, 4, 256>(sg, lds);
    sg[0] = p.rms ? 0.0f : sg[0] * p.inv_dg;
    sg[1] *= p.inv_dg;
    for (int64_t c = threadIdx.x / 8; c < p.Dg; c += 32) {
      float sw = 0.0f, sb = 0.0f;
      if (on) {
        const float w = p.weight ? p.weight[ch + c] : 1.0f, xh = (get1(x + c * p.L) - mu) * k;
        float dm = get1(dy + c * p.L);
        if (z) {
          const float zj = get1(z + c * p.L), s = sigmoid(zj);
          put1(static_cast<Gr*>(p.dz) + at + c * p.L, dm * __builtin_fmaf(xh, w, p.bias ? p.bias[ch + c] : 0.0f) * s *
                                                          __builtin_fmaf(zj, 1.0f - s, 1.0f));
          dm *= zj * s;
        }
        put1(static_cast<Gr*>(p.dx) + at + c * p.L, k * (__builtin_fmaf(dm, w, -sg[0]) - xh * sg[1]));
        sw = dm * xh;
        sb = dm;
      }
      sw = lane_sum<8>(sw);
      sb = lane_sum<8>(sb);
      if (t == 0) {
        sums[c] = first ? sw : sums[c] + sw;
        sums[p.D + c] = first ? sb : sums[p.D + c] + sb;
      }
    }
  }
}

// Token-major: a workgroup takes a group of channels and every parts-th share of the tokens, one a team of lanes
// (or one at a time) at once; 8 channels a thread, the last thread the group's last 8 whole (see
// norm_row_fwd_kernel).  Its teams' sums of dw and db are added up at the end.
template <typename T, typename Gr, bool kBlock>
__global__ __launch_bounds__(kBlock ? 1024 : 256) void norm_row_bwd_kernel(NormParams p) {
  __shared__ float lds[kBlock ? 3 * 16 : 4 * 64 * 16];
  const int team = p.team, teams = kBlock ? 1 : 256 / team, own = kBlock ? 0 : threadIdx.x / team;
  const int at = (kBlock ? threadIdx.x : threadIdx.x % team) * 8, Dg = (int)p.Dg;
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  const bool on = at < Dg;
  const int c = at < Dg - 8 ? at : Dg - 8, dup = on ? at - c : 8;
  Raw8<float> wr, br;
  if (p.weight) wr = load_all8(p.weight + ch + c);
  if (p.bias) br = load_all8(p.bias + ch + c);
  float sw[8], sb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sw[j] = sb[j] = 0.0f;
  // A wave's lanes stay together: a team past the last token goes through that one again and leaves it out.
  for (int64_t first = part * teams; first < p.B; first += p.parts * teams) {
    const bool mine = first + own < p.B;
    const int64_t b = mine ? first + own : p.B - 1;
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
      if (on && mine) store8(static_cast<Gr*>(p.dz) + out, o, 8, 8);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j] = k * (__builtin_fmaf(dm[j], p.weight ? get8(wr, j) : 1.0f, -mg) - xh[j] * mx);
      if (mine) {
        sw[j] = __builtin_fmaf(dm[j], xh[j], sw[j]);
        sb[j] += dm[j];
      }
    }
    if (on && mine) store8(static_cast<Gr*>(p.dx) + out, o, 8, 8);
  }
  if constexpr (!kBlock) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int m = team; m < 64; m *= 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sw[j] += __shfl_xor(sw[j], m);
        sb[j] += __shfl_xor(sb[j], m);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      lds[(wave * 64 + lane) * 16 + j] = sw[j];
      lds[(wave * 64 + lane) * 16 + 8 + j] = sb[j];
    }
    __syncthreads();
    if (own) return;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sw[j] = sb[j] = 0.0f;
      for (int w = 0; w < 4; ++w) {
        sw[j] += lds[(w * 64 + lane) * 16 + j];
        sb[j] += lds[(w * 64 + lane) * 16 + 8 + j];
      }
    }
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

// dweight and dbias from their parts: 16 channels x 16 shares of them per workgroup, four loads under way.
__global__ __launch_bounds__(256) void norm_sum_kernel(NormParams p) {
  __shared__ float share[16][16];
  const int64_t n = 2 * p.D, c = (int64_t)blockIdx.x * 16 + (threadIdx.x & 15);
  const int y = threadIdx.x >> 4;
  float o = 0.0f;
  if (c < n) o = strided_sum(p.part + c, n, y, p.parts);
  share[y][threadIdx.x & 15] = o;
  __syncthreads();
  if (y || c >= n) return;
  for (int w = 1; w < 16; ++w) o += share[w][threadIdx.x];
  if (c < p.D) p.dweight[c] = o;
  else p.dbias[c - p.D] = o;
}

template <typename T, typename Gr, int kI>
hipError_t col_t(const NormParams& p, unsigned grid, hipStream_t s) {
  constexpr NormShape q = sizeof(T) + sizeof(Gr) == 4 ? kNormBwd2[kI] : kNormBwd4[kI];
  const unsigned lds = (unsigned)((p.z ? 4 : 3) * p.Dg * sizeof(float));
  if (p.z)
    hipLaunchKernelGGL((norm_col_bwd_kernel<T, Gr, true, q.threads, q.lanes, q.chans>), dim3(grid), dim3(q.threads), lds, s, p);
  else
    hipLaunchKernelGGL((norm_col_bwd_kernel<T, Gr, false, q.threads, q.lanes, q.chans>), dim3(grid), dim3(q.threads), lds, s, p);
  return hipGetLastError();
}

template <typename T, typename Gr>
hipError_t main_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const unsigned grid = (unsigned)(p.parts * p.G);
  switch (q.kind) {
    case 0: return col_t<T, Gr, 0>(p, grid, s);
    case 1: return col_t<T, Gr, 1>(p, grid, s);
    case 2: return col_t<T, Gr, 2>(p, grid, s);
    case kNormColTwo: return p.z ? norm_two<T, Gr, true, true>(p, q, s) : norm_two<T, Gr, true, false>(p, q, s);
    case kNormColLong:
      hipLaunchKernelGGL((norm_col_long_bwd_kernel<T, Gr>), dim3(grid), dim3(256), 0, s, p);
      break;
    case kNormRowTeam:
      hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, false>), dim3(grid), dim3(256), 0, s, p);
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
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((2 * p.D + 15) / 16)), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormParams& p, const NormPlan& q, Dt in, Dt grad, hipStream_t s) {
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, q, s) : bwd_t<uint16_t, float>(p, q, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, q, s) : bwd_t<float, float>(p, q, s);
}

}  // namespace mamba
