// layer_norm_bwd.hip -- gradients of the layer norm over channels (gfx950).
//
// With xh = (x - mean) k, m = xh w + b, y = m silu(z), dm = dy silu(z) and g = dm w, per token:
//     dx = k (g - mean(g) - xh mean(g xh))   (rms: without mean(g)),   dz = dy m sigma (1 + z (1 - sigma))
// and over tokens dw = sum dm xh, db = sum dm.  The sums of g, g (x - mean) and (x - mean)^2 are taken in one
// sweep once the mean is known.  What HBM has to carry is one read of x, dy (z) and one write of dx (dz); the
// tile of x and dy stays in registers between the sweeps, z with it where a thread has at most four channels,
// and is read again from the caches otherwise.  The layouts are those of layer_norm.hip.  A workgroup takes every
// parts-th tile and keeps its channels' sums of dw and db on the chip, so that one partial sum per workgroup and
// channel is written; one small launch (norm_sum_kernel, 4 us) adds those up in a fixed order.
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
  const bool past = past_caches(p.dx, p.L * sizeof(Gr), (kGate ? 2 : 1) * p.B * p.D * p.L * sizeof(Gr),
                                kGate || sizeof(Gr) == 2);
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
            if (on) store_all8(lane_at(dz + (kk + q) * step, at), o, past);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float xh = (get8(r[kk + q], j) - mu[j]) * v[j];
            o[j] = v[j] * (__builtin_fmaf(dm[j], w, -v[8 + j]) - xh * v[16 + j]);
            const float one = j < dup ? 0.0f : dm[j];
            sw = __builtin_fmaf(one, j < dup ? 0.0f : xh, sw);
            sb += one;
          }
          if (on) store_all8(lane_at(dx + (kk + q) * step, at), o, past);
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

// Token-major: a workgroup takes a group of channels and every parts-th share of the tokens, one a team at once: of
// lanes, or (kWaves) of as many waves as the group needs.  8 channels a thread, the last thread the group's last 8
// whole (see norm_row_fwd_kernel); kRagged: Dg is no multiple of 8.  A token waits for its loads and then for two sums
// over the team, so the next token's inputs are loaded while one is worked on, where the registers allow (128 of them:
// not z beside 4-byte inputs, none of the gate's four 4-byte streams).  The teams' sums of dw and db are added up
// at the end.  8192 tokens of 5120 channels, bf16: 66 us (HBM 49), gated 110 us (82), fp32 106 us (98); 8192 of
// 512: 14 us, of which the sum over parts is 4.
template <typename T, typename Gr, bool kWaves, bool kRagged, bool kGate>
__global__ __launch_bounds__(1024) void norm_row_bwd_kernel(NormParams p) {
  __shared__ float lds[3 * 16];
  __shared__ float fold[16 * 64 * 8];
  const int team = p.team, teams = blockDim.x / team, own = threadIdx.x / team, lane = threadIdx.x % team;
  const int Dg = (int)p.Dg;
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  const bool on = lane * 8 < Dg;
  const int c = lane * 8 < Dg - 8 ? lane * 8 : Dg - 8, dup = on ? lane * 8 - c : 8;
  float w[8];
  Raw8<float> wr, br;
  if (p.weight) wr = load_all8(p.weight + ch + c);
  if (kGate && p.bias) br = load_all8(p.bias + ch + c);
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = p.weight ? get8(wr, j) : 1.0f;
  float sw[8], sb[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) sw[j] = sb[j] = 0.0f;
  const T* x = static_cast<const T*>(p.x) + ch + c;
  const Gr* dy = static_cast<const Gr*>(p.dy) + ch + c;
  // The teams stay together: one past the last token goes through that one again and leaves it out.
  auto token = [&](int64_t first) { return first + own < p.B ? first + own : p.B - 1; };
  const int64_t stride = p.parts * teams;
  const T* z = kGate ? static_cast<const T*>(p.z) + ch + c : nullptr;
  constexpr bool kAhead = kGate && sizeof(T) == 2;       // z too, where there are registers for it
  Raw8<T> zn;
  if constexpr (kAhead) zn = load_all8(z + token(part * teams) * p.z_stride);
  constexpr bool kNext = !kGate || sizeof(T) + sizeof(Gr) < 8;
  Raw8<T> rn;
  Raw8<Gr> dn;
  if constexpr (kNext) {
    rn = load_all8(x + token(part * teams) * p.x_stride);
    dn = load_all8(dy + token(part * teams) * p.D);
  }
  for (int64_t first = part * teams; first < p.B; first += stride) {
    const bool mine = first + own < p.B;
    const int64_t b = token(first);
    Raw8<T> r = rn, zr;
    Raw8<Gr> dr = dn;
    if constexpr (kAhead) zr = zn;
    else if constexpr (kGate) zr = load_all8(z + b * p.z_stride);
    if constexpr (!kNext) {
      r = load_all8(x + b * p.x_stride);
      dr = load_all8(dy + b * p.D);
    } else if (first + stride < p.B) {
      if constexpr (kAhead) zn = load_all8(z + token(first + stride) * p.z_stride);
      rn = load_all8(x + token(first + stride) * p.x_stride);
      dn = load_all8(dy + token(first + stride) * p.D);
    }
    float mu[1] = {0.0f}, v[3] = {0.0f, 0.0f, 0.0f}, d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = get8(r, j);
    if (!p.rms) {
#pragma unroll
      for (int j = 0; j < 8; ++j) mu[0] += !on || (kRagged && j < dup) ? 0.0f : d[j];
      team_sum<1, kWaves>(mu, team, lds);
      mu[0] *= p.inv_dg;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] -= mu[0];
    }
    if (on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float gj = get8(dr, j) * w[j];
        if constexpr (kGate) gj *= silu(get8(zr, j));
        const float dj = kRagged && j < dup ? 0.0f : d[j];
        if (kRagged && j < dup) gj = 0.0f;
        v[0] = __builtin_fmaf(dj, dj, v[0]);
        v[1] += gj;
        v[2] = __builtin_fmaf(gj, dj, v[2]);
      }
    }
    team_sum<3, kWaves>(v, team, lds);
    // dx = k (g - mean(g) - xh mean(g xh)) with xh = k d
    const float k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
    const float mg = p.rms ? 0.0f : -k * v[1] * p.inv_dg, mx = -k * k * (v[2] * k * p.inv_dg);
    float o[8];
    const int64_t out = b * p.D + ch + c;
    if (on && mine) {
      float dm[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dm[j] = get8(dr, j);
      if constexpr (kGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float zj = get8(zr, j), s = sigmoid(zj);
          o[j] = dm[j] * __builtin_fmaf(d[j] * k, w[j], p.bias ? get8(br, j) : 0.0f) * s * __builtin_fmaf(zj, 1.0f - s, 1.0f);
          dm[j] *= zj * s;
        }
        store8(static_cast<Gr*>(p.dz) + out, o, 8, 8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        o[j] = __builtin_fmaf(d[j], mx, __builtin_fmaf(k, dm[j] * w[j], mg));
        sw[j] = __builtin_fmaf(dm[j], d[j] * k, sw[j]);
        sb[j] += dm[j];
      }
      store8(static_cast<Gr*>(p.dx) + out, o, 8, 8);
    }
  }
  // Teams of a wave first, then a thread of the first team takes the same channels of the others, once for sw and
  // once for sb.
  const int of = kWaves ? team >> 6 : 1, waves = blockDim.x >> 6, at = threadIdx.x & 63;
#pragma unroll
  for (int turn = 0; turn < 2; ++turn) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = turn ? sb[j] : sw[j];
    if constexpr (!kWaves) {
      for (int m = team; m < 64; m *= 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += __shfl_xor(v[j], m);
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) fold[((threadIdx.x >> 6) * 64 + at) * 8 + j] = v[j];
    __syncthreads();
    if (own == 0 && on) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = 0.0f;
      for (int w = threadIdx.x >> 6; w < waves; w += of) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += fold[(w * 64 + at) * 8 + j];
      }
      // channels that two threads have: both hold the same sums
      store8<float, false>(p.part + (part * 2 + turn) * p.D + ch + c, v, 8, 8);
    }
  }
}

// Token-major, groups of 8193 to 16384 channels: a workgroup per token, 2 x 8 channels a thread.  Weights, bias and z
// come from the caches again for each token: the sums of dw and db, x and dy fill the 128 registers, and with the
// gate's work beside them the sums live in LDS, a thread's own 32 numbers (with 4-byte x and z, x comes again too).
// 8192 tokens of 10240 channels, bf16: 143 us (HBM 98), gated 258 us (164).
template <typename T, typename Gr, bool kGate>
__global__ __launch_bounds__(1024) void norm_row_wide_bwd_kernel(NormParams p) {
  __shared__ float lds[3 * 16];
  const int Dg = (int)p.Dg;
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  bool on[2];
  int c[2], dup[2];
  float sw[kGate ? 1 : 2][8], sb[kGate ? 1 : 2][8];
  __shared__ float4 own_sums[kGate ? 8 : 1][kGate ? 1024 : 1];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int own = (threadIdx.x + i * blockDim.x) * 8;
    on[i] = own < Dg;
    c[i] = own < Dg - 8 ? own : Dg - 8;
    dup[i] = on[i] ? own - c[i] : 8;
    if constexpr (kGate) {
#pragma unroll
      for (int q = 0; q < 4; ++q) own_sums[i * 4 + q][threadIdx.x] = float4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) sw[i][j] = sb[i][j] = 0.0f;
    }
  }
  for (int64_t b = part; b < p.B; b += p.parts) {
    const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch;
    const T* z = kGate ? static_cast<const T*>(p.z) + b * p.z_stride + ch : nullptr;
    const int64_t row = b * p.D + ch;
    const float* weight = p.weight ? p.weight + ch : nullptr;
    const float* shift = p.bias ? p.bias + ch : nullptr;
    const Gr* dy = static_cast<const Gr*>(p.dy) + row;
    Raw8<T> r[2];
    Raw8<Gr> dr[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r[i] = load_all8(lane_at(x, c[i]));
      dr[i] = load_all8(lane_at(dy, c[i]));
    }
    float mu[1] = {0.0f}, v[3] = {0.0f, 0.0f, 0.0f};
    if (!p.rms) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) mu[0] += j < dup[i] ? 0.0f : get8(r[i], j);
      team_sum<1, true, true>(mu, blockDim.x, lds);
      mu[0] *= p.inv_dg;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      keep(r[i]);
      keep(dr[i]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      asm("" : "+s"(weight), "+s"(z), "+v"(v[0]));       // loaded piece by piece: not worth registers for longer
      Raw8<float> w;
      Raw8<T> zr;
      if (weight) w = load_all8(lane_at(weight, c[i]));
      if constexpr (kGate) zr = load_all8(lane_at(z, c[i]));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = j < dup[i] ? 0.0f : get8(r[i], j) - mu[0];
        float g = get8(dr[i], j) * (weight ? get8(w, j) : 1.0f);
        if constexpr (kGate) g *= silu(get8(zr, j));
        g = j < dup[i] ? 0.0f : g;
        v[0] = __builtin_fmaf(d, d, v[0]);
        v[1] += g;
        v[2] = __builtin_fmaf(g, d, v[2]);
      }
    }
    team_sum<3, true, true>(v, blockDim.x, lds);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (!kGate || sizeof(T) == 2) keep(r[i]);
      keep(dr[i]);
    }
    const float k = norm_root(__builtin_fmaf(v[0], p.inv_dg, p.eps));
    const float mg = p.rms ? 0.0f : -k * v[1] * p.inv_dg, mx = -k * k * (v[2] * k * p.inv_dg);
    float last = 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      asm("" : "+s"(weight), "+s"(shift), "+s"(z), "+s"(x), "+v"(last));
      if (!on[i]) continue;
      if constexpr (kGate && sizeof(T) == 4) r[i] = load_all8(lane_at(x, c[i]));
      Raw8<float> w;
      if (weight) w = load_all8(lane_at(weight, c[i]));
      float o[8], dm[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) dm[j] = get8(dr[i], j);
      if constexpr (kGate) {
        const Raw8<T> zr = load_all8(lane_at(z, c[i]));
        Raw8<float> bias;
        if (shift) bias = load_all8(lane_at(shift, c[i]));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float zj = get8(zr, j), s = sigmoid(zj), xh = (get8(r[i], j) - mu[0]) * k;
          o[j] = dm[j] * __builtin_fmaf(xh, weight ? get8(w, j) : 1.0f, shift ? get8(bias, j) : 0.0f) * s *
                 __builtin_fmaf(zj, 1.0f - s, 1.0f);
          dm[j] *= zj * s;
        }
        store8(lane_at(static_cast<Gr*>(p.dz) + row, c[i]), o, 8, 8);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = get8(r[i], j) - mu[0];
        o[j] = __builtin_fmaf(d, mx, __builtin_fmaf(k, dm[j] * (weight ? get8(w, j) : 1.0f), mg));
        if constexpr (!kGate) {
          sw[i][j] = __builtin_fmaf(dm[j], d * k, sw[i][j]);
          sb[i][j] += dm[j];
        }
      }
      last = o[7];
      store8(lane_at(static_cast<Gr*>(p.dx) + row, c[i]), o, 8, 8);
      if constexpr (kGate) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4 t = own_sums[i * 4 + q][threadIdx.x];
          float* a = &t.x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int j = (q & 1) * 4 + e;
            a[e] = q < 2 ? __builtin_fmaf(dm[j], (get8(r[i], j) - mu[0]) * k, a[e]) : a[e] + dm[j];
          }
          own_sums[i * 4 + q][threadIdx.x] = t;
        }
      }
    }
  }
  float* sums = p.part + part * 2 * p.D + ch;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!on[i]) continue;                                // channels that two threads have: both hold the same sums
    if constexpr (kGate) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 t = own_sums[i * 4 + q][threadIdx.x];
        (q < 2 ? sw : sb)[0][(q & 1) * 4] = t.x;
        (q < 2 ? sw : sb)[0][(q & 1) * 4 + 1] = t.y;
        (q < 2 ? sw : sb)[0][(q & 1) * 4 + 2] = t.z;
        (q < 2 ? sw : sb)[0][(q & 1) * 4 + 3] = t.w;
      }
    }
    store8<float, false>(sums + c[i], sw[kGate ? 0 : i], 8, 8);
    store8<float, false>(sums + p.D + c[i], sb[kGate ? 0 : i], 8, 8);
  }
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
    team_sum<2, true, true>(sg, 256, lds);
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

// dweight and dbias from their parts: 64 channels x 16 shares of the parts per workgroup.
__global__ __launch_bounds__(1024) void norm_sum_kernel(NormParams p) {
  __shared__ float share[16][64];
  const int64_t n = 2 * p.D, c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int y = threadIdx.x >> 6;
  float o = 0.0f;
  if (c < n) o = strided_sum(p.part + c, n, y, p.parts);
  share[y][threadIdx.x & 63] = o;
  __syncthreads();
  if (y || c >= n) return;
#pragma unroll
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

template <typename T, typename Gr, bool kWaves>
hipError_t row_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const dim3 grid((unsigned)(p.parts * p.G)), block(q.threads);
  if (p.Dg % 8) {
    if (p.z) hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, kWaves, true, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, kWaves, true, false>), grid, block, 0, s, p);
  } else {
    if (p.z) hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, kWaves, false, true>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((norm_row_bwd_kernel<T, Gr, kWaves, false, false>), grid, block, 0, s, p);
  }
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
    case kNormRowTeam: return row_t<T, Gr, false>(p, q, s);
    case kNormRowBlock: return row_t<T, Gr, true>(p, q, s);
    case kNormRowWide:
      if (p.z) hipLaunchKernelGGL((norm_row_wide_bwd_kernel<T, Gr, true>), dim3(grid), dim3(q.threads), 0, s, p);
      else hipLaunchKernelGGL((norm_row_wide_bwd_kernel<T, Gr, false>), dim3(grid), dim3(q.threads), 0, s, p);
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
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((2 * p.D + 63) / 64)), dim3(1024), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_bwd(const NormParams& p, const NormPlan& q, Dt in, Dt grad, hipStream_t s) {
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, q, s) : bwd_t<uint16_t, float>(p, q, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, q, s) : bwd_t<float, float>(p, q, s);
}

}  // namespace mamba
