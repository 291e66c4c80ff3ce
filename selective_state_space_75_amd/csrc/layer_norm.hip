// layer_norm.hip -- the layer norm over channels, forward (gfx950), and the plan of both passes.
//
// Per token and group of Dg channels: xh = (x - mean) k, k = 1 / sqrt(var + eps) (rms: mean = 0 and the
// mean of x^2), y = (xh w + b) silu(z).  One read of x (and z) and one write of y is what HBM has to
// carry, so the tile stays on the chip between the sweeps for the mean, the variance and the result.
//
// Channel-major (L > 1): channels are L apart, so a thread takes 8 consecutive tokens (one load) of every
// CL-th channel, neighbouring lanes the tokens after them, and the sums run over a workgroup's CL channel
// lanes.  Groups too large for that go through layer_norm_two.hpp.  Token-major (L = 1): a row's channels lie
// together; a thread takes 8 of them.
// bf16: 4 x 5120 channels in 40 groups, L = 2048: 30 us, 8192 token-major rows of 5120: 33 us (HBM: 33); in one
// group, channel-major: 43 us in two launches.  128 rows of 5120 channels: 4 us on the GPU, one token's latency.
#include "layer_norm_two.hpp"

namespace mamba {
namespace {

template <typename T, typename O, int kThreads, int kT, int kC>
__global__ __launch_bounds__(kThreads) void norm_col_fwd_kernel(NormParams p) {
  constexpr int kCL = kThreads / kT;
  __shared__ float lds[(kThreads / 64 + 1) * kT * 8];
  extern __shared__ float affine[];                      // weight, bias of the group
  const int64_t id = by_xcd(blockIdx.x, gridDim.x);
  const int64_t bg = id / p.tiles, tile = id - bg * p.tiles;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int Dg = (int)p.Dg, c0 = threadIdx.x / kT;
  // The last lane of a row takes its last 8 tokens whole: those that the lane before it has too come out
  // of the same sums, with the same bits.
  const int64_t t0 = tile * (8 * kT) + (threadIdx.x % kT) * 8;
  const bool on = t0 < p.L;
  const int64_t t = t0 < p.L - 8 ? t0 : p.L - 8;
  const uint32_t at = (uint32_t)(c0 * p.L + t);
  const int64_t step = kCL * p.L;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L : nullptr;
  O* y = static_cast<O*>(p.y) + (b * p.D + ch) * p.L;
  const bool past = past_caches(p.y, p.L * sizeof(O), p.B * p.D * p.L * sizeof(O), sizeof(O) == 2);

  Raw8<T> r[kC];
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    if (c0 + k * kCL < Dg) r[k] = load_all8(lane_at(x + k * step, at));
  }
  for (int c = threadIdx.x; c < Dg; c += kThreads) {
    affine[c] = p.weight ? p.weight[ch + c] : 1.0f;
    affine[Dg + c] = p.bias ? p.bias[ch + c] : 0.0f;
  }
  float mu[8], v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) mu[j] = v[j] = 0.0f;
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
#pragma unroll
  for (int k = 0; k < kC; ++k) {
    if (c0 + k * kCL < Dg) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = get8(r[k], j) - mu[j];
        v[j] = __builtin_fmaf(d, d, v[j]);
      }
    }
  }
  group_sum<kT, 8, kThreads>(v, lds);                    // its barriers also publish `affine`
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = norm_root(__builtin_fmaf(v[j], p.inv_dg, p.eps));
#pragma unroll
  for (int k = 0; k < kC; ++k)
    if (k * kCL < Dg) keep(r[k]);
#pragma unroll
  for (int kk = 0; kk < kC; kk += 4) {
    if (kk * kCL >= Dg) continue;
    Raw8<T> zr[4];
    if (z) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c0 + (kk + i) * kCL < Dg) zr[i] = load_all8(lane_at(z + (kk + i) * step, at));
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = c0 + (kk + i) * kCL;
      if (c < Dg && on) {
        const float w = affine[c], bias = affine[Dg + c];
        float o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf((get8(r[kk + i], j) - mu[j]) * v[j], w, bias);
        if (z) {
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr[i], j));
        }
        store_all8(lane_at(y + (kk + i) * step, at), o, past);
      }
    }
  }
}

// Fewer than 8 tokens: a token a lane, 8 token lanes, three sweeps over the group.
template <typename T, typename O>
__global__ __launch_bounds__(256) void norm_col_long_fwd_kernel(NormParams p) {
  __shared__ float lds[5 * 8 * 4];
  const int64_t b = blockIdx.x / p.G, ch = (blockIdx.x - b * p.G) * p.Dg;
  const int t = threadIdx.x % 8;
  const bool on = t < p.L;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch * p.L + t;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch * p.L + t : nullptr;
  O* y = static_cast<O*>(p.y) + (b * p.D + ch) * p.L + t;
  float mu, k;
  norm_short_stats(p, x, on, mu, k, lds);
  for (int64_t c = threadIdx.x / 8; c < p.Dg && on; c += 32) {
    float o = __builtin_fmaf((get1(x + c * p.L) - mu) * k, p.weight ? p.weight[ch + c] : 1.0f, p.bias ? p.bias[ch + c] : 0.0f);
    if (z) o *= silu(get1(z + c * p.L));
    put1(y + c * p.L, o);
  }
}

// Token-major, groups of up to 512 channels: a team of lanes per token and group, 8 channels a lane.  The last lane
// takes the group's last 8 channels whole; those that the one before it has too (the first `dup` of them) are
// left out of the sums.
template <typename T, typename O>
__global__ __launch_bounds__(256) void norm_row_fwd_kernel(NormParams p) {
  const int team = p.team;
  const int64_t id = (int64_t)blockIdx.x * (256 / team) + threadIdx.x / team;
  const int at = (threadIdx.x % team) * 8, Dg = (int)p.Dg;
  const bool on = at < Dg && id < p.B * p.G;
  const int64_t bg = id < p.B * p.G ? id : 0;
  const int64_t b = bg / p.G, ch = (bg - b * p.G) * p.Dg;
  const int c = at < Dg - 8 ? at : Dg - 8, dup = on ? at - c : 8;
  const Raw8<T> r = load_all8(static_cast<const T*>(p.x) + b * p.x_stride + ch + c);
  Raw8<T> zr;
  Raw8<float> w, bias;
  if (p.z) zr = load_all8(static_cast<const T*>(p.z) + b * p.z_stride + ch + c);
  if (p.weight) w = load_all8(p.weight + ch + c);
  if (p.bias) bias = load_all8(p.bias + ch + c);
  float mu[1] = {0.0f}, k[1] = {0.0f};
  if (!p.rms) {
#pragma unroll
    for (int j = 0; j < 8; ++j) mu[0] += j < dup ? 0.0f : get8(r, j);
    team_sum<1, false>(mu, team, nullptr);
    mu[0] *= p.inv_dg;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = j < dup ? 0.0f : get8(r, j) - mu[0];
    k[0] = __builtin_fmaf(d, d, k[0]);
  }
  team_sum<1, false>(k, team, nullptr);
  k[0] = norm_root(__builtin_fmaf(k[0], p.inv_dg, p.eps));
  if (!on) return;
  float o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    o[j] = __builtin_fmaf((get8(r, j) - mu[0]) * k[0], p.weight ? get8(w, j) : 1.0f, p.bias ? get8(bias, j) : 0.0f);
  if (p.z) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr, j));
  }
  store8(static_cast<O*>(p.y) + b * p.D + ch + c, o, 8, 8);
}

// Token-major, a workgroup of the group's width, kC times 8 channels a thread: it takes every parts-th token, keeps
// the weights (8 bytes a channel, twice what a token's bf16 x and y are), and has the next token's x and z loaded
// while one is worked on (8192 rows of 5120 channels, bf16: 33 us, a workgroup per token 43; of 10240 channels: 65).
// The sums keep team_sum's branch for two waves where there are never so few: it ends the scheduler's block in front
// of the sum, and the loads ahead stay early (79 without it).
template <typename T, typename O, bool kGate, int kC>
__global__ __launch_bounds__(1024) void norm_row_block_fwd_kernel(NormParams p) {
  __shared__ float lds[16];
  const int Dg = (int)p.Dg;
  const int64_t part = blockIdx.x / p.G, ch = (blockIdx.x - part * p.G) * p.Dg;
  const T* x = static_cast<const T*>(p.x) + ch;
  const T* z = kGate ? static_cast<const T*>(p.z) + ch : nullptr;
  O* y = static_cast<O*>(p.y) + ch;
  bool on[kC];
  int c[kC], dup[kC];
  float w[kC][8], bias[kC][8];
  Raw8<T> rn[kC], zn[kC];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int at = (threadIdx.x + i * blockDim.x) * 8;
    on[i] = at < Dg;
    c[i] = at < Dg - 8 ? at : Dg - 8;
    dup[i] = on[i] ? at - c[i] : 8;
    rn[i] = load_all8(x + part * p.x_stride + c[i]);
    if constexpr (kGate) zn[i] = load_all8(z + part * p.z_stride + c[i]);
  }
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    Raw8<float> wr, br;
    if (p.weight) wr = load_all8(p.weight + ch + c[i]);
    if (p.bias) br = load_all8(p.bias + ch + c[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[i][j] = p.weight ? get8(wr, j) : 1.0f;
      bias[i][j] = p.bias ? get8(br, j) : 0.0f;
    }
  }
  for (int64_t b = part; b < p.B; b += p.parts) {
    Raw8<T> r[kC], zr[kC];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      r[i] = rn[i];
      if constexpr (kGate) zr[i] = zn[i];
    }
    if (b + p.parts < p.B) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        rn[i] = load_all8(x + (b + p.parts) * p.x_stride + c[i]);
        if constexpr (kGate) zn[i] = load_all8(z + (b + p.parts) * p.z_stride + c[i]);
      }
    }
    float mu[1] = {0.0f}, k[1] = {0.0f};
    if (!p.rms) {
#pragma unroll
      for (int i = 0; i < kC; ++i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) mu[0] += j < dup[i] ? 0.0f : get8(r[i], j);
      }
      team_sum<1, true>(mu, blockDim.x, lds);
      mu[0] *= p.inv_dg;
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = j < dup[i] ? 0.0f : get8(r[i], j) - mu[0];
        k[0] = __builtin_fmaf(d, d, k[0]);
      }
    }
    team_sum<1, true>(k, blockDim.x, lds);
    k[0] = norm_root(__builtin_fmaf(k[0], p.inv_dg, p.eps));
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      if (!on[i]) continue;
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = __builtin_fmaf((get8(r[i], j) - mu[0]) * k[0], w[i][j], bias[i][j]);
      if constexpr (kGate) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr[i], j));
      }
      store8(y + b * p.D + c[i], o, 8, 8);
    }
  }
}

// Token-major, any group: a workgroup per token and group, three sweeps.
template <typename T, typename O>
__global__ __launch_bounds__(256) void norm_row_long_fwd_kernel(NormParams p) {
  __shared__ float lds[4];
  const int64_t b = blockIdx.x / p.G, ch = (blockIdx.x - b * p.G) * p.Dg;
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + ch;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + ch : nullptr;
  O* y = static_cast<O*>(p.y) + b * p.D + ch;
  float mu, k;
  norm_row_stats(p, x, mu, k, lds);
  for (int64_t c = threadIdx.x; c < p.Dg; c += 256) {
    float o = __builtin_fmaf((get1(x + c) - mu) * k, p.weight ? p.weight[ch + c] : 1.0f, p.bias ? p.bias[ch + c] : 0.0f);
    if (z) o *= silu(get1(z + c));
    put1(y + c, o);
  }
}

template <typename T, typename O, int kI>
hipError_t col_t(const NormParams& p, unsigned grid, hipStream_t s) {
  constexpr NormShape q = sizeof(T) == 2 ? kNormFwd2[kI] : kNormFwd4[kI];
  hipLaunchKernelGGL((norm_col_fwd_kernel<T, O, q.threads, q.lanes, q.chans>), dim3(grid), dim3(q.threads),
                     (unsigned)(2 * p.Dg * sizeof(float)), s, p);
  return hipGetLastError();
}

template <typename T, typename O, int kC>
hipError_t block_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const dim3 grid((unsigned)(p.parts * p.G)), block(q.threads);
  if (p.z) hipLaunchKernelGGL((norm_row_block_fwd_kernel<T, O, true, kC>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((norm_row_block_fwd_kernel<T, O, false, kC>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t fwd_t(const NormParams& p, const NormPlan& q, hipStream_t s) {
  const unsigned items = (unsigned)(p.B * p.G), grid = (unsigned)(p.B * p.G * q.tiles);
  switch (q.kind) {
    case 0: return col_t<T, O, 0>(p, grid, s);
    case 1: return col_t<T, O, 1>(p, grid, s);
    case 2: return col_t<T, O, 2>(p, grid, s);
    case 3: return col_t<T, O, 3>(p, grid, s);
    case kNormColTwo: return p.z ? norm_two<T, O, false, true>(p, q, s) : norm_two<T, O, false, false>(p, q, s);
    case kNormColLong:
      hipLaunchKernelGGL((norm_col_long_fwd_kernel<T, O>), dim3(grid), dim3(256), 0, s, p);
      break;
    case kNormRowTeam:
      hipLaunchKernelGGL((norm_row_fwd_kernel<T, O>), dim3((items + 256 / p.team - 1) / (256 / p.team)), dim3(256), 0, s, p);
      break;
    case kNormRowBlock: return block_t<T, O, 1>(p, q, s);
    case kNormRowWide: return block_t<T, O, 2>(p, q, s);
    default:
      hipLaunchKernelGGL((norm_row_long_fwd_kernel<T, O>), dim3(items), dim3(256), 0, s, p);
  }
  return hipGetLastError();
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

NormPlan norm_plan(int64_t B, int64_t D, int64_t L, int64_t G, int in_width, int grad_width, bool gate) {
  const int64_t Dg = D / G;
  const bool bwd = grad_width != 0;
  NormPlan q{};
  int64_t cu = 4;                                      // workgroups that a CU holds at once
  q.tiles = 1;
  q.threads = 256;
  if (L == 1) {
    q.kind = Dg < 8 || Dg > 16384 ? kNormRowLong : Dg > 8192 ? kNormRowWide : Dg > 512 ? kNormRowBlock : kNormRowTeam;
    q.lanes = 1;                                       // threads of a token
    while (q.kind == kNormRowTeam && q.lanes * 8 < Dg) q.lanes *= 2;
    if (q.kind == kNormRowBlock) q.threads = q.lanes = (int)((Dg + 511) / 512) * 64;
    if (q.kind == kNormRowWide) q.threads = q.lanes = (int)((Dg + 1023) / 1024) * 64;
    if (bwd && q.kind != kNormRowLong) q.threads = 1024 / q.lanes * q.lanes;     // as many teams as that holds
  } else if (L < 8) {
    q.kind = kNormColLong;
    q.lanes = 8;
  } else {
    const NormShape* shapes = bwd ? (in_width + grad_width == 4 ? kNormBwd2 : kNormBwd4) : in_width == 2 ? kNormFwd2 : kNormFwd4;
    q.kind = kNormColTwo;
    for (int i = 0; i < (bwd ? (int)kNormBwdShapes : (int)kNormShapes); ++i) {
      const int64_t lanes = shapes[i].threads / shapes[i].lanes;      // channel lanes
      if (Dg > lanes * shapes[i].chans || L >= (int64_t(1) << 30) / (lanes + 1)) continue;   // 32-bit byte offsets
      q.kind = i;
      cu = gate ? shapes[i].cu_gate : shapes[i].cu;
      q.threads = shapes[i].threads;
      q.lanes = shapes[i].lanes;
      break;
    }
    if (q.kind == kNormColTwo) {
      q.threads = kNormStatThreads;
      q.lanes = kNormStatLanes;
    }
    q.tiles = ceil_div(L, 8 * q.lanes);
  }
  if (q.kind == kNormColTwo) {
    // Statistics: 4 to 40 channels a thread, in as few pieces as give every CU a workgroup.
    const int64_t lanes = kNormStatThreads / kNormStatLanes, blocks = B * G * q.tiles;
    const int64_t least = ceil_div(Dg, 40 * lanes), most = Dg / (4 * lanes) < 16 ? Dg / (4 * lanes) + 1 : 16;
    q.chunks = blocks < 256 ? 256 / blocks : 1;
    if (q.chunks > most) q.chunks = most;
    if (q.chunks < least) q.chunks = least;
    q.chunk = ceil_div(Dg, q.chunks);
    q.chunks = ceil_div(Dg, q.chunk);
    q.apply_lanes = L > 256 ? 64 : 8;
    q.apply_chans = kNormApplyThreads / q.apply_lanes * (bwd ? 8 : 4);
    q.parts = B * ceil_div(L, 8 * q.apply_lanes);
    return q;
  }
  const bool rows = q.kind == kNormRowTeam || q.kind == kNormRowBlock || q.kind == kNormRowWide;
  const int64_t work = rows ? ceil_div(B, bwd ? q.threads / q.lanes : 1) : B * q.tiles;
  if (bwd && q.kind < kNormColTwo) {
    // Every workgroup takes `each` tiles, in rounds of what the chip holds at once: the fewest tiles one after
    // the other, and among equals the fewest parts of the weight's sums (4 x 5120 channels, 40 groups, L = 2048, bf16,
    // gated: 5120 tiles, 768 workgroups at once, seven tiles each 108 us; five each, a second round of a third, 131).
    const int64_t all = work * G, once = 256 * cu, last = ceil_div(all, once);
    int64_t each = last < work ? last : work, least = ceil_div(ceil_div(work, each) * G, once) * each;
    for (int64_t n = each - 1; n > 0 && n >= last - 64; --n) {
      const int64_t rounds = ceil_div(ceil_div(work, n) * G, once) * n;
      if (rounds < least) {
        least = rounds;
        each = n;
      }
    }
    q.parts = ceil_div(work, each);
    return q;
  }
  // Backward, workgroups that fill the chip and no more: every part of the weight's sums is written and read.
  // Token-major that is one a CU, or two for one team of up to 640 threads (4097 to 5120 channels), no gate,
  // 2-byte numbers: 8192 tokens of 5120 channels, bf16, 66 us, with one 76; fp32 110, 105; gated 109, 108; of 512
  // channels, where one workgroup holds 1024 threads, 17.5, 13.6; of 7168, 99, 92.  The registers hold two of 704 or 768
  // threads as well, which is faster for many tokens and slower for few (one, two; one set of arrays: 8192 tokens of 2816
  // channels 34.8, 31.7, of 5632 63.9, 55.1, of 6144 64.2, 57.4; 1000 tokens 17.6, 17.4; 19.8, 22.0; 19.8, 22.3).  Forward (kNormRowBlock,
  // kNormRowWide) a CU gets the power of two that makes up to 2048 threads: two workgroups of 640 for 5120 channels
  // 33 us, three 38; two of 896 for 7168 channels 51 us, one 68.
  const bool two = q.kind == kNormRowBlock && q.threads <= 640 && !gate && in_width + grad_width == 4;
  int64_t fit = !rows ? 4 : bwd && two ? 2 : 1;
  while (!bwd && rows && 2 * fit * q.threads <= 2048) fit *= 2;
  int64_t most = 256 * fit / G;
  if (most < 1) most = 1;
  if (most > work) most = work;
  q.parts = ceil_div(work, ceil_div(work, most));
  return q;
}

hipError_t launch_norm_fwd(const NormParams& p, const NormPlan& q, Dt in, Dt out, hipStream_t s) {
  if (in == Dt::BF16) return out == Dt::BF16 ? fwd_t<uint16_t, uint16_t>(p, q, s) : fwd_t<uint16_t, float>(p, q, s);
  return out == Dt::BF16 ? fwd_t<float, uint16_t>(p, q, s) : fwd_t<float, float>(p, q, s);
}

}  // namespace mamba
