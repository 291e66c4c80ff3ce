// glr.hip -- the gated linear recurrence over sequences and one token at a time (gfx950).  Rows of up to 256 tokens:
// glr_short.hip.
//
// Per channel, one state h: h_t = a_t h_(t-1) + u_t with the gates of glr.hpp, y_t = h_t silu(z_t).
// A stretch of tokens takes the state in front of it, h, to P h + H with P the product of its
// decays and H its end state from zero, and stretches compose, so a row is scanned in
// parallel: a lane has 8 consecutive tokens (16 or 32 bytes of each input, one load), a wave
// 512, a workgroup's waves lie one after the other on the row and take it in such tiles, the
// state carried from tile to tile.  Inside a lane the tokens run in sequence twice (for its
// (P, H), and again from its true state), lanes are scanned in six exchanges, waves through LDS.
//
// Every input is read once and every output written once, and HBM bounds it where there are rows enough: 20480 rows,
// L = 2048, bf16 with both gates, 76 us for 419 MB, 5.5 TB/s where a plain copy reaches 5.1; 4096 rows,
// L = 32768, 248 us for 1.34 GB, 5.4 TB/s.  Vector instructions take 0.75 to 0.86 of the issue cycles beside that (the
// exponentials of three gates a token), so there is little left on either side.  One token of 4096 channels takes
// 3 us on the GPU.
#include "glr.hpp"

namespace mamba {
namespace {

// kSummary: only the (P, H) of each segment but the last.  kEdge: rows whose last lane has four to seven tokens, through
// Share (32768 rows of 333 tokens, bf16: 60 us without, 41 with it).  With fewer tokens there the lane's own loads cost
// no more (7680 rows of 1003 tokens: 22.3, 23.4), nor do 4-byte ones (333 tokens: 47, 54), and past 8 waves Share's
// registers cost two workgroups of 16 waves their place on a CU (16381 tokens: 118, 131).
template <typename T, typename O, bool kBlend, bool kSummary, bool kEdge>
__global__ __launch_bounds__(1024) void glr_fwd_kernel(GlrParams p) {
  __shared__ float totals[2][2][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t rows = p.B * p.D;
  const int64_t seg = blockIdx.x / rows, row = blockIdx.x - seg * rows;
  const int64_t b = row / p.D, d = row - b * p.D;
  const int64_t t0 = seg * p.seg_len;
  const int64_t t1 = p.L - t0 < p.seg_len ? p.L : t0 + p.seg_len;
  const int64_t len = glr_length(p, b);
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + d * p.L;
  const T* r = static_cast<const T*>(p.r) + b * p.r_stride + d * p.L;
  const T* ig = p.i ? static_cast<const T*>(p.i) + b * p.i_stride + d * p.L : nullptr;
  const T* z = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + d * p.L : nullptr;
  O* y = static_cast<O*>(p.y) + row * p.L;
  const GlrChannel channel = glr_channel<kBlend>(p, d, len);
  const float A2 = channel.A2, rb = channel.rb, ib = channel.ib;

  Affine all;                         // kSummary: the segment so far
  float carry = 0.0f;                 // state in front of the tile
  if constexpr (!kSummary) {
    carry = p.init ? p.init[row] : 0.0f;
    if (seg) carry = glr_enter(p.sum + row * p.S * 2, 2, seg, carry, lane);
  }
  int turn = 0;
  for (int64_t tile = t0; tile < t1; tile += (int64_t)waves * kGlrWave, turn ^= 1) {
    const int64_t t = tile + (int64_t)threadIdx.x * kGlrLane;
    Share q;
    const int live = clamp8((len < t1 ? len : t1) - t);
    if constexpr (kEdge) q = glr_share(p.L, t1, len, t);
    auto load = [&](const T* from, uint32_t dead) {
      if constexpr (kEdge) return load_share(from, p.L, q, dead);
      else return load_raw8(from + t, live);
    };
    const Raw8<T> xr = load(x, 0), rr = load(r, kMinusInf<T>);
    Raw8<T> ir, zr;
    if (ig) ir = load(ig, 0);
    if constexpr (!kSummary)
      if (z) zr = load(z, 0);
    float a[8], u[8];
    Affine v;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const GlrGate g = glr_gate<kBlend>(kEdge ? get8(rr, j) : glr_r(rr, j, live), rb, A2);
      a[j] = g.a;
      u[j] = g.n * get8(xr, j);
    }
    if (ig) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] *= hw_rcp(1.0f + hw_exp2(__builtin_fmaf(get8(ir, j), -kLog2e, ib)));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v.P *= a[j];
      v.H = __builtin_fmaf(a[j], v.H, u[j]);
    }
    const Affine incl = scan_up(v);
    const Affine excl = shift_up(incl);
    Affine tile_total, before;        // the tile, and its waves in front of this one
    if (waves == 1) {
      tile_total.P = lane_of(incl.P, 63);
      tile_total.H = lane_of(incl.H, 63);
    } else {
      if (lane == 63) {
        totals[turn][0][wave] = incl.P;
        totals[turn][1][wave] = incl.H;
      }
      __syncthreads();                // the other half of `totals` may still be read: the next tile writes that one
      for (int w = 0; w < waves; ++w) {
        if (w == wave) before = tile_total;
        tile_total = glr_through(tile_total, Affine{totals[turn][0][w], totals[turn][1][w]});
      }
    }
    if constexpr (kSummary) {
      all = glr_through(all, tile_total);
    } else {
      float h = __builtin_fmaf(before.P, carry, before.H);
      h = __builtin_fmaf(excl.P, h, excl.H);
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        h = __builtin_fmaf(a[j], h, u[j]);
        o[j] = h;
      }
      if (z) {
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr, j));
      }
      // Past the caches where whole lines are written at once; 4-byte outputs take two stores a line.  20480 rows,
      // L = 2048, fp32 out: 94.8 us past the caches, 89.6 through them; 4096 rows, L = 32768, bf16: 250, 260.
      if constexpr (kEdge) store_share<O, sizeof(O) == 2>(y, o, q);
      else store8<O, sizeof(O) == 2>(y + t, o, live, clamp8(t1 - t));
      carry = __builtin_fmaf(tile_total.P, carry, tile_total.H);
    }
  }
  if (threadIdx.x == 0) {
    if constexpr (kSummary) {
      p.sum[(row * p.S + seg) * 2] = all.P;
      p.sum[(row * p.S + seg) * 2 + 1] = all.H;
    } else if (p.final_state && seg == p.S - 1) {
      p.final_state[row] = carry;
    }
  }
}

// One token: a channel of a row per thread.
template <typename T, typename O, bool kBlend>
__global__ __launch_bounds__(256) void glr_update_kernel(GlrParams p) {
  const int64_t per_row = (p.D + 255) / 256;
  const int64_t b = blockIdx.x / per_row;
  const int64_t d = (blockIdx.x - b * per_row) * 256 + threadIdx.x;
  if (d >= p.D) return;
  const int64_t slot = p.slots ? (int64_t)p.slots[b] : b;
  const bool on = slot >= 0 && slot < p.n_slots;          // uniform over the workgroup
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride;
  const T* r = static_cast<const T*>(p.r) + b * p.r_stride;
  const T* ig = static_cast<const T*>(p.i) + b * p.i_stride;
  const T* z = static_cast<const T*>(p.z) + b * p.z_stride;
  float o = 0.0f;
  if (on) {
    float* st = p.final_state + slot * p.D;
    const GlrChannel channel = glr_channel<kBlend>(p, d, 1);
    const GlrGate g = glr_gate<kBlend>(get1(r + d), channel.rb, channel.A2);
    float u = g.n * get1(x + d);
    if (p.i) u *= sigmoid(get1(ig + d) + (p.i_bias ? p.i_bias[d] : 0.0f));
    const float h = __builtin_fmaf(g.a, st[d], u);
    st[d] = h;
    o = p.z ? h * silu(get1(z + d)) : h;
  }
  put1(static_cast<O*>(p.y) + b * p.D + d, o);
}

template <typename T>
hipError_t summary_t(const GlrParams& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.B * p.D * (p.S - 1))), block(64u * p.waves);
  if (p.blend) hipLaunchKernelGGL((glr_fwd_kernel<T, T, true, true, false>), grid, block, 0, s, p);
  else hipLaunchKernelGGL((glr_fwd_kernel<T, T, false, true, false>), grid, block, 0, s, p);
  return hipGetLastError();
}

template <typename T, typename O, bool kBlend>
hipError_t fwd_b(const GlrParams& p, hipStream_t s) {
  const unsigned rows = (unsigned)(p.B * p.D), threads = 64u * p.waves;
  if (p.S > 1) {
    const hipError_t e = summary_t<T>(p, s);
    if (e != hipSuccess) return e;
  }
  if constexpr (sizeof(T) == 2) {
    if (p.L % kGlrLane > 3 && p.waves <= 8) {
      hipLaunchKernelGGL((glr_fwd_kernel<T, O, kBlend, false, true>), dim3(rows * (unsigned)p.S), dim3(threads), 0, s, p);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((glr_fwd_kernel<T, O, kBlend, false, false>), dim3(rows * (unsigned)p.S), dim3(threads), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t fwd_t(const GlrParams& p, hipStream_t s) {
  return p.blend ? fwd_b<T, O, true>(p, s) : fwd_b<T, O, false>(p, s);
}

template <typename T, typename O>
hipError_t upd_t(const GlrParams& p, hipStream_t s) {
  const unsigned wgs = (unsigned)(p.B * ((p.D + 255) / 256));
  if (p.blend) hipLaunchKernelGGL((glr_update_kernel<T, O, true>), dim3(wgs), dim3(256), 0, s, p);
  else hipLaunchKernelGGL((glr_update_kernel<T, O, false>), dim3(wgs), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_fwd(const GlrParams& p, Dt in, Dt out, hipStream_t s) {
  if (p.lanes) return launch_glr_short_fwd(p, in, out, s);
  if (in == Dt::BF16) return out == Dt::BF16 ? fwd_t<uint16_t, uint16_t>(p, s) : fwd_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? fwd_t<float, uint16_t>(p, s) : fwd_t<float, float>(p, s);
}

// (P, H) of every segment but a row's last.
hipError_t launch_glr_summary(const GlrParams& p, Dt in, hipStream_t s) {
  return in == Dt::BF16 ? summary_t<uint16_t>(p, s) : summary_t<float>(p, s);
}

hipError_t launch_glr_update(const GlrParams& p, Dt in, Dt out, hipStream_t s) {
  if (in == Dt::BF16) return out == Dt::BF16 ? upd_t<uint16_t, uint16_t>(p, s) : upd_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? upd_t<float, uint16_t>(p, s) : upd_t<float, float>(p, s);
}

}  // namespace mamba
