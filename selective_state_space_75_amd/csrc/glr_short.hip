// glr_short.hip -- the gated linear recurrence over short rows, forward and backward (gfx950).
//
// The mathematics of glr.hip and glr_bwd.hip, with several rows in a wave: a row has `p.lanes` neighbouring lanes (a power
// of two, 8 tokens each), scans and sums run over those, and a workgroup of four waves takes 256 / lanes rows.
// A wave per row would leave most lanes without a token, and the chip waiting for workgroups that do next to nothing:
// 32768 rows of 8 tokens, bf16: forward 30 us so, 6 here, backward 63, 10; of 256 tokens 30, 24 and 62, 45 (HBM 16, 30).
// Up to 64 tokens a row the launch and one round trip to memory bound it, then the shuffles of the scans beside HBM.
#include "glr.hpp"

namespace mamba {
namespace {

struct Lane : Share {
  int64_t b, d, row, len;       // len: tokens of the row that count
  int sub;                      // lane of the row
  bool mine;                    // there is such a row
};

__device__ __forceinline__ Lane glr_lane(const GlrParams& p) {
  Lane o;
  const int shift = __builtin_ctz(p.lanes);
  const uint32_t rows = (uint32_t)(p.B * p.D), D = (uint32_t)p.D;                  // below 2^26: a wave per row would be a launch
  uint32_t row = blockIdx.x * (256u >> shift) + (threadIdx.x >> shift);
  o.sub = threadIdx.x & (p.lanes - 1);
  o.mine = row < rows;
  if (!o.mine) row = rows - 1;
  o.row = row;
  o.b = row / D;
  o.d = row - (uint32_t)o.b * D;
  o.len = glr_length(p, o.b);
  static_cast<Share&>(o) = glr_share(p.L, o.mine ? p.L : 0, o.len, o.sub * kGlrLane);
  return o;
}

// (P, H) of the row's lanes up to this one, and from this one on (composed from the last to the first).
__device__ __forceinline__ Affine share_up(Affine v, int sub, int lanes) {
  for (int m = 1; m < lanes; m *= 2) {
    const float P = __shfl_up(v.P, m), H = __shfl_up(v.H, m);
    if (sub >= m) {
      v.H = __builtin_fmaf(v.P, H, v.H);
      v.P *= P;
    }
  }
  return v;
}
__device__ __forceinline__ Affine share_down(Affine v, int sub, int lanes) {
  for (int m = 1; m < lanes; m *= 2) {
    const float P = __shfl_down(v.P, m), H = __shfl_down(v.H, m);
    if (sub + m < lanes) {
      v.H = __builtin_fmaf(v.P, H, v.H);
      v.P *= P;
    }
  }
  return v;
}

template <typename T, typename O, bool kBlend>
__global__ __launch_bounds__(256) void glr_short_fwd_kernel(GlrParams p) {
  const Lane q = glr_lane(p);
  const int64_t at = q.d * p.L;
  const Raw8<T> xr = load_share(static_cast<const T*>(p.x) + q.b * p.x_stride + at, p.L, q, 0);
  const Raw8<T> rr = load_share(static_cast<const T*>(p.r) + q.b * p.r_stride + at, p.L, q, kMinusInf<T>);
  Raw8<T> ir, zr;
  if (p.i) ir = load_share(static_cast<const T*>(p.i) + q.b * p.i_stride + at, p.L, q, 0);
  if (p.z) zr = load_share(static_cast<const T*>(p.z) + q.b * p.z_stride + at, p.L, q, 0);
  const GlrChannel channel = glr_channel<kBlend>(p, q.d, q.len);
  const float A2 = channel.A2, rb = channel.rb, ib = channel.ib;
  const float before = p.init ? p.init[q.row] : 0.0f;
  float a[8], u[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const GlrGate g = glr_gate<kBlend>(get8(rr, j), rb, A2);
    a[j] = g.a;
    u[j] = g.n * get8(xr, j);
  }
  if (p.i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] *= hw_rcp(1.0f + hw_exp2(__builtin_fmaf(get8(ir, j), -kLog2e, ib)));
  }
  Affine v;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v.P *= a[j];
    v.H = __builtin_fmaf(a[j], v.H, u[j]);
  }
  v = share_up(v, q.sub, p.lanes);
  Affine front{__shfl_up(v.P, 1), __shfl_up(v.H, 1)};
  if (q.sub == 0) front = Affine{};
  float h = __builtin_fmaf(front.P, before, front.H), o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    h = __builtin_fmaf(a[j], h, u[j]);
    o[j] = h;
  }
  if (p.z) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] *= silu(get8(zr, j));
  }
  store_share<O, false>(static_cast<O*>(p.y) + q.row * p.L, o, q);
  if (p.final_state && q.mine && q.sub == p.lanes - 1) p.final_state[q.row] = __builtin_fmaf(v.P, before, v.H);
}

template <typename T, typename Gr, bool kBlend>
__global__ __launch_bounds__(256) void glr_short_bwd_kernel(GlrParams p) {
  const Lane q = glr_lane(p);
  const int64_t at = q.d * p.L, out = q.row * p.L;
  Raw8<T> xr = load_share(static_cast<const T*>(p.x) + q.b * p.x_stride + at, p.L, q, 0);
  const Raw8<T> rr = load_share(static_cast<const T*>(p.r) + q.b * p.r_stride + at, p.L, q, kMinusInf<T>);
  Raw8<Gr> yr = load_share(static_cast<const Gr*>(p.dy) + out, p.L, q, 0);
  Raw8<T> ir, zr;
  if (p.i) ir = load_share(static_cast<const T*>(p.i) + q.b * p.i_stride + at, p.L, q, 0);
  if (p.z) zr = load_share(static_cast<const T*>(p.z) + q.b * p.z_stride + at, p.L, q, 0);
  const GlrChannel channel = glr_channel<kBlend>(p, q.d, q.len);
  const float A = channel.A, A2 = channel.A2, rb = channel.rb, ib = channel.ib;
  const float before = p.init ? p.init[q.row] : 0.0f, after = p.dfinal ? p.dfinal[q.row] : 0.0f;
  float a[8], s[8], c1[8], ng[8], ra[8], one[8], e[8], sz[8];      // as in glr_bwd.hip
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const GlrGate k = glr_gate<kBlend>(get8(rr, j), rb, A2);
    a[j] = k.a; s[j] = k.s; c1[j] = k.c; ng[j] = k.n; ra[j] = k.ra;
    if (p.i) {
      const float ei = hw_exp2(__builtin_fmaf(get8(ir, j), -kLog2e, ib)), g = hw_rcp(1.0f + ei);
      ng[j] *= g;
      ra[j] *= g;
      one[j] = one_less(g, ei);
    }
    sz[j] = p.z ? sigmoid(get8(zr, j)) : 1.0f;
    e[j] = get8(yr, j);
    if (p.z) e[j] *= get8(zr, j) * sz[j];
  }
  Affine f, k;                                 // forwards and backwards over the lane's tokens
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    f.P *= a[j];
    f.H = __builtin_fmaf(a[j], f.H, ng[j] * get8(xr, j));
  }
#pragma unroll
  for (int j = 7; j >= 0; --j) k.H = a[j] * (k.H + e[j]);
  k.P = f.P;
  f = share_up(f, q.sub, p.lanes);
  k = share_down(k, q.sub, p.lanes);
  Affine front{__shfl_up(f.P, 1), __shfl_up(f.H, 1)}, behind{__shfl_down(k.P, 1), __shfl_down(k.H, 1)};
  if (q.sub == 0) front = Affine{};
  if (q.sub == p.lanes - 1) behind = Affine{};
  float h = __builtin_fmaf(front.P, before, front.H), c = __builtin_fmaf(behind.P, after, behind.H);
  if (p.dinit && q.mine && q.sub == 0) p.dinit[q.row] = __builtin_fmaf(k.P, after, k.H);
  float hp[8], o[8];                           // hp: state in front of each token
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    hp[j] = h;
    h = __builtin_fmaf(a[j], h, ng[j] * get8(xr, j));
  }
  if (p.z) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float hj = j < 7 ? hp[j < 7 ? j + 1 : 7] : h;
      o[j] = get8(yr, j) * hj * sz[j] * __builtin_fmaf(get8(zr, j), 1.0f - sz[j], 1.0f);
    }
    store_share<Gr, false>(static_cast<Gr*>(p.dz) + out, o, q);
  }
  float dr[8], sums[3] = {0.0f, 0.0f, 0.0f};   // of A, r_bias, i_bias
#pragma unroll
  for (int j = 7; j >= 0; --j) {
    const float y = e[j] + c, xj = get8(xr, j);
    c = a[j] * y;
    o[j] = y * ng[j];
    if constexpr (kBlend) {
      dr[j] = y * __builtin_fmaf(ng[j], xj, -s[j] * hp[j]) * a[j];       // n = s
    } else {
      const float ds = y * __builtin_fmaf(a[j], hp[j], -xj * ra[j]) * s[j];
      sums[0] += ds;
      dr[j] = ds * A * c1[j];
    }
    sums[1] += dr[j];
  }
  store_share<Gr, false>(static_cast<Gr*>(p.dx) + out, o, q);
  store_share<Gr, false>(static_cast<Gr*>(p.dr) + out, dr, q);
  if (p.i) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      o[j] *= get8(xr, j) * one[j];
      sums[2] += o[j];
    }
    store_share<Gr, false>(static_cast<Gr*>(p.di) + out, o, q);
  }
  for (int m = 1; m < p.lanes; m *= 2) {
#pragma unroll
    for (int j = 0; j < 3; ++j) sums[j] += __shfl_xor(sums[j], m);
  }
  if (q.sub || !q.mine) return;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    float* dst = p.B > 1 ? p.part + (q.b * 3 + j) * p.D : j == 0 ? p.dA : j == 1 ? p.dr_bias : p.di_bias;
    if (dst) dst[q.d] = sums[j];
  }
}

template <typename T, typename O, bool kBlend>
hipError_t fwd_b(const GlrParams& p, hipStream_t s) {
  hipLaunchKernelGGL((glr_short_fwd_kernel<T, O, kBlend>), dim3((unsigned)((p.B * p.D * p.lanes + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename T, typename O>
hipError_t fwd_t(const GlrParams& p, hipStream_t s) {
  return p.blend ? fwd_b<T, O, true>(p, s) : fwd_b<T, O, false>(p, s);
}
template <typename T, typename Gr, bool kBlend>
hipError_t bwd_b(const GlrParams& p, hipStream_t s) {
  hipLaunchKernelGGL((glr_short_bwd_kernel<T, Gr, kBlend>), dim3((unsigned)((p.B * p.D * p.lanes + 255) / 256)), dim3(256), 0, s, p);
  return hipGetLastError();
}
template <typename T, typename Gr>
hipError_t bwd_t(const GlrParams& p, hipStream_t s) {
  return p.blend ? bwd_b<T, Gr, true>(p, s) : bwd_b<T, Gr, false>(p, s);
}

}  // namespace

hipError_t launch_glr_short_fwd(const GlrParams& p, Dt in, Dt out, hipStream_t s) {
  if (in == Dt::BF16) return out == Dt::BF16 ? fwd_t<uint16_t, uint16_t>(p, s) : fwd_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? fwd_t<float, uint16_t>(p, s) : fwd_t<float, float>(p, s);
}
hipError_t launch_glr_short_bwd(const GlrParams& p, Dt in, Dt grad, hipStream_t s) {
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, s) : bwd_t<uint16_t, float>(p, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, s) : bwd_t<float, float>(p, s);
}

}  // namespace mamba
