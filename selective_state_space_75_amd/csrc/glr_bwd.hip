// glr_bwd.hip -- gradients of the gated linear recurrence (gfx950).
//
// With e_t = dy_t silu(z_t), the adjoint of h_t is q_t = e_t + c_(t+1), where c_t = a_t q_t is what
// a token hands to the one before it (c_L: the gradient of the final state).  So c runs through
// the row backwards with the decays that h runs with forwards, c_t = a_t c_(t+1) + a_t e_t, and a
// stretch of tokens takes c behind it to P c + C in front of it, P being the same product.
//     dx = q n g,  di = dx x (1 - g),  dz = dy h sigma (1 + z (1 - sigma)), sigma = sigmoid(z)
//     dl = q (a h_prev - g x a^2 / n),  dr = dl A s (1 - s),  dA = sum dl s   (decay rule, l = A s)
//     dr = q (g x - h_prev) s a                                                (blend)
// A workgroup has a tile of up to 8192 tokens (16 waves of 512) on the chip: its five inputs stay in
// registers, both scans run at once and the gradients are written from there.  A longer row is cut into
// tiles, whose entering states come from the (P, H) of the tiles before them, left by a first launch that reads
// x, r and i (mamba::launch_glr_summary).  Where there are rows enough, a workgroup takes all tiles of its row
// from the last to the first and c stays with it; few rows have a workgroup per tile, and the first launch
// (kSummary below, all five inputs) leaves C too.
// dA and the biases' gradients: a sum per workgroup, then one small launch over batch rows and workgroups of a row.
// HBM bounds it: 20480 rows, L = 2048, bf16 with both gates, 150 us for 755 MB, 5.0 TB/s; vector instructions take
// 0.8 of the issue cycles beside that.
#include "glr.hpp"

namespace mamba {
namespace {

// kSummary: only the (P, H, C) of each tile.  kLoop: more than one tile a workgroup.  kEdge: rows that do not end with a
// whole lane, through Share (the others go without its registers: 20480 rows, L = 2048, bf16: 148 us, with it 168).
template <typename T, typename Gr, bool kBlend, bool kSummary, bool kLoop, bool kEdge, int kThreads>
__global__ __launch_bounds__(kThreads) void glr_bwd_kernel(GlrParams p) {
  __shared__ float totals[2][3][16];
  __shared__ float sums[3][16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int64_t rows = p.B * p.D;
  const int64_t own = blockIdx.x / rows, row = blockIdx.x - own * rows;     // of the row's workgroups
  const int64_t b = row / p.D, d = row - b * p.D;
  const int64_t len = glr_length(p, b);
  const T* x = static_cast<const T*>(p.x) + b * p.x_stride + d * p.L;
  const T* r = static_cast<const T*>(p.r) + b * p.r_stride + d * p.L;
  const T* ig = p.i ? static_cast<const T*>(p.i) + b * p.i_stride + d * p.L : nullptr;
  const T* zg = p.z ? static_cast<const T*>(p.z) + b * p.z_stride + d * p.L : nullptr;
  const Gr* dy = static_cast<const Gr*>(p.dy) + row * p.L;
  const GlrChannel channel = glr_channel<kBlend>(p, d, len);
  const float A = channel.A, A2 = channel.A2, rb = channel.rb, ib = channel.ib;
  const int width = p.groups > 1 ? 3 : 2;                                   // numbers of a tile's summary
  const float* sum = p.S > 1 ? p.sum + row * p.S * width : nullptr;
  const int64_t lo = own * p.group, hi = p.S < lo + p.group ? p.S : lo + p.group;

  float c_in = 0.0f;                           // what the tiles behind hand to this one
  if constexpr (!kSummary) {
    c_in = p.dfinal ? p.dfinal[row] : 0.0f;
    for (int64_t base = p.S - 1; base >= hi; base -= 64) {
      Affine v;
      if (base - lane >= hi) v = Affine{sum[(base - lane) * 3], sum[(base - lane) * 3 + 2]};
      v = scan_up(v);
      c_in = __builtin_fmaf(lane_of(v.P, 63), c_in, lane_of(v.H, 63));
    }
  }
  float sA = 0.0f, sr = 0.0f, si = 0.0f;
  int turn = 0;
  for (int64_t seg = hi - 1; seg >= (kLoop ? lo : hi - 1); --seg, turn ^= 1) {
    const int64_t t0 = seg * p.seg_len;
    const int64_t t1 = p.L - t0 < p.seg_len ? p.L : t0 + p.seg_len;
    const int64_t t = t0 + (int64_t)threadIdx.x * kGlrLane;
    Share q;
    const int live = clamp8((len < t1 ? len : t1) - t);
    if constexpr (kEdge) q = glr_share(p.L, t1, len, t);
    auto load = [&](const auto* from, uint32_t dead) {
      if constexpr (kEdge) return load_share(from, p.L, q, dead);
      else return load_raw8(from + t, live);
    };
    Raw8<T> xr = load(x, 0), rr = load(r, kMinusInf<T>);
    Raw8<Gr> yr = load(dy, 0);
    Raw8<T> ir, zr;
    if (ig) ir = load(ig, 0);
    if (zg) zr = load(zg, 0);

    // Of n, g and a^2 / n only the products with g are needed.  one: 1 - g
    float a[8], s[8], c1[8], ng[8], ra[8], one[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const GlrGate k = glr_gate<kBlend>(kEdge ? get8(rr, j) : glr_r(rr, j, live), rb, A2);
      a[j] = k.a; s[j] = k.s; c1[j] = k.c; ng[j] = k.n; ra[j] = k.ra;
    }
    if (ig) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float ei = hw_exp2(__builtin_fmaf(get8(ir, j), -kLog2e, ib)), g = hw_rcp(1.0f + ei);
        ng[j] *= g;
        ra[j] *= g;
        one[j] = one_less(g, ei);
      }
    }
    float e[8], sz[8];
    if (zg) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sz[j] = sigmoid(get8(zr, j));
        e[j] = get8(yr, j) * get8(zr, j) * sz[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) e[j] = get8(yr, j);
    }
    Affine f, k;                               // forwards and backwards over the lane's tokens
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      f.P *= a[j];
      f.H = __builtin_fmaf(a[j], f.H, ng[j] * get8(xr, j));
    }
#pragma unroll
    for (int j = 7; j >= 0; --j) k.H = a[j] * (k.H + e[j]);
    k.P = f.P;
    f = scan_up(f);
    k = scan_down(k, lane);
    if (lane == 63) {
      totals[turn][0][wave] = f.P;
      totals[turn][1][wave] = f.H;
    }
    if (lane == 0) totals[turn][2][wave] = k.H;
    __syncthreads();                           // the other half of `totals` may still be read: the next tile writes that one
    Affine front, behind, all, back;           // waves in front of this one, behind it, and all of them
    for (int w = 0; w < waves; ++w) {
      if (w == wave) front = all;
      all = glr_through(all, Affine{totals[turn][0][w], totals[turn][1][w]});
    }
    for (int w = waves - 1; w >= 0; --w) {
      if (w == wave) behind = back;
      back = glr_through(back, Affine{totals[turn][0][w], totals[turn][2][w]});
    }
    if constexpr (kSummary) {
      if (threadIdx.x == 0) {
        float* o = p.sum + (row * p.S + seg) * 3;
        o[0] = all.P; o[1] = all.H; o[2] = back.H;
      }
      continue;
    }
    keep(xr);
    keep(yr);
    if (zg) keep(zr);
    float h = p.init ? p.init[row] : 0.0f, c = c_in;
    if (seg) h = glr_enter(sum, width, seg, h, lane);
    c_in = __builtin_fmaf(back.P, c_in, back.H);
    h = __builtin_fmaf(front.P, h, front.H);
    c = __builtin_fmaf(behind.P, c, behind.H);
    const Affine fe = shift_up(f), ke = shift_down(k);
    h = __builtin_fmaf(fe.P, h, fe.H);
    c = __builtin_fmaf(ke.P, c, ke.H);

    const int there = clamp8(t1 - t);
    const int64_t at = row * p.L + (kEdge ? 0 : t);
    auto store = [&](void* to, const float (&v)[8]) {
      if constexpr (kEdge) store_share<Gr, true>(static_cast<Gr*>(to) + at, v, q);
      else store8(static_cast<Gr*>(to) + at, v, live, there);
    };
    float hp[8];                               // state in front of each token
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      hp[j] = h;
      h = __builtin_fmaf(a[j], h, ng[j] * get8(xr, j));
    }
    if (zg) {
      float o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float hj = j < 7 ? hp[j < 7 ? j + 1 : 7] : h;
        o[j] = get8(yr, j) * hj * sz[j] * __builtin_fmaf(get8(zr, j), 1.0f - sz[j], 1.0f);
      }
      store(p.dz, o);
    }
    float dx[8], dr[8];
#pragma unroll
    for (int j = 7; j >= 0; --j) {
      const float v = e[j] + c;
      c = a[j] * v;
      dx[j] = v * ng[j];
      const float xj = get8(xr, j);
      if constexpr (kBlend) {
        dr[j] = v * __builtin_fmaf(ng[j], xj, -s[j] * hp[j]) * a[j];     // n = s
      } else {
        const float ds = v * __builtin_fmaf(a[j], hp[j], -xj * ra[j]) * s[j];
        sA += ds;
        dr[j] = ds * A * c1[j];
      }
      sr += dr[j];
    }
    store(p.dx, dx);
    store(p.dr, dr);
    if (ig) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        dx[j] *= get8(xr, j) * one[j];
        si += dx[j];
      }
      store(p.di, dx);
    }
  }
  if constexpr (kSummary) return;
  if (p.dinit && lo == 0 && threadIdx.x == 0) p.dinit[row] = c_in;
  sA = wave_sum63(sA);
  sr = wave_sum63(sr);
  si = wave_sum63(si);
  if (lane == 63) {
    sums[0][wave] = sA;
    sums[1][wave] = sr;
    sums[2][wave] = si;
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float o = 0.0f;
    for (int w = 0; w < waves; ++w) o += sums[threadIdx.x][w];
    if (p.B * p.groups == 1) {                 // nothing to add up
      float* dst = threadIdx.x == 0 ? p.dA : threadIdx.x == 1 ? p.dr_bias : p.di_bias;
      if (dst) dst[d] = o;
    } else {
      p.part[((b * p.groups + own) * 3 + threadIdx.x) * p.D + d] = o;
    }
  }
}

// Sums over batch rows and workgroups of a row: 16 channels x 16 shares of them per workgroup.
__global__ __launch_bounds__(256) void glr_sum_kernel(GlrParams p) {
  __shared__ float share[16][16];
  const int64_t blocks = (p.D + 15) / 16;
  const int k = (int)(blockIdx.x / blocks);
  const int64_t d = (blockIdx.x - k * blocks) * 16 + (threadIdx.x & 15);
  const int y = threadIdx.x >> 4;
  float o = 0.0f;
  if (d < p.D) o = strided_sum(p.part + k * p.D + d, 3 * p.D, y, p.B * p.groups);
  share[y][threadIdx.x & 15] = o;
  __syncthreads();
  if (y || d >= p.D) return;
  for (int w = 1; w < 16; ++w) o += share[w][threadIdx.x];
  float* dst = k == 0 ? p.dA : k == 1 ? p.dr_bias : p.di_bias;
  if (dst) dst[d] = o;
}

template <typename T, typename Gr, bool kBlend, bool kEdge, int kThreads>
hipError_t bwd_n(const GlrParams& p, hipStream_t s) {
  const unsigned rows = (unsigned)(p.B * p.D);
  const dim3 block(64u * p.waves), grid(rows * (unsigned)p.groups);
  hipError_t e = hipSuccess;
  if (p.groups > 1) {
    GlrParams one = p;
    one.group = 1;
    hipLaunchKernelGGL((glr_bwd_kernel<T, Gr, kBlend, true, false, kEdge, kThreads>), dim3(rows * (unsigned)p.S), block, 0, s, one);
    e = hipGetLastError();
  } else if (p.S > 1) {
    e = launch_glr_summary(p, sizeof(T) == 2 ? Dt::BF16 : Dt::F32, s);
  }
  if (e != hipSuccess) return e;
  if constexpr (kThreads == 512) {             // more waves are only taken for one tile
    if (p.group > 1) hipLaunchKernelGGL((glr_bwd_kernel<T, Gr, kBlend, false, true, kEdge, 512>), grid, block, 0, s, p);
    else hipLaunchKernelGGL((glr_bwd_kernel<T, Gr, kBlend, false, false, kEdge, 512>), grid, block, 0, s, p);
  } else {
    hipLaunchKernelGGL((glr_bwd_kernel<T, Gr, kBlend, false, false, kEdge, kThreads>), grid, block, 0, s, p);
  }
  return hipGetLastError();
}

template <typename T, typename Gr, int kThreads>
hipError_t bwd_e(const GlrParams& p, hipStream_t s) {
  if (p.L % kGlrLane) return p.blend ? bwd_n<T, Gr, true, true, kThreads>(p, s) : bwd_n<T, Gr, false, true, kThreads>(p, s);
  return p.blend ? bwd_n<T, Gr, true, false, kThreads>(p, s) : bwd_n<T, Gr, false, false, kThreads>(p, s);
}

template <typename T, typename Gr>
hipError_t bwd_t(const GlrParams& p, hipStream_t s) {
  return p.waves <= 8 ? bwd_e<T, Gr, 512>(p, s) : bwd_e<T, Gr, 1024>(p, s);
}

}  // namespace

hipError_t launch_glr_bwd(const GlrParams& p, Dt in, Dt grad, hipStream_t s) {
  hipError_t e;
  if (p.lanes) e = launch_glr_short_bwd(p, in, grad, s);
  else if (in == Dt::BF16) e = grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, s) : bwd_t<uint16_t, float>(p, s);
  else e = grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, s) : bwd_t<float, float>(p, s);
  if (e != hipSuccess || p.B * p.groups == 1) return e;
  hipLaunchKernelGGL(glr_sum_kernel, dim3((unsigned)(3 * ((p.D + 15) / 16))), dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace mamba
