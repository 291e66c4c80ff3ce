// glr.hpp -- device helpers shared by the gated linear recurrence's and the layer norm's kernels (gfx950).
#pragma once

#include "device_math.hpp"
#include "kernels.hpp"

namespace mamba {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
// The same at any element's alignment: the target takes unaligned global accesses.
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));

// Eight consecutive numbers of a row as they lie in memory.
template <typename T>
struct Raw8 {
  u32x4 w[sizeof(T) / 2];
};

// n < 8: only the first n are there, the others read as zero.
template <typename T>
__device__ __forceinline__ Raw8<T> load_raw8(const T* p, int n) {
  Raw8<T> o;
  if (n >= 8) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) o.w[k] = *(reinterpret_cast<const u32x4_u*>(p) + k);
  } else {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) o.w[k] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j < n) {
        if constexpr (sizeof(T) == 2) o.w[0][j / 2] |= (uint32_t)p[j] << (16 * (j & 1));
        else o.w[j / 4][j & 3] = __builtin_bit_cast(uint32_t, p[j]);
      }
    }
  }
  return o;
}

__device__ __forceinline__ float get8(const Raw8<uint16_t>& r, int j) {
  return (j & 1) ? bf16_hi(r.w[0][j / 2]) : bf16_lo(r.w[0][j / 2]);
}
__device__ __forceinline__ float get8(const Raw8<float>& r, int j) {
  const uint32_t w = r.w[j / 4][j & 3];      // a copy: a bit cast of a vector's element itself reads element 0
  return __builtin_bit_cast(float, w);
}

// The numbers as they lie in memory are what stays in registers between two sweeps: without this the
// compiler keeps the widened and centred ones of the first for the second, twice the registers and more.
template <typename T>
__device__ __forceinline__ void keep(Raw8<T>& o) {
#pragma unroll
  for (int k = 0; k < (int)sizeof(T) / 2; ++k) asm("" : "+v"(o.w[k]));
}

__device__ __forceinline__ void put1(float* p, float x) { *p = x; }
__device__ __forceinline__ void put1(uint16_t* p, float x) { *p = f32_to_bf16(x); }
__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ float get1(const uint16_t* p) { return bf16_to_f32(*p); }

// Two numbers rounded by one instruction (halves rounded by themselves take four to put together).
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  typedef float F2 __attribute__((ext_vector_type(2)));
  typedef __bf16 B2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((F2{lo, hi}), B2));
}

// Eight consecutive numbers written: the first `live` as they are, up to `n` as zeros.
template <typename O, bool kNT = true>
__device__ __forceinline__ void store8(O* p, const float (&v)[8], int live, int n) {
  if (live >= 8) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(O) / 2; ++k) {
      u32x4 w;
      if constexpr (sizeof(O) == 2) {
        w = u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7])};
      } else {
        w = u32x4{__builtin_bit_cast(uint32_t, v[4 * k]), __builtin_bit_cast(uint32_t, v[4 * k + 1]),
                  __builtin_bit_cast(uint32_t, v[4 * k + 2]), __builtin_bit_cast(uint32_t, v[4 * k + 3])};
      }
      u32x4_u* q = reinterpret_cast<u32x4_u*>(p) + k;
      if constexpr (kNT) __builtin_nontemporal_store((u32x4_u)w, q);
      else *q = w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < n) put1(p + j, j < live ? v[j] : 0.0f);
  }
}

__device__ __forceinline__ float sigmoid(float x) { return hw_rcp(1.0f + hw_exp2(-x * kLog2e)); }

// One lane exchange of the scans: `old` where the control reaches no lane or the row mask leaves one out.
template <int kCtrl, int kRows>
__device__ __forceinline__ float dpp(float old, float x) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, x),
                                                               kCtrl, kRows, 0xf, false));
}
__device__ __forceinline__ float lane_of(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// A stretch of the recurrence: it takes the state h in front of it to P h + H behind it.
struct Affine {
  float P = 1.0f, H = 0.0f;
};

// The stretch v, then the stretch `by`.
__device__ __forceinline__ Affine glr_through(Affine v, Affine by) {
  v.H = __builtin_fmaf(by.P, v.H, by.H);
  v.P *= by.P;
  return v;
}

// (P, H) of lanes 0 .. this one, in order, in every lane.  Four shifts inside the rows of 16
// lanes, then the rows' last lanes handed on.
__device__ __forceinline__ Affine scan_up(Affine v) {
#define GLR_STEP(ctrl, rows)                                   \
  {                                                            \
    const float p = dpp<ctrl, rows>(1.0f, v.P);                \
    const float h = dpp<ctrl, rows>(0.0f, v.H);                \
    v.H = __builtin_fmaf(v.P, h, v.H);                         \
    v.P *= p;                                                  \
  }
  GLR_STEP(0x111, 0xf)
  GLR_STEP(0x112, 0xf)
  GLR_STEP(0x114, 0xf)
  GLR_STEP(0x118, 0xf)
  GLR_STEP(0x142, 0xa)
  GLR_STEP(0x143, 0xc)
#undef GLR_STEP
  return v;
}
// The lane below's; nothing for lane 0.
__device__ __forceinline__ Affine shift_up(const Affine& v) {
  Affine o;
  o.P = dpp<0x138, 0xf>(1.0f, v.P);
  o.H = dpp<0x138, 0xf>(0.0f, v.H);
  return o;
}

// The same from lane 63 down to this one.  There is no broadcast from a row to the row below
// it, so the rows' totals travel through scalar registers.
__device__ __forceinline__ Affine scan_down(Affine v, int lane) {
#define GLR_STEP(ctrl)                                         \
  {                                                            \
    const float p = dpp<ctrl, 0xf>(1.0f, v.P);                 \
    const float h = dpp<ctrl, 0xf>(0.0f, v.H);                 \
    v.H = __builtin_fmaf(v.P, h, v.H);                         \
    v.P *= p;                                                  \
  }
  GLR_STEP(0x101)
  GLR_STEP(0x102)
  GLR_STEP(0x104)
  GLR_STEP(0x108)
#undef GLR_STEP
  const float p1 = lane_of(v.P, 16), h1 = lane_of(v.H, 16);
  const float p3 = lane_of(v.P, 48), h3 = lane_of(v.H, 48);
  const int row = lane >> 4;
  const float pa = row == 0 ? p1 : row == 2 ? p3 : 1.0f, ha = row == 0 ? h1 : row == 2 ? h3 : 0.0f;
  v.H = __builtin_fmaf(v.P, ha, v.H);
  v.P *= pa;
  const float p2 = lane_of(v.P, 32), h2 = lane_of(v.H, 32);
  const float pb = row < 2 ? p2 : 1.0f, hb = row < 2 ? h2 : 0.0f;
  v.H = __builtin_fmaf(v.P, hb, v.H);
  v.P *= pb;
  return v;
}
__device__ __forceinline__ Affine shift_down(const Affine& v) {
  Affine o;
  o.P = dpp<0x130, 0xf>(1.0f, v.P);
  o.H = dpp<0x130, 0xf>(0.0f, v.H);
  return o;
}

// State in front of segment `seg`: the initial state through the segments before it, 64 at a
// time.  sum: this row's (P, H) pairs, `stride` floats from one segment to the next.
__device__ __forceinline__ float glr_enter(const float* sum, int stride, int64_t seg, float h, int lane) {
  for (int64_t base = 0; base < seg; base += 64) {
    Affine v;
    if (base + lane < seg) {
      v.P = sum[(base + lane) * stride];
      v.H = sum[(base + lane) * stride + 1];
    }
    v = scan_up(v);
    h = __builtin_fmaf(lane_of(v.P, 63), h, lane_of(v.H, 63));
  }
  return h;
}

// Sum over the wave in lane 63 (fixed order).
__device__ __forceinline__ float wave_sum63(float x) {
  x += dpp<0x111, 0xf>(0.0f, x);
  x += dpp<0x112, 0xf>(0.0f, x);
  x += dpp<0x114, 0xf>(0.0f, x);
  x += dpp<0x118, 0xf>(0.0f, x);
  x += dpp<0x142, 0xa>(0.0f, x);
  x += dpp<0x143, 0xc>(0.0f, x);
  return x;
}

// Sum of a[i * stride] over i = y, y + 16, ... below n, eight loads under way at a time.
__device__ __forceinline__ float strided_sum(const float* a, int64_t stride, int64_t y, int64_t n) {
  float o = 0.0f;
  int64_t i = y;
  for (; i + 112 < n; i += 128) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = a[(i + 16 * k) * stride];
#pragma unroll
    for (int k = 0; k < 8; ++k) o += v[k];
  }
  for (; i < n; i += 16) o += a[i * stride];
  return o;
}

// 1 - e^(2 l) for l = x2 ln2 <= 0, a = 2^x2 given.  For |2 l| < 1/8 the Taylor series to
// (2 l)^5 (truncation below (1/8)^5 / 720 = 4.3e-8 relative); otherwise 1 - a^2 in one rounding,
// where the error of a (about one unit of 2^-24) is at most 1e-6 of the result, 5e-7 of its root.
__device__ __forceinline__ float glr_rest(float x2, float a) {
  const float y = x2 * (2.0f * kLn2);
  float p = __builtin_fmaf(y, 1.0f / 120.0f, 1.0f / 24.0f);
  p = __builtin_fmaf(y, p, 1.0f / 6.0f);
  p = __builtin_fmaf(y, p, 0.5f);
  p = __builtin_fmaf(y, p, 1.0f);
  return y > -0.125f ? -y * p : __builtin_fmaf(-a, a, 1.0f);
}

// 1 - s of a sigmoid s = 1 / (1 + e), as e s: right to its own last bits where the difference would have 2^-24 of 1.  e may be
// infinite where s is 0.
__device__ __forceinline__ float one_less(float s, float e) { return s == 0.0f ? 1.0f : e * s; }

// The gates of a token.
struct GlrGate {
  float a, n, s, c;   // decay, input factor, sigmoid of r and one less it
  float ra;           // a^2 / n: minus the derivative of n with respect to log a (decay rule)
};

// nb: -bias log2(e); A2: A log2(e), both as glr_channel holds them.  r = -inf stands for a token that is not there: s = 0, a = 1.
// Decay rule: n is held to 3e-19 or more, so that its reciprocal stays finite where s underflows.
template <bool kBlend>
__device__ __forceinline__ GlrGate glr_gate(float r, float nb, float A2) {
  GlrGate o;
  const float e = hw_exp2(__builtin_fmaf(r, -kLog2e, nb));
  o.s = hw_rcp(1.0f + e);
  o.c = one_less(o.s, e);
  if constexpr (kBlend) {
    o.a = o.c;
    o.n = o.s;
    o.ra = 0.0f;
  } else {
    const float x2 = A2 * o.s;
    o.a = hw_exp2(x2);
    float q = glr_rest(x2, o.a);
    // a comparison, so that a NaN stays one; of the size, so that A > 0 (below zero by 2 A s) gives a NaN
    q = __builtin_fabsf(q) < 1e-37f ? 1e-37f : q;
    const float rs = __builtin_amdgcn_rsqf(q);
    o.n = q * rs;
    o.ra = o.a * o.a * rs;
  }
  return o;
}

// Tokens of batch row b that count: all L, or lengths[b] held to 0 .. L.
__device__ __forceinline__ int64_t glr_length(const GlrParams& p, int64_t b) {
  if (!p.lengths) return p.L;
  const int64_t n = p.lengths[b];
  return n < 0 ? 0 : n > p.L ? p.L : n;
}

// A channel's parameters as the gates of a row of `len` tokens take them: A, A log2(e), -bias log2(e).  Kept finite, so that a token
// that is not there (r = -inf, zeros) stays absent, s = 0 and a = 1, for gates that an infinite bias holds open and for A = -inf.
// A row without tokens looks at none of them.
struct GlrChannel {
  float A = 0.0f, A2 = 0.0f, rb = 0.0f, ib = 0.0f;
};
template <bool kBlend>
__device__ __forceinline__ GlrChannel glr_channel(const GlrParams& p, int64_t d, int64_t len) {
  GlrChannel o;
  if (len == 0) return o;
  auto held = [](float v) { return v < -2e38f ? -2e38f : v; };     // a comparison, so that a NaN stays one
  if constexpr (!kBlend) {
    o.A = held(p.A[d]);
    o.A2 = o.A * kLog2e;
  }
  if (p.r_bias) o.rb = held(-p.r_bias[d] * kLog2e);
  if (p.i_bias) o.ib = -p.i_bias[d] * kLog2e;
  return o;
}

__device__ __forceinline__ int clamp8(int64_t n) { return n < 0 ? 0 : n > 8 ? 8 : (int)n; }

// r of a token that is not there.
template <typename T>
__device__ __forceinline__ float glr_r(const Raw8<T>& r, int j, int live) {
  return j < live ? get8(r, j) : -__builtin_inff();
}

// A lane's 8 tokens of a row: from t on, its own ones lo .. lo + there, the first `live` of which count.  The last lane of
// a row of 8 tokens or more takes the row's last 8, so that it loads them whole like every other; those that the lane before
// it has too (the first `lo`) are left out like those behind the row's length: r = -inf (s = 0, a = 1) and zeros
// in the other inputs.  (Token by token that lane holds its wave up: 20480 rows, L = 2047, bf16: forward 174 us, so 98,
// backward 358, 204.)
struct Share {
  int64_t t;
  int lo, there, live;
  uint32_t on;                  // a bit for each token that counts
};

// Of a row of L tokens, `len` of which count, the 8 from `first` on; the stretch ends at t1 (L, or a multiple of 8).
__device__ __forceinline__ Share glr_share(int64_t L, int64_t t1, int64_t len, int64_t first) {
  Share o;
  const int64_t last = L - kGlrLane, end = len < t1 ? len : t1;
  o.t = last < 0 ? 0 : first < last ? first : last;
  o.there = clamp8(t1 - first);
  o.live = clamp8(end - first);
  o.lo = o.there ? (int)(first - o.t) : 0;
  o.on = ((1u << o.live) - 1) << o.lo;
  return o;
}

// `dead`: the bits in the place of tokens that do not count.
template <typename T>
__device__ __forceinline__ Raw8<T> load_share(const T* row, int64_t L, const Share& q, uint32_t dead) {
  Raw8<T> o;
  if (L >= kGlrLane) {
#pragma unroll
    for (int k = 0; k < (int)sizeof(T) / 2; ++k) o.w[k] = *(reinterpret_cast<const u32x4_u*>(row + q.t) + k);
  } else {
    o = load_raw8(row, (int)L);
  }
  if (q.on != 0xff) {
#pragma unroll
    for (int j = 0; j < 4 * (int)sizeof(T); j += 2) {
      const int e = sizeof(T) == 2 ? j : j / 2;          // the word's first (or only) token
      uint32_t w = o.w[j / 8][j / 2 & 3];
      if constexpr (sizeof(T) == 2) {
        const uint32_t m = (q.on >> e & 1 ? 0xffffu : 0u) | (q.on >> (e + 1) & 1 ? 0xffff0000u : 0u);
        w = (w & m) | (dead & ~m);
      } else {
        w = q.on >> e & 1 ? w : dead;
      }
      o.w[j / 8][j / 2 & 3] = w;
    }
  }
  return o;
}
template <typename T>
constexpr uint32_t kMinusInf = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;

// The lane's own tokens, zeros for those that do not count.
template <typename O, bool kNT>
__device__ __forceinline__ void store_share(O* row, const float (&v)[8], const Share& q) {
  if (q.live == 8) {
    store8<O, kNT>(row + q.t, v, 8, 8);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j >= q.lo && j < q.lo + q.there) put1(row + q.t + j, j < q.lo + q.live ? v[j] : 0.0f);
  }
}

}  // namespace mamba
