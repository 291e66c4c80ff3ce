// gdr_step.hip -- the gated delta rule token by token (gfx950): one token per
// sequence on a pool of states (decoding), and short sequences.
//
// Per value head, with state S (P x N), a = exp(A delta), b = sigmoid(beta_raw):
//   S' = a S;  u = b (v - S' k);  S = S' + u k^T;  y = scale S q.
// Both products of a token are taken on the old state, in one pass over it:
//   S' k = a (S k),   S q = a (S q) + u (k . q),
// so that a token reads and writes every number of the state once.  The rows
// of S (value channels) are independent given k and q: 16 lanes share a row,
// each with kE = 4 or 8 of its N <= 128 numbers in registers, a wave has four
// rows (times kSets), and the two sums over a row are four lane exchanges.
//
// One token moves 8 bytes per number of the state (fp32 read and written in
// place) and computes 7 flops on it: HBM-bound, like mamba_state_update.  128 rows of 32
// heads of 128 x 128: 116 us, 4.6 TB/s (a large copy: 4.78).  Sequences are read one number
// per lane at a stride of L, which is slow where L is a multiple of 4: 32 heads, L = 15, 16, 17: 27,
// 38, 30 us.
#include "device_math.hpp"
#include "gdr.hpp"
#include "kernels.hpp"

namespace mamba {
namespace {

// kVec: N % 4 == 0 and the states 16-byte aligned.
template <typename T, typename O, int kE, bool kVec, int kSets>
__global__ __launch_bounds__(256) void gdr_step_kernel(GdrParams p) {
  const int lane = threadIdx.x & 63, c = lane & 15;
  const int64_t wave = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int64_t tiles = (p.P + 4 * kSets - 1) / (4 * kSets);
  const int64_t bh = wave / tiles;
  if (bh >= p.B * p.H) return;
  const int64_t b = bh / p.H, h = bh % p.H, g = h / (p.H / p.G);
  const int64_t row0 = (wave % tiles) * (4 * kSets) + (lane >> 4);
  int64_t slot = b;
  if (p.slots) slot = p.slots[b];
  const bool live = slot >= 0 && slot < p.n_slots;       // uniform over the wave
  const int64_t len = live ? gdr_length(p, b) : 0;

  const T* q = static_cast<const T*>(p.q) + b * p.q_stride + g * p.N * p.L;
  const T* k = static_cast<const T*>(p.k) + b * p.k_stride + g * p.N * p.L;
  const T* v = static_cast<const T*>(p.v) + b * p.v_stride + h * p.P * p.L;
  const T* dl = static_cast<const T*>(p.delta) + bh * p.L;
  const T* be = static_cast<const T*>(p.beta) + bh * p.L;
  O* y = static_cast<O*>(p.y) + bh * p.P * p.L;

  float S[kSets][kE];
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int64_t row = row0 + 4 * s;
    const float* src = p.init ? p.init + ((live ? slot : 0) * p.H + h) * p.P * p.N + row * p.N : nullptr;
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const int64_t n = 16 * e + 4 * c;
      if constexpr (kVec) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (src && live && row < p.P && n < p.N) x = *reinterpret_cast<const float4*>(src + n);
        S[s][e] = x.x; S[s][e + 1] = x.y; S[s][e + 2] = x.z; S[s][e + 3] = x.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) S[s][e + j] = (src && live && row < p.P && n + j < p.N) ? src[n + j] : 0.0f;
      }
    }
  }
  const float A = p.A[h], bias = p.bias ? p.bias[h] : 0.0f;
  for (int64_t t = 0; t < len; ++t) {
    float kv[kE], qv[kE], vv[kSets];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      const int64_t n = 16 * (e & ~3) + 4 * c + (e & 3);
      kv[e] = n < p.N ? gdr_load(k + n * p.L + t) : 0.0f;
      qv[e] = n < p.N ? gdr_load(q + n * p.L + t) : 0.0f;
    }
#pragma unroll
    for (int s = 0; s < kSets; ++s) vv[s] = row0 + 4 * s < p.P ? gdr_load(v + (row0 + 4 * s) * p.L + t) : 0.0f;
    const float a = gdr_decay(gdr_load(dl + t) + bias, A);
    const float bt = gdr_sigmoid(gdr_load(be + t));
    float kk = 0.0f, qq = 0.0f, kq = 0.0f;
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      kk = __builtin_fmaf(kv[e], kv[e], kk);
      qq = __builtin_fmaf(qv[e], qv[e], qq);
      kq = __builtin_fmaf(kv[e], qv[e], kq);
    }
    float rk = 1.0f, rq = p.scale;
    if (p.norm) {
      rk = gdr_rnorm(gdr_sum16(kk));
      rq *= gdr_rnorm(gdr_sum16(qq));
    }
    kq = gdr_sum16(kq) * rk * rq;
#pragma unroll
    for (int s = 0; s < kSets; ++s) {
      float sk = 0.0f, sq = 0.0f;
#pragma unroll
      for (int e = 0; e < kE; ++e) {
        sk = __builtin_fmaf(S[s][e], kv[e], sk);
        sq = __builtin_fmaf(S[s][e], qv[e], sq);
      }
      sk = gdr_sum16(sk);
      sq = gdr_sum16(sq);
      const float u = bt * (vv[s] - a * rk * sk);
      const float w = u * rk;
#pragma unroll
      for (int e = 0; e < kE; ++e) S[s][e] = __builtin_fmaf(w, kv[e], a * S[s][e]);
      const float o = __builtin_fmaf(a * rq, sq, u * kq);
      if (c == 0 && row0 + 4 * s < p.P) gdr_store(y + (row0 + 4 * s) * p.L + t, o);
    }
  }
  // tokens past the end of a padded row (the whole row when it has no slot)
  for (int64_t t = len + c; t < p.L; t += 16) {
#pragma unroll
    for (int s = 0; s < kSets; ++s)
      if (row0 + 4 * s < p.P) gdr_store(y + (row0 + 4 * s) * p.L + t, 0.0f);
  }
  if (!p.final_state || !live) return;
#pragma unroll
  for (int s = 0; s < kSets; ++s) {
    const int64_t row = row0 + 4 * s;
    if (row >= p.P) continue;
    float* dst = p.final_state + ((slot * p.H + h) * p.P + row) * p.N;
#pragma unroll
    for (int e = 0; e < kE; e += 4) {
      const int64_t n = 16 * e + 4 * c;
      if constexpr (kVec) {
        if (n < p.N) *reinterpret_cast<float4*>(dst + n) = make_float4(S[s][e], S[s][e + 1], S[s][e + 2], S[s][e + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (n + j < p.N) dst[n + j] = S[s][e + j];
      }
    }
  }
}

template <typename T, typename O, int kE, bool kVec, int kSets>
hipError_t step_launch(const GdrParams& p, hipStream_t s) {
  hipLaunchKernelGGL((gdr_step_kernel<T, O, kE, kVec, kSets>), dim3((unsigned)gdr_step_workgroups(p)), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t step_t(const GdrParams& p, hipStream_t s) {
  const bool wide = p.N > 64, many = gdr_step_sets(p) == 4;
  if (!p.state_vec) return wide ? step_launch<T, O, 8, false, 1>(p, s) : step_launch<T, O, 4, false, 1>(p, s);
  if (wide) return many ? step_launch<T, O, 8, true, 4>(p, s) : step_launch<T, O, 8, true, 1>(p, s);
  return many ? step_launch<T, O, 4, true, 4>(p, s) : step_launch<T, O, 4, true, 1>(p, s);
}

}  // namespace

hipError_t launch_gdr_step(const GdrParams& p, Dt in, Dt out, hipStream_t s) {
  if (in == Dt::BF16) return out == Dt::BF16 ? step_t<uint16_t, uint16_t>(p, s) : step_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? step_t<float, uint16_t>(p, s) : step_t<float, float>(p, s);
}

}  // namespace mamba
