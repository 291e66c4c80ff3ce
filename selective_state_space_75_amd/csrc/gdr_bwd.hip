// gdr_bwd.hip -- gradients of the gated delta rule over sequences (gfx950).
//
// Notation of gdr_chunk.hip, for one chunk with entering state S0 and the gradient
// dS of the state that leaves it (unit keys and queries when they are normalised):
//   updates  u = T (V - exp(G) K S0^T)
//   dV  = T^T (E K dS^T + Pm^T dY),  E = diag exp(G_C - G), Pm the scaled query matrix
//   dS0 = exp(G_C) dS + (s exp(G) dY)^T Q - (exp(G) dV)^T K
//   M1 = s tril(D o dY U^T),  M2 = stril(D o dV U^T)
//   dQ  = s exp(G) dY S0 + M1 K
//   dK  = E U dS + M1^T Q - (M2 + M2^T) K - exp(G) dV S0
//   dbeta_raw_t = (dV_t . U_t) / b_t (1 - b_t)         (u = b (v - p), dV = b du)
// The gradient of token t's log decay is everything that passes from before t to t
// or after it:
//   dg_t = sum_(i >= t > j) [M1_ij q_i.k_j - M2_ij k_i.k_j] + sum_(i >= t) X_i
//          + sum_(j < t) Y_j + exp(G_C) <dS, S0>,
//   X_i = q_i . (s exp(G) dY S0)_i - k_i . (exp(G) dV S0)_i,  Y_j = k_j . (E U dS)_j.
// (The shorter identity dg_t = <dS, S> + sum_(i >= t) (q_i . dQ_i - v_i . dV_i) subtracts
// the tokens' own terms again, which are larger than what is left: it loses an order
// of magnitude in fp32 and the sums over tokens lose more.)
//
// Five launches after the preparation (gdr_chunk.hip, which leaves T, T^T, Pm^T):
//   states  forward along L: U of every chunk, S at every block of 4 chunks;
//   adjoint backward along L: dV and dS of every chunk;
//   pairs   all chunks at once: M1 and M2 as operands (over T's planes, which are not
//           needed any more), and what of dg and dbeta follows from them alone;
//   grads   all blocks at once: the states inside a block are rebuilt forward from S,
//           everything else is products;
//   sums    dA and ddelta_bias from the blocks' partial sums, in a fixed order.
// The chains are cut over value channels (16 per wave, gdr_chunk.hip); the grads
// launch is cut over the N numbers of the keys (16 per wave), where dQ and dK are
// sums over value channels that stay inside a wave.  One workgroup takes all value
// heads of a key head, so dQ and dK need no reduction between workgroups.
//
// Measured after warm-up, bf16, 40 heads of 128 x 128, batch 4, L = 2048 (422 MB, 88 us at a large
// copy's rate): preparation 72 us, states 225, adjoint 451, pairs 174, grads 588, sums 5; the call
// 1.52 ms, 5.6 GB of HBM traffic.  The chains are bound as the forward's (320 workgroups on 256
// CUs); the adjoint also writes dS of every chunk (671 MB) so that the grads need no second
// backward sweep.  The grads hold S and dS in registers, which leaves one workgroup per CU,
// and the variant with 128 channels a slab spills 11 vector and 136 scalar registers.
#include "gdr_mfma.hpp"

namespace mamba {
namespace {

// ----------------------------------------------------------------------------- adjoint chain
template <typename T, typename O, int kN>
__global__ __launch_bounds__(256, 2) void gdr_adjoint_kernel(GdrChunkParams p) {
  constexpr int kParts = GdrIn<T>::kParts;
  constexpr int kGParts = GdrIn<O>::kParts;
  constexpr int kTile = kN * kGdrRow * kParts;
  constexpr int kNT = kN / 16, kNB = kN / 32;
  constexpr int kBuf = kParts == 1 ? 2 : 1;
  __shared__ __align__(16) uint16_t Kt[kBuf][kTile];
  __shared__ __align__(16) uint16_t Qt[kBuf][kTile];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15, g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t slices = (q.P + 63) / 64;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);
  const int64_t slice = it % slices, h = (it / slices) % q.H, b = it / (slices * q.H);
  const int64_t bh = b * q.H + h, g = h / (q.H / q.G);
  const int64_t ch = slice * 64 + 16 * w + i16;
  const bool mine = ch < q.P, some = slice * 64 + 16 * w < q.P;
  const int64_t vch = mine ? ch : q.P - 1;       // lanes past the last channel run along on it
  const int64_t len = gdr_length(q, b), ce = (len + kC - 1) / kC;

  const T* krows = static_cast<const T*>(q.k) + b * q.k_stride + g * q.N * q.L;
  const T* qrows = static_cast<const T*>(q.q) + b * q.q_stride + g * q.N * q.L;
  const T* tail_k = static_cast<const T*>(p.tail_k) + (b * q.G + g) * q.N * kC;
  const T* tail_q = static_cast<const T*>(p.tail_q) + (b * q.G + g) * q.N * kC;
  const O* dyrow = static_cast<const O*>(p.dy) + (bh * q.P + vch) * q.L + 4 * g4;
  const O* tail_dy = static_cast<const O*>(p.tail_dy) + (bh * q.P + vch) * kC + 4 * g4;
  O* dvrow = static_cast<O*>(p.dv) + (bh * q.P + vch) * q.L;
  const int64_t blk0 = block_of(p, b, h, 0), Pp = slices * 64;
  const uint16_t* planes = p.planes + blk0 * 9 * kGdrPlane;
  const float* vec = p.vec + blk0 * p.vec_stride;

  f32x4 S[kNT];                                  // dS: column ch, rows of the key numbers
#pragma unroll
  for (int tn = 0; tn < kNT; ++tn) {
    S[tn] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (p.dfinal) S[tn] = gdr_load_state(p.dfinal + (bh * q.P + vch) * q.N, 16 * tn + 4 * g4, q.N, q.state_vec);
  }

  bf16x8 tf[2][3], pf[2][3];
  typename GdrIn<O>::Four dy[2];
  f32x4 fk[2], fq[2], fu[2];
  float dec = 0.0f;
  GdrTile<T, kN> tk, tq;
  tk.init(q.N, tid);
  tq.init(q.N, tid);
  auto load_tiles = [&](int64_t c) {
    const GdrChunkSrc<T> sk(krows, q.L, tail_k, c, len), sq(qrows, q.L, tail_q, c, len);
    tk.load(sk.at, sk.stride, tid);
    tq.load(sq.at, sq.stride, tid);
  };
  auto load_rest = [&](int64_t c) {
    const O* src = (c + 1) * kC <= len ? dyrow + c * kC : tail_dy;
    dy[0].load(src);
    dy[1].load(src + 16);
    const uint16_t* pl = planes + c * 9 * kGdrPlane;
    const float* vc = vec + c * p.vec_stride;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
#pragma unroll
      for (int s = 0; s < 3; ++s) {
        tf[rt][s] = lane_load<bf16x8>(pl + (3 + s) * kGdrPlane + rt * 512, lane * 16);
        pf[rt][s] = lane_load<bf16x8>(pl + (6 + s) * kGdrPlane + rt * 512, lane * 16);
      }
      fk[rt] = lane_load<f32x4>(vc + 16 * rt, g4 * 16);
      fq[rt] = lane_load<f32x4>(vc + 32 + 16 * rt, g4 * 16);
      fu[rt] = lane_load<f32x4>(vc + 64 + 16 * rt, g4 * 16);
    }
    dec = vec[c * p.vec_stride + 96];
  };
  if (ce > 0) {
    load_tiles(ce - 1);
    tk.put(Kt[0], tid);
    tq.put(Qt[0], tid);
    load_rest(ce - 1);
    __syncthreads();
  }
  for (int64_t c = ce - 1; c >= 0; --c) {
    const int buf = kBuf == 2 ? (int)((ce - 1 - c) & 1) : 0;
    const uint16_t *K = Kt[buf], *Q = Qt[buf];
    const int64_t cn = c > 0 ? c - 1 : 0;                  // the first chunk loads itself again
    load_tiles(cn);
    {
      // in tiles of 16 channels x 16 keys: 1 KB a store, and what a wave of the grads reads
      float* dst = p.chunk_dS + ((blk0 + c) * Pp + slice * 64 + 16 * w) * kN + 16 * i16 + 4 * g4;
#pragma unroll
      for (int tn = 0; tn < kNT; ++tn)
        *reinterpret_cast<f32x4*>(dst + 256 * tn) = mine ? S[tn] : f32x4{0.f, 0.f, 0.f, 0.f};
    }
    // right-hand side E K dS^T + Pm^T dY
    f32x4 R[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
    bf16x8 ka[2][2][kParts];
    auto load_a = [&](int kb) {
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) gdr_frags_t<T, kN>(K, 32 * kb, 16 * rt, lane, ka[kb & 1][rt]);
    };
    load_a(0);
#pragma unroll
    for (int kb = 0; kb < kNB; ++kb) {
      if (kb + 1 < kNB) load_a(kb + 1);
      bf16x8 sb[3];
      gdr_split<3>(S[2 * kb], S[2 * kb + 1], sb);
      gdr_mma_rows<3>(ka[kb & 1], sb, R);
      __builtin_amdgcn_sched_barrier(0);
    }
    const f32x4 d0 = dy[0].get(), d1 = dy[1].get();
    bf16x8 db[kGParts];
    gdr_split<kGParts>(d0, d1, db);
    R[0] *= fu[0];
    R[1] *= fu[1];
    gdr_mma_rows<3>(pf, db, R);
    bf16x8 rb[3];
    gdr_split<3>(R[0], R[1], rb);
    f32x4 W[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};     // dV
    gdr_mma_rows<3>(tf, rb, W);
    bf16x8 wk[3], wq[3];
    gdr_split<3>(-fk[0] * W[0], -fk[1] * W[1], wk);
    gdr_split<3>(fq[0] * d0, fq[1] * d1, wq);
    const float dc = dec;
    load_rest(cn);
#pragma unroll
    for (int tn = 0; tn < kNT; ++tn) {
      bf16x8 a[kParts], aq[kParts];
      gdr_frags<T, kN>(K, 16 * tn, 0, lane, a);
      gdr_frags<T, kN>(Q, 16 * tn, 0, lane, aq);
      // Summed from zero and added once: on top of dS each of the six products would round at
      // its size (dA, a sum over tokens that cancels, was 1.5 times as far off, and 10 us went
      // into waiting for the accumulators).
      const f32x4 x = gdr_mma<3>(aq, wq, f32x4{0.f, 0.f, 0.f, 0.f});
      S[tn] = gdr_fma(S[tn], f32x4{dc, dc, dc, dc}, gdr_mma<3>(a, wk, x));
    }
    float* wdst = p.dvw + ((blk0 + c) * Pp + ch) * kC + 4 * g4;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
      *reinterpret_cast<f32x4*>(wdst + 16 * rt) = mine ? W[rt] : f32x4{0.f, 0.f, 0.f, 0.f};
    if (some && (c + 1) * kC <= len) {                     // (the chunk of the row's end: after the loop)
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) gdr_store_whole4(dvrow + c * kC + 16 * rt + 4 * g4, W[rt]);
    }
    if constexpr (kBuf == 1) __syncthreads();
    tk.put(Kt[kBuf == 2 ? buf ^ 1 : 0], tid);
    tq.put(Qt[kBuf == 2 ? buf ^ 1 : 0], tid);
    __syncthreads();
  }
  if (p.dinit) {
    const int64_t ch0 = slice * 64 + 16 * w;
    gdr_store_rows(p.dinit + (bh * q.P + ch0) * q.N, q.P - ch0, q.N, q.state_vec, S, lane);
  }
  if (mine) {
    if (ce * kC > len) {
      const float* wsrc = p.dvw + ((blk0 + ce - 1) * Pp + ch) * kC + 4 * g4;
      const f32x4 W[2] = {*reinterpret_cast<const f32x4*>(wsrc), *reinterpret_cast<const f32x4*>(wsrc + 16)};
      gdr_store_end(dvrow, (ce - 1) * kC, len, q.L, W, g4);
    }
    // tokens behind the row's end
    for (int64_t t = ce * kC + 4 * g4; t < q.L; t += 16) gdr_store4(dvrow, t, q.L, f32x4{0.f, 0.f, 0.f, 0.f});
  }
}

// ----------------------------------------------------------------------------- the rest, block by block
// kRows rows of 32 tokens, loaded by the workgroup into registers and put into operand
// planes later; rows past the last one are zeros.
template <typename T, int kRows, int kThreads>
struct Rows {
  static constexpr int kCount = (kRows * 4 + kThreads - 1) / kThreads;
  static constexpr bool kSome = kRows * 4 % kThreads != 0;     // fewer pieces than threads
  typename GdrIn<T>::Raw raw[kCount];
  __device__ __forceinline__ void load(const T* src, int64_t stride, int64_t rows, int tid) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int64_t n = (tid + kThreads * j) >> 2;
      raw[j].whole(src + (n < rows ? n : rows - 1) * stride + 8 * (tid & 3));
    }
  }
  // all kRows rows, one after the other
  __device__ __forceinline__ void load_dense(const T* src, int tid) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int id = tid + kThreads * j;
      raw[j].whole(reinterpret_cast<const T*>(reinterpret_cast<const char*>(src) +
                                              (uint32_t)(kSome && id >= kRows * 4 ? 0 : id) * 8u * sizeof(T)));
    }
  }
  __device__ __forceinline__ void put(uint16_t* tile, int rows, int tid) const {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int n = (tid + kThreads * j) >> 2;
      static_assert(kRows % 16 == 0, "a wave has 16 rows or none");
      if (kSome && __builtin_amdgcn_readfirstlane(n) >= kRows) continue;
      uint16_t* dst = tile + n * kGdrRow + 8 * (tid & 3);
      raw[j].template put<kRows * kGdrRow>(dst, rows == kRows || n < rows ? ~0u : 0u);
    }
  }
};

template <int kParts, int kRows>
__device__ __forceinline__ void plane_frags_t(const uint16_t* tile, int row0, int col0, int lane, bf16x8 (&f)[kParts]) {
#pragma unroll
  for (int s = 0; s < kParts; ++s) f[s] = gdr_frag_t<kGdrRow>(tile + s * kRows * kGdrRow, row0, col0, lane);
}
template <int kParts, int kRows>
__device__ __forceinline__ void plane_frags(const uint16_t* tile, int row0, int col0, int lane, bf16x8 (&f)[kParts]) {
#pragma unroll
  for (int s = 0; s < kParts; ++s) f[s] = gdr_frag<kGdrRow>(tile + s * kRows * kGdrRow, row0, col0, lane);
}

// Four tokens 16 rt + 4 g .. of row n of a tile as fp32 (the parts added up).
template <int kParts, int kRows>
__device__ __forceinline__ f32x4 tile_four(const uint16_t* tile, int n, int t) {
  f32x4 r = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = kParts - 1; s >= 0; --s) {
    const uint2 x = *reinterpret_cast<const uint2*>(tile + s * kRows * kGdrRow + n * kGdrRow + t);
    r += f32x4{bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y)};
  }
  return r;
}

// One workgroup per (batch row, value head, chunk): the 32 x 32 products dV U^T, dY U^T
// (64 value channels at a time), K K^T and Q K^T, lower tiles only.  Leaves M1 (columns
// times 1/|k|), M1^T (times 1/|q|) and -(M2 + M2^T) (times 1/|k|) as operand planes of
// the products with K and Q, and per token the pairs' part of dg and dV_t . U_t / b_t.
template <typename T, typename O, int kN>
__global__ __launch_bounds__(256) void gdr_pair_kernel(GdrChunkParams p) {
  constexpr int kParts = GdrIn<T>::kParts, kGParts = GdrIn<O>::kParts, kPS = 64;
  __shared__ __align__(16) uint16_t dOt[kGParts * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t dVt[3 * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t Ut[3 * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t Kt[kParts * kN * kGdrRow];
  __shared__ __align__(16) uint16_t Qt[kParts * kN * kGdrRow];
  __shared__ float m[4][32 * 33];                          // M2, M1, Q K^T, K K^T
  __shared__ double cum[32];
  __shared__ __align__(16) float rk[32], rq[32], dvu[33];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15,
            g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);
  const int64_t c = it % p.n_chunks, bh = it / p.n_chunks, b = bh / q.H, h = bh % q.H, g = h / (q.H / q.G);
  const int64_t len = gdr_length(q, b), bg = b * q.G + g;
  if (c * kC >= len) return;
  const int64_t bl = block_of(p, b, h, c), Pp = (q.P + 63) / 64 * 64;
  float* vec = p.vec + bl * p.vec_stride;
  const GdrChunkSrc<T> sk(static_cast<const T*>(q.k) + b * q.k_stride + g * q.N * q.L, q.L,
                          static_cast<const T*>(p.tail_k) + bg * q.N * kC, c, len);
  const GdrChunkSrc<T> sq(static_cast<const T*>(q.q) + b * q.q_stride + g * q.N * q.L, q.L,
                          static_cast<const T*>(p.tail_q) + bg * q.N * kC, c, len);
  const GdrChunkSrc<O> sy(static_cast<const O*>(p.dy) + bh * q.P * q.L, q.L,
                          static_cast<const O*>(p.tail_dy) + bh * q.P * kC, c, len);
  Rows<O, kPS, 256> ldo;
  Rows<float, kPS, 256> ldv, ldu;
  auto load = [&](int64_t p0) {
    ldo.load(sy.at + p0 * sy.stride, sy.stride, q.P - p0 < kPS ? q.P - p0 : kPS, tid);
    ldv.load_dense(p.dvw + (bl * Pp + p0) * kC, tid);
    ldu.load_dense(p.u + (bl * Pp + p0) * kC, tid);
  };
  float braw;
  {
    Rows<T, kN, 256> ldk, ldq;
    ldk.load(sk.at, sk.stride, q.N, tid);
    ldq.load(sq.at, sq.stride, q.N, tid);
    const double lcum = lane_load<double>(vec + 192, (lane & 31) * 8);
    const float lrk = lane_load<float>(vec + 128, (lane & 31) * 4), lrq = lane_load<float>(vec + 160, (lane & 31) * 4);
    const int64_t tok = c * kC + (lane & 31);
    braw = gdr_load(static_cast<const T*>(q.beta) + bh * q.L + (tok < len ? tok : len - 1));
    load(0);
    ldk.put(Kt, (int)q.N, tid);
    ldq.put(Qt, (int)q.N, tid);
    if (w == 0) {
      cum[lane & 31] = lcum;
      rk[lane & 31] = lrk;
      rq[lane & 31] = lrq;
    }
  }
  // tile t of the lower triangle: rows 16 (t > 0), columns 16 (t > 1)
  f32x4 acc[3];                                            // waves 0 to 2: tile w of dV U^T; wave 3: dY U^T
#pragma unroll
  for (int t = 0; t < 3; ++t) acc[t] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int64_t p0 = 0; p0 < q.P; p0 += kPS) {
    const int rows = (int)(q.P - p0 < kPS ? q.P - p0 : kPS);
    if (p0 > 0) __syncthreads();
    ldo.put(dOt, rows, tid);
    ldv.put(dVt, kPS, tid);
    ldu.put(Ut, kPS, tid);
    if (p0 + kPS < q.P) load(p0 + kPS);
    __syncthreads();
    if (w < 3) {
      const int rt = w > 0, ct = w > 1;
#pragma unroll
      for (int kb = 0; kb < kPS / 32; ++kb) {
        bf16x8 a[3], u[3];
        plane_frags_t<3, kPS>(dVt, 32 * kb, 16 * rt, lane, a);
        plane_frags_t<3, kPS>(Ut, 32 * kb, 16 * ct, lane, u);
        acc[0] = gdr_mma<3>(a, u, acc[0]);
      }
    } else {
#pragma unroll
      for (int kb = 0; kb < kPS / 32; ++kb) {
        bf16x8 a[2][kGParts], u[2][3];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          plane_frags_t<kGParts, kPS>(dOt, 32 * kb, 16 * t, lane, a[t]);
          plane_frags_t<3, kPS>(Ut, 32 * kb, 16 * t, lane, u[t]);
        }
        acc[0] = gdr_mma<3>(a[0], u[0], acc[0]);
        acc[1] = gdr_mma<3>(a[1], u[0], acc[1]);
        acc[2] = gdr_mma<3>(a[1], u[1], acc[2]);
      }
    }
  }
  auto put = [&](int kind, int t, f32x4 v) {
    const int j = (t > 1 ? 16 : 0) + i16;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = (t > 0 ? 16 : 0) + 4 * g4 + r;
      float x = v[r];
      if (kind == 0) dvu[i == j ? i : 32] = x;             // dV_t . U_t (32: dropped)
      if (kind < 2) {
        const float d = hw_exp2((float)(cum[i] - cum[j]));
        x = (kind == 0 ? i > j : i >= j) ? x * d * (kind == 0 ? 1.0f : q.scale) : 0.0f;
      }
      m[kind][i * 33 + j] = x;
    }
  };
  if (w < 3) {
    put(0, w, acc[0]);
#pragma unroll
    for (int kind = 2; kind < 4; ++kind) {
      const uint16_t* rows = kind == 2 ? Qt : Kt;
      const int rt = w > 0, ct = w > 1;
      f32x4 x = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kb = 0; kb < kN / 32; ++kb) {
        bf16x8 a[kParts], k[kParts];
        gdr_frags_t<T, kN>(rows, 32 * kb, 16 * rt, lane, a);
        gdr_frags_t<T, kN>(Kt, 32 * kb, 16 * ct, lane, k);
        x = gdr_mma<3>(a, k, x);
      }
      put(kind, w, x);
    }
  } else {
#pragma unroll
    for (int t = 0; t < 3; ++t) put(1, t, acc[t]);
  }
  __syncthreads();
  if (w < 3) {
    // operands (kind w), the lengths of the contracted rows folded in; read first, chosen
    // afterwards (what the upper tile holds is dropped)
    const float* mk = m[w == 2 ? 0 : 1];
    const f32x4* lens = reinterpret_cast<const f32x4*>(w == 1 ? rq : rk);
    const f32x4 l0 = lens[g4], l1 = lens[4 + g4];
    uint16_t* planes = p.planes + (bl * 9 + 3 * w) * kGdrPlane;
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const int row = 16 * rt + i16;
      f32x4 x[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = (e < 4 ? 0 : 16) + 4 * g4 + (e & 3);
        const int hi = row > col ? row : col, lo = row > col ? col : row;
        const float v = mk[hi * 33 + lo] * (e < 4 ? l0 : l1)[e & 3];
        const bool in = w == 0 ? row >= col : w == 1 ? col >= row : row != col;
        x[e >> 2][e & 3] = in ? (w == 2 ? -v : v) : 0.0f;
      }
      bf16x8 f[3];
      gdr_split<3>(x[0], x[1], f);
#pragma unroll
      for (int s = 0; s < 3; ++s) *reinterpret_cast<bf16x8*>(planes + s * kGdrPlane + rt * 512 + lane * 8) = f[s];
    }
  } else {
    // the pairs across each token: lane (half, j) has rows 16 half .. + 15 of column j and
    // walks them from the last up
    const int j = lane & 31, half = lane >> 5;
    float wv[16], all = 0.0f;
    const float kj = rk[j];
#pragma unroll
    for (int t16 = 0; t16 < 16; ++t16) {
      const int t = 16 * half + t16, at = t * 33 + j;
      const float v = m[1][at] * rq[t] * m[2][at] - m[0][at] * rk[t] * m[3][at];
      wv[t16] = t > j ? kj * v : 0.0f;                     // (the upper tile holds nothing)
      all += wv[t16];
    }
    const float above = __shfl_xor(all, 32);
    float s0 = half ? 0.0f : above;
    wave_sync();                                           // m[3] is this wave's from here on
#pragma unroll
    for (int t16 = 15; t16 >= 0; --t16) {
      const int t = 16 * half + t16;
      s0 += wv[t16];
      m[3][t * 33 + j] = j < t ? s0 : 0.0f;
    }
    wave_sync();
    float s1 = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) s1 += m[3][j * 33 + 16 * half + k];
    s1 += __shfl_xor(s1, 32);
    const float bt = gdr_sigmoid(braw);
    float ratio = dvu[j] / (bt > 0.0f ? bt : 1.0f);        // dV_t . U_t / b_t (b = 0: 0 / 1)
    // dV and U each carry b, and the matrix cores drop what is below 2^-126: their product is
    // gone below b = 2^-63, its third parts (2^-16) below 2^-55.  From 2^-40 on, which leaves 30
    // bits for the sizes of dV / b and U / b, it is summed again with both times 2^-e, b = m 2^e.
    if (__builtin_expect(__ballot(bt > 0.0f && bt < 0x1p-40f) != 0, 0)) {
      const uint32_t e = __builtin_bit_cast(uint32_t, bt) >> 23;
      const float up = __builtin_bit_cast(float, (254u - e) << 23), down = __builtin_bit_cast(float, e << 23);
      float x = 0.0f;
      for (int64_t ch = half; ch < q.P; ch += 2) {
        const int64_t at = (bl * Pp + ch) * kC + j;
        x = __builtin_fmaf(p.dvw[at] * up, p.u[at] * up, x);
      }
      x += __shfl_xor(x, 32);
      ratio = bt > 0.0f && bt < 0x1p-40f ? x * down / (bt * up) : ratio;
    }
    vec[lane] = half ? ratio : s1;                         // over the factors of k and q
  }
}

// kPS: value channels taken at a time (a slab); every sum over value channels is
// linear, so slabs and value heads are one loop of turns.  A turn walks the block's
// chunks with the state in accumulators (column n of the keys, all value channels of
// the slab); the next chunk's operands are loaded into registers meanwhile.
template <typename T, typename O, int kN, int kPS>
__global__ __launch_bounds__(kN * 4) void gdr_grad_kernel(GdrChunkParams p) {
  constexpr int kParts = GdrIn<T>::kParts, kGParts = GdrIn<O>::kParts;
  constexpr int kW = kN / 16, kThreads = 64 * kW;
  constexpr int kPT = kPS / 16, kPB = kPS / 32;
  constexpr int kMf = (9 * kGdrPlane / 8 + kThreads - 1) / kThreads;      // 16-byte pieces of the planes per thread
  __shared__ __align__(16) uint16_t dOt[kGParts * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t dVt[3 * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t Ut[3 * kPS * kGdrRow];
  __shared__ __align__(16) uint16_t Kt[kParts * kN * kGdrRow];
  __shared__ __align__(16) uint16_t Qt[kParts * kN * kGdrRow];
  __shared__ __align__(16) uint16_t mf[kMf * kThreads * 8];               // operands made of M1, M1^T and M2 + M2^T
  __shared__ double cum[32];
  __shared__ __align__(16) float gam[32], en[32], rk[32], rq[32];
  __shared__ __align__(16) float red[2][kW][32];
  __shared__ float X[kGdrBlk][kW][32], Y[kGdrBlk][kW][32], Z[kGdrBlk][kW], decs[kGdrBlk];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15,
            g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);
  const int64_t blk = it % p.n_blks, bg = it / p.n_blks, g = bg % q.G, b = bg / q.G;
  const int64_t len = gdr_length(q, b), nl = (len + kC - 1) / kC;
  const int64_t cb = blk * kGdrBlk, rep = q.H / q.G;
  const int nc = (int)(nl - cb < 0 ? 0 : nl - cb < kGdrBlk ? nl - cb : kGdrBlk);      // live chunks
  const int64_t tb = cb * kC, te = tb + kGdrBlk * kC < q.L ? tb + kGdrBlk * kC : q.L;
  const int n = 16 * w + i16;                              // this lane's key number

  const T* krows = static_cast<const T*>(q.k) + b * q.k_stride + g * q.N * q.L;
  const T* qrows = static_cast<const T*>(q.q) + b * q.q_stride + g * q.N * q.L;
  const T* tail_k = static_cast<const T*>(p.tail_k) + bg * q.N * kC;
  const T* tail_q = static_cast<const T*>(p.tail_q) + bg * q.N * kC;
  // this lane's row of dQ and dK (n < N) and its tokens of chunk c, worked out where it is used
  // (not before the loops: that would hold registers over them)
  auto drow = [&](int c) {
    int own = n;
    asm volatile("" : "+v"(own), "+s"(c));
    return (bg * q.N + own) * q.L + (cb + c) * kC + 4 * g4;
  };
  O *dq = static_cast<O*>(p.dq), *dk = static_cast<O*>(p.dk);

  const int64_t Pp = (q.P + 63) / 64 * 64;
  const int64_t slabs = (q.P + kPS - 1) / kPS, turns = nc > 0 ? rep * slabs : 0;
  Rows<T, kN, kThreads> ldk, ldq;
  Rows<O, kPS, kThreads> ldo;
  Rows<float, kPS, kThreads> ldv, ldu;
  uint4 ldm[kMf];
  double lcum, llast;                                      // the next chunk's cumulated decay and lengths
  float lrk, lrq;
  f32x4 S[kPT], D[kPT];                                    // S and dS: column n, rows of the value channels
  auto four = [&](const float* v, int rt) { return *reinterpret_cast<const f32x4*>(v + 16 * rt + 4 * g4); };

  // dQ and dK of a wave with lanes past the last key number, and of the chunk of the row's end,
  // are stored after the last turn; until then they take the place of the four first tiles of
  // dS (of the chunk, last head and last slab) that this wave alone reads.
  const bool split = 16 * w + 16 > q.N;
  auto kept = [&](int64_t bl, int64_t p0) { return p.chunk_dS + (bl * Pp + p0) * kN + w * 256; };

  for (int64_t turn = 0; turn < turns; ++turn) {
    const int64_t h = g * rep + turn / slabs, bh = b * q.H + h, p0 = (turn % slabs) * kPS;
    const bool first = turn % slabs == 0, last = turn % slabs == slabs - 1;
    const int prow = (int)(q.P - p0 < kPS ? q.P - p0 : kPS);  // channels of this slab
    const int64_t bl0 = block_of(p, b, h, cb);
    auto load_rows = [&](int c) {
      const int64_t cc = cb + c, bl = bl0 + c;
      const GdrChunkSrc<T> sk(krows, q.L, tail_k, cc, len), sq(qrows, q.L, tail_q, cc, len);
      const GdrChunkSrc<O> sy(static_cast<const O*>(p.dy) + (bh * q.P + p0) * q.L, q.L,
                              static_cast<const O*>(p.tail_dy) + (bh * q.P + p0) * kC, cc, len);
      const float* vec = p.vec + bl * p.vec_stride;
      lrk = lane_load<float>(vec + 128, (lane & 31) * 4);
      lrq = lane_load<float>(vec + 160, (lane & 31) * 4);
      lcum = lane_load<double>(vec + 192, (lane & 31) * 8);
      llast = *reinterpret_cast<const double*>(vec + 192 + 62);
      ldk.load(sk.at, sk.stride, q.N, tid);
      ldq.load(sq.at, sq.stride, q.N, tid);
      ldo.load(sy.at, sy.stride, prow, tid);
      ldv.load_dense(p.dvw + (bl * Pp + p0) * kC, tid);
      ldu.load_dense(p.u + (bl * Pp + p0) * kC, tid);
      const uint16_t* planes = p.planes + bl * 9 * kGdrPlane;
#pragma unroll
      for (int j = 0; j < kMf; ++j) {
        const uint32_t at = (tid + kThreads * j) * 16;
        ldm[j] = lane_load<uint4>(planes, at < 9 * kGdrPlane * 2 ? at : 0);
      }
    };
    const uint32_t soff = (uint32_t)(4 * g4 * kN + n) * 4u;
    auto load_state = [&](const float* src, f32x4 (&x)[kPT]) {
#pragma unroll
      for (int tp = 0; tp < kPT; ++tp)
#pragma unroll
        for (int r = 0; r < 4; ++r) x[tp][r] = lane_load<float>(src + (16 * tp + r) * kN, soff);
    };
    auto load_dstate = [&](int64_t bl) {
      const float* src = p.chunk_dS + (bl * Pp + p0) * kN + w * 256;
#pragma unroll
      for (int tp = 0; tp < kPT; ++tp)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          D[tp][r] = lane_load<float>(src + tp * 16 * kN + 16 * r, (uint32_t)(64 * g4 + i16) * 4u);
    };
    load_rows(0);
    load_state(p.blk_S + ((bh * p.n_blks + blk) * Pp + p0) * kN, S);
    load_dstate(bl0);
    for (int c = 0; c < nc; ++c) {
      const int64_t cc = cb + c;
      const int cn = c + 1 < nc ? c + 1 : c;
      __syncthreads();                                     // the chunk before is done with LDS
      ldk.put(Kt, (int)q.N, tid);
      ldq.put(Qt, (int)q.N, tid);
      ldo.put(dOt, prow, tid);
      ldv.put(dVt, kPS, tid);
      ldu.put(Ut, kPS, tid);
#pragma unroll
      for (int j = 0; j < kMf; ++j) *reinterpret_cast<uint4*>(&mf[(tid + kThreads * j) * 8]) = ldm[j];
      if (w == 0) {
        const int t = lane & 31;
        cum[t] = lcum;
        gam[t] = hw_exp2((float)lcum);
        en[t] = hw_exp2((float)(llast - lcum));
        rk[t] = lrk;
        rq[t] = lrq;
        decs[c] = hw_exp2((float)llast);
      }
      __syncthreads();
      const float dec = decs[c];

      // through the states that enter and leave
      f32x4 Rq[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}, Rk[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
      f32x4 Ru[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
      float z = 0.0f;
#pragma unroll
      for (int kb = 0; kb < kPB; ++kb) {
        bf16x8 sb[3], db[3], ao[2][kGParts], av[2][3], au[2][3];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          plane_frags_t<kGParts, kPS>(dOt, 32 * kb, 16 * rt, lane, ao[rt]);
          plane_frags_t<3, kPS>(dVt, 32 * kb, 16 * rt, lane, av[rt]);
        }
        gdr_split<3>(S[2 * kb], S[2 * kb + 1], sb);
        gdr_mma_rows<3>(ao, sb, Rq);
        gdr_mma_rows<3>(av, sb, Rk);
        gdr_split<3>(D[2 * kb], D[2 * kb + 1], db);
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) plane_frags_t<3, kPS>(Ut, 32 * kb, 16 * rt, lane, au[rt]);
        gdr_mma_rows<3>(au, db, Ru);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          z = __builtin_fmaf(S[2 * kb][r], D[2 * kb][r], z);
          z = __builtin_fmaf(S[2 * kb + 1][r], D[2 * kb + 1][r], z);
        }
        __builtin_amdgcn_sched_barrier(0);                 // one block's operands in registers at a time
      }
      // what the turns before left of this chunk, and the next one
      f32x4 aq[2], ak[2];
      const int64_t acc_at = ((bg * p.n_chunks + cc) * kN + n) * kC + 4 * g4;
      if (turn > 0) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          aq[rt] = *reinterpret_cast<const f32x4*>(p.acc_dq + acc_at + 16 * rt);
          ak[rt] = *reinterpret_cast<const f32x4*>(p.acc_dk + acc_at + 16 * rt);
        }
      } else {
        aq[0] = aq[1] = ak[0] = ak[1] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      load_dstate(bl0 + cn);
      z = gdr_sum16(z);
      z += __shfl_xor(z, 16);
      z += __shfl_xor(z, 32);
      Z[c][w] = first ? z : Z[c][w] + z;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const f32x4 ga = four(gam, rt), kt4 = four(rk, rt) * tile_four<kParts, kN>(Kt, n, 16 * rt + 4 * g4);
        const f32x4 qt4 = four(rq, rt) * tile_four<kParts, kN>(Qt, n, 16 * rt + 4 * g4);
        Rq[rt] *= ga * q.scale;
        Rk[rt] *= ga;
        Ru[rt] *= four(en, rt);
        const f32x4 xs = qt4 * Rq[rt] - kt4 * Rk[rt], ys = kt4 * Ru[rt];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float *x = &X[c][w][16 * rt + 4 * g4 + r], *y = &Y[c][w][16 * rt + 4 * g4 + r];
          const float a = gdr_sum16(xs[r]), e = gdr_sum16(ys[r]);
          *x = first ? a : *x + a;
          *y = first ? e : *y + e;
        }
        Ru[rt] -= Rk[rt];
      }
      // within the chunk: M1 and M2 are sums over all slabs, so a head's first one adds them
      if (first) {
        bf16x8 kb_[kParts], qb[kParts], a[2][3];
        plane_frags<kParts, kN>(Kt, 16 * w, 0, lane, kb_);
        plane_frags<kParts, kN>(Qt, 16 * w, 0, lane, qb);
        auto get = [&](int kind) {
#pragma unroll
          for (int rt = 0; rt < 2; ++rt)
#pragma unroll
            for (int s = 0; s < 3; ++s)
              a[rt][s] = *reinterpret_cast<const bf16x8*>(&mf[(3 * kind + s) * kGdrPlane + rt * 512 + lane * 8]);
        };
        get(0);
        gdr_mma_rows<3>(a, kb_, Rq);
        get(1);
        gdr_mma_rows<3>(a, qb, Ru);
        get(2);
        gdr_mma_rows<3>(a, kb_, Ru);
      }
      __builtin_amdgcn_sched_barrier(0);
      load_rows(cn);
      // the state after the chunk
      {
        bf16x8 kb3[3];
        gdr_split<3>(four(en, 0) * four(rk, 0) * tile_four<kParts, kN>(Kt, n, 4 * g4),
                     four(en, 1) * four(rk, 1) * tile_four<kParts, kN>(Kt, n, 16 + 4 * g4), kb3);
#pragma unroll
        for (int tp = 0; tp < kPT; tp += 2) {
          bf16x8 a[2][3];
          plane_frags<3, kPS>(Ut, 16 * tp, 0, lane, a[0]);
          plane_frags<3, kPS>(Ut, 16 * tp + 16, 0, lane, a[1]);
          f32x4 s2[2] = {S[tp] * dec, S[tp + 1] * dec};
          gdr_mma_rows<3>(a, kb3, s2);
          S[tp] = s2[0];
          S[tp + 1] = s2[1];
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        aq[rt] += Rq[rt];
        ak[rt] += Ru[rt];
      }
      if (turn + 1 < turns) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) {
          *reinterpret_cast<f32x4*>(p.acc_dq + acc_at + 16 * rt) = aq[rt];
          *reinterpret_cast<f32x4*>(p.acc_dk + acc_at + 16 * rt) = ak[rt];
        }
      } else {                                             // all of dQ and dK: through the normalisation, out
        if (q.norm) {
          f32x4 kh[2], qh[2];
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
            kh[rt] = four(rk, rt) * tile_four<kParts, kN>(Kt, n, 16 * rt + 4 * g4);
            qh[rt] = four(rq, rt) * tile_four<kParts, kN>(Qt, n, 16 * rt + 4 * g4);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              red[0][w][16 * rt + 4 * g4 + r] = gdr_sum16(qh[rt][r] * aq[rt][r]);
              red[1][w][16 * rt + 4 * g4 + r] = gdr_sum16(kh[rt][r] * ak[rt][r]);
            }
          }
          __syncthreads();
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
            f32x4 sq4 = f32x4{0.f, 0.f, 0.f, 0.f}, sk4 = sq4;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
              sq4 += *reinterpret_cast<const f32x4*>(&red[0][k][16 * rt + 4 * g4]);
              sk4 += *reinterpret_cast<const f32x4*>(&red[1][k][16 * rt + 4 * g4]);
            }
            aq[rt] = four(rq, rt) * (aq[rt] - qh[rt] * sq4);
            ak[rt] = four(rk, rt) * (ak[rt] - kh[rt] * sk4);
          }
        }
        if (split || (cc + 1) * kC > len) {                // kept where this wave's dS was, stored last
          int here = c;
          asm volatile("" : "+s"(here));
          float* at = kept(bl0 + here, p0);
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
            lane_store(at + rt * 16 * kN, lane * 16u, aq[rt]);
            lane_store(at + (2 + rt) * 16 * kN, lane * 16u, ak[rt]);
          }
        } else {
          const int64_t at = drow(c);
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) {
            gdr_store_whole4(dq + at + 16 * rt, aq[rt]);
            gdr_store_whole4(dk + at + 16 * rt, ak[rt]);
          }
        }
      }
    }
    __syncthreads();

    // ---- gates of this head
    if (last && w == 0) {
      const int t = lane & 31;
      float sA = 0.0f, sb = 0.0f;
      const float A = q.A[h], bias = q.bias ? q.bias[h] : 0.0f;
      for (int c = 0; c < nc; ++c) {
        const float* vec = p.vec + (bl0 + c) * p.vec_stride;
        float x = 0.0f, y = 0.0f, f = 0.0f;
#pragma unroll
        for (int k = 0; k < kW; ++k) {
          x += X[c][k][t];
          y += Y[c][k][t];
          f += Z[c][k];
        }
        float xs = x, ys = y;                              // sums over i >= t and over j <= t
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const float o = __shfl_down(xs, d, 32), u = __shfl_up(ys, d, 32);
          xs += t + d < 32 ? o : 0.0f;
          ys += t >= d ? u : 0.0f;
        }
        const float dg = vec[t] + xs + (ys - y) + decs[c] * f;
        const int64_t tok = (cb + c) * kC + t, at = bh * q.L + (tok < len ? tok : len - 1);
        const float xr = gdr_load(static_cast<const T*>(q.delta) + at) + bias;
        const float br = gdr_load(static_cast<const T*>(q.beta) + at);
        const float step = softplus(xr);
        const float dd = dg * A * gdr_sigmoid(xr);
        const float db = vec[32 + t] * gdr_sigmoid(-br);
        sA += tok < len && dg != 0.0f ? dg * step : 0.0f;   // (an infinite step: a and dg are 0)
        sb += tok < len ? dd : 0.0f;
        const int64_t at0 = bh * q.L + (cb + c) * kC, left = len - (cb + c) * kC;
        gdr_store_within(static_cast<O*>(p.ddelta) + at0, left, t, dd);
        gdr_store_within(static_cast<O*>(p.dbeta) + at0, left, t, db);
      }
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        sA += __shfl_xor(sA, d);
        sb += __shfl_xor(sb, d);
      }
      float* dst = p.part + ((b * p.n_blks + blk) * q.H + h) * 2;
      dst[0] = sA;
      dst[1] = sb;
    }
  }

  // tokens behind the row's end: gates and whole chunks of dQ and dK
  for (int64_t hh = 0; hh < rep; ++hh) {
    const int64_t bh = b * q.H + g * rep + hh;
    for (int64_t t = (len > tb ? len : tb) + tid; t < te; t += kThreads) {
      gdr_store(static_cast<O*>(p.ddelta) + bh * q.L + t, 0.0f);
      gdr_store(static_cast<O*>(p.dbeta) + bh * q.L + t, 0.0f);
    }
    if (nc == 0 && tid < 2) p.part[((b * p.n_blks + blk) * q.H + g * rep + hh) * 2 + tid] = 0.0f;
  }
  if (n < q.N) {
    O *dqrow = dq + (bg * q.N + n) * q.L, *dkrow = dk + (bg * q.N + n) * q.L;
    for (int c = 0; c < nc; ++c) {
      if (!split && (cb + c + 1) * kC <= len) continue;
      const float* src = kept(block_of(p, b, g * rep + rep - 1, cb + c), (slabs - 1) * kPS);
      f32x4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const f32x4*>(src + j * 16 * kN + lane * 4);
      gdr_store_end(dqrow, (cb + c) * kC, len, q.L, {x[0], x[1]}, g4);
      gdr_store_end(dkrow, (cb + c) * kC, len, q.L, {x[2], x[3]}, g4);
    }
    for (int64_t t = tb + nc * kC + 4 * g4; t < te; t += 16) {
      gdr_store4(dqrow, t, q.L, f32x4{0.f, 0.f, 0.f, 0.f});
      gdr_store4(dkrow, t, q.L, f32x4{0.f, 0.f, 0.f, 0.f});
    }
  }
}

// dA and ddelta_bias of one head per workgroup: the blocks' sums in a fixed order, in fp64.
__global__ __launch_bounds__(64) void gdr_gate_sum_kernel(GdrChunkParams p) {
  const int64_t h = blockIdx.x, rows = p.g.B * p.n_blks;
  double a = 0.0, s = 0.0;
  for (int64_t r = threadIdx.x; r < rows; r += 64) {
    a += p.part[(r * p.g.H + h) * 2];
    s += p.part[(r * p.g.H + h) * 2 + 1];
  }
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    a += __shfl_xor(a, d);
    s += __shfl_xor(s, d);
  }
  if (threadIdx.x == 0) {
    p.dA[h] = (float)a;
    p.dbias[h] = (float)s;
  }
}

template <typename T, typename O, int kN>
hipError_t bwd_n(const GdrChunkParams& p, hipStream_t s) {
  const GdrParams& q = p.g;
  hipLaunchKernelGGL((gdr_adjoint_kernel<T, O, kN>), dim3((unsigned)(q.B * q.H * ((q.P + 63) / 64))), dim3(256), 0, s, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((gdr_pair_kernel<T, O, kN>), dim3((unsigned)(q.B * q.H * p.n_chunks)), dim3(256), 0, s, p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  const dim3 grid((unsigned)(q.B * q.G * p.n_blks));
  // 128 channels at a time where the operands have one plane each (LDS) and the padded
  // channels come in pairs of 64
  constexpr bool kOne = GdrIn<T>::kParts == 1 && GdrIn<O>::kParts == 1;
  if (kOne && (q.P + 63) / 64 % 2 == 0)
    hipLaunchKernelGGL((gdr_grad_kernel<T, O, kN, kOne ? 128 : 64>), grid, dim3(kN * 4), 0, s, p);
  else
    hipLaunchKernelGGL((gdr_grad_kernel<T, O, kN, 64>), grid, dim3(kN * 4), 0, s, p);
  if ((e = hipGetLastError()) != hipSuccess) return e;
  hipLaunchKernelGGL(gdr_gate_sum_kernel, dim3((unsigned)q.H), dim3(64), 0, s, p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t bwd_t(const GdrChunkParams& p, hipStream_t s) {
  return p.g.N > 64 ? bwd_n<T, O, 128>(p, s) : bwd_n<T, O, 64>(p, s);
}

}  // namespace

hipError_t launch_gdr_bwd(const GdrChunkParams& p, Dt in, Dt grad, hipStream_t s) {
  hipError_t e = launch_gdr_prep(p, in, grad, true, s);
  if (e != hipSuccess) return e;
  if ((e = launch_gdr_states(p, in, s)) != hipSuccess) return e;
  if (in == Dt::BF16) return grad == Dt::BF16 ? bwd_t<uint16_t, uint16_t>(p, s) : bwd_t<uint16_t, float>(p, s);
  return grad == Dt::BF16 ? bwd_t<float, uint16_t>(p, s) : bwd_t<float, float>(p, s);
}

}  // namespace mamba
