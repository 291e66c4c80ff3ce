// gdr_chunk.hip -- the gated delta rule over sequences, in chunks of C = 32
// tokens on the matrix cores (gfx950).
//
// For a chunk with entering state S0 (P x N), rows k_i, q_i, v_i, cumulated log
// decay G_i (from the chunk's first token, inclusive) and D_ij = exp(G_i - G_j):
//   the updates u_i solve u_i = b_i (v_i - exp(G_i) S0 k_i - sum_(j<i) D_ij (k_i . k_j) u_j),
//   a unit lower-triangular system, so with A_ij = b_i D_ij k_i . k_j (j < i) and
//   T = (1 + A)^-1 diag(b):
//     R = V - diag(exp G) K S0^T          (C x P)
//     U = T R
//     Y = scale (diag(exp G) Q S0^T + tril(D o Q K^T) U)
//     S1 = exp(G_C) S0 + (diag(exp(G_C - G)) U)^T K
// T, the scaled query matrix and the factors do not depend on the state: a first
// kernel makes them for every (batch row, head, chunk) in parallel; the second runs
// the chain of chunks.  Differences G_i - G_j are taken in fp64 of sums from the
// chunk's start, so a hard reset inside a chunk does not cost the later tokens
// their digits; lengths of unit keys are folded into T, the query matrix and the
// factors, so that raw bf16 keys stay exact operands.
//
// The chain is cut over the P value channels, which are independent: one wave owns
// 16 channels and their 16 x N state in MFMA accumulators, four waves (64 channels)
// share the chunk's K and Q tiles in LDS.  Per chunk and wave at N = 128 and bf16:
// 24 + 16 + 12 + 6 + 24 MFMAs of 16 cycles each (K S0, Q S0, T R, query x U, U K);
// every result is the next product's operand in place (gdr_mfma.hpp).
//
// Few heads over a long L: L is cut into segments.  A summary launch runs every
// segment but the last from a zero state and, since a segment maps its entering
// state linearly (S1 = S0 M + h), with N more rows that start as the identity and
// have no values; they end as M.  A carry kernel chains the segments, and the full
// launch runs all of them at once.
//
// Measured after warm-up, bf16, 128 x 128.  40 heads, batch 4, L = 2048 (263 MB, 55 us at the
// 4.78 TB/s of a large copy): preparation 53 us, chain 216 us; a call is 268 us traced, 258 us not.
// The chain's 320 workgroups meet 256 CUs, and the CUs with two of them set its time: 256
// workgroups (32 heads) take 144 us, 512 (64 heads) 255 us.  With one per CU a chunk takes
// 2.2 us, 5300 cycles: its 82 products 1312, the rest the issue of 420 vector instructions by
// one wave per SIMD, operand reads and waits (0.28 of a wave's time it waits to issue, 0.23 for
// memory or LDS).  16 heads, batch 1, L = 32768: preparation 132, summary 305, carry 21, full launch
// 266 us.  Registers: at 256 the variants for N > 64 with fp32 inputs or outputs spill 8 to 24.
#include "gdr_mfma.hpp"

namespace mamba {
namespace {

// ----------------------------------------------------------------------------- preparation
// One workgroup per (batch row, key head, chunk).  K K^T and Q K^T once for all value
// heads of the key head (wave w: rows 16 (w & 1) of K or Q), then a wave per value
// head: gates, the triangular solve, and the operand planes.  The solve is column by
// column in registers: lane 32 half + c holds rows i = 2 m + half of column c of the
// inverse; once row j is final, every later row takes its multiple of it, 15 fused
// multiply-adds at most per lane and step with no dependence among them.
template <typename T, typename O, int kN, bool kBwd>
__global__ __launch_bounds__(256) void gdr_prep_kernel(GdrChunkParams p) {
  constexpr int kParts = GdrIn<T>::kParts;
  constexpr int kTile = kN * kGdrRow * kParts;
  constexpr int kM = 36;                                   // floats per row of a wave's matrix
  constexpr int kWaveM = 32 * kM;
  constexpr size_t kTileBytes = 2 * kTile * 2, kMBytes = 4 * kWaveM * 4;
  __shared__ __align__(16) char mem[kTileBytes > kMBytes ? kTileBytes : kMBytes];
  __shared__ float prod[2][32 * 33];                       // K K^T, Q K^T
  __shared__ float red[2][8][32];
  __shared__ float rlen[2][32];                            // 1 / |k|, 1 / |q| (1 without normalisation)
  __shared__ double cums[4][32];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15, g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);
  const int64_t c = it % p.n_chunks, bg = it / p.n_chunks, g = bg % q.G, b = bg / q.G;
  const int64_t len = gdr_length(q, b), t0 = c * kC;
  if (t0 >= len) return;
  uint16_t* Kt = reinterpret_cast<uint16_t*>(mem);
  uint16_t* Qt = Kt + kTile;
  {
    GdrTile<T, kN> tk, tq;
    tk.init(q.N, tid);
    tq.init(q.N, tid);
    const T* krows = static_cast<const T*>(q.k) + b * q.k_stride + g * q.N * q.L + t0;
    const T* qrows = static_cast<const T*>(q.q) + b * q.q_stride + g * q.N * q.L + t0;
    if (t0 + kC <= len) {
      tk.load(krows, q.L, tid);
      tq.load(qrows, q.L, tid);
    } else {                     // the row ends here: leave padded copies for the chain
      tk.load_part(krows, q.L, len - t0, tid);
      tq.load_part(qrows, q.L, len - t0, tid);
      tk.save(static_cast<T*>(p.tail_k) + bg * q.N * kC, tid);
      tq.save(static_cast<T*>(p.tail_q) + bg * q.N * kC, tid);
      const int64_t rows = q.H / q.G * q.P, first = (b * q.H + g * (q.H / q.G)) * q.P;
      const T* v = static_cast<const T*>(q.v) + b * q.v_stride + g * rows * q.L + t0;
      T* tv = static_cast<T*>(p.tail_v) + first * kC;
      for (int64_t id = tid; id < rows * 4; id += 256) {
        typename GdrIn<T>::Raw x;
        x.part(v + (id >> 2) * q.L + 8 * (id & 3), len - t0 - 8 * (id & 3));
        x.save(tv + 8 * id);
      }
      if constexpr (kBwd) {
        const O* dy = static_cast<const O*>(p.dy) + first * q.L + t0;
        O* td = static_cast<O*>(p.tail_dy) + first * kC;
        for (int64_t id = tid; id < rows * 4; id += 256) {
          typename GdrIn<O>::Raw x;
          x.part(dy + (id >> 2) * q.L + 8 * (id & 3), len - t0 - 8 * (id & 3));
          x.save(td + 8 * id);
        }
      }
    }
    tk.put(Kt, tid);
    tq.put(Qt, tid);
  }
  __syncthreads();
  {
    const uint16_t* src = (w & 2) ? Qt : Kt;
    const int rt = w & 1;
    f32x4 acc[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
    for (int kb = 0; kb < kN / 32; ++kb) {
      bf16x8 a[kParts], b0[kParts], b1[kParts];
      gdr_frags_t<T, kN>(src, 32 * kb, 16 * rt, lane, a);
      gdr_frags_t<T, kN>(Kt, 32 * kb, 0, lane, b0);
      acc[0] = gdr_mma<3>(a, b0, acc[0]);
      gdr_frags_t<T, kN>(Kt, 32 * kb, 16, lane, b1);
      acc[1] = gdr_mma<3>(a, b1, acc[1]);
    }
#pragma unroll
    for (int ct = 0; ct < 2; ++ct)
#pragma unroll
      for (int r = 0; r < 4; ++r) prod[w >> 1][(16 * rt + 4 * g4 + r) * 33 + 16 * ct + i16] = acc[ct][r];
  }
  if (q.norm) {
    const int t = tid & 31, part = tid >> 5;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const uint16_t* tile = m ? Qt : Kt;
      float ss = 0.0f;
      for (int n = part * (kN / 8); n < (part + 1) * (kN / 8); ++n) {
        float x = 0.0f;
#pragma unroll
        for (int s = kParts - 1; s >= 0; --s) x += bf16_to_f32(tile[s * kN * kGdrRow + n * kGdrRow + t]);
        ss = __builtin_fmaf(x, x, ss);
      }
      red[m][part][t] = ss;
    }
  }
  __syncthreads();
  if (tid < 64) {
    const int m = tid >> 5, t = tid & 31;
    float r = 1.0f;
    if (q.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int part = 0; part < 8; ++part) ss += red[m][part][t];
      r = gdr_rnorm(ss);
    }
    rlen[m][t] = r;
  }
  __syncthreads();

  float* M = reinterpret_cast<float*>(mem) + w * kWaveM;    // the tiles are no longer needed
  const int c32 = lane & 31, half = lane >> 5;
  const int64_t rep = q.H / q.G;
  for (int64_t hh = w; hh < rep; hh += 4) {
    const int64_t h = g * rep + hh, bh = b * q.H + h;
    const int64_t blk = block_of(p, b, h, c);
    uint16_t* planes = p.planes + blk * (int64_t)(kBwd ? 9 : 3 + p.p_parts) * kGdrPlane;
    float* vec = p.vec + blk * p.vec_stride;
    // gates: base-2 log decay, held at 2^-1000 per token (zero in fp32) so that a
    // reset by an infinite step leaves differences finite
    const int64_t t = t0 + c32;
    double cum = 0.0;
    float beta = 0.0f;
    if (t < len) {
      const float x = gdr_load(static_cast<const T*>(q.delta) + bh * q.L + t) + (q.bias ? q.bias[h] : 0.0f);
      const float g2 = softplus(x) * q.A[h] * kLog2e;
      cum = g2 < -1000.0f ? -1000.0 : (double)g2;
      beta = gdr_sigmoid(gdr_load(static_cast<const T*>(q.beta) + bh * q.L + t));
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const double o = __shfl_up(cum, d, 32);
      if (c32 >= d) cum += o;
    }
    if (half == 0) cums[w][c32] = cum;
    const double last = __shfl(cum, 31, 32);
    const float rk = rlen[0][c32], rq = rlen[1][c32] * q.scale;
    const float dec = hw_exp2((float)cum);
    if (half == 0) {
      vec[c32] = beta == beta ? dec * rk : beta;           // a NaN shows in the token's residual
      vec[32 + c32] = dec * rq;
      vec[64 + c32] = hw_exp2((float)(last - cum)) * rk;
      if (c32 == 0) vec[96] = hw_exp2((float)last);
      if constexpr (kBwd) {
        vec[128 + c32] = rk;
        vec[160 + c32] = rlen[1][c32];
        reinterpret_cast<double*>(vec + 192)[c32] = cum;
      }
    }
    wave_sync();
    // M[j][i]: column j of the strictly lower-triangular A, its rows i with even i first
    {
      const int pos = (c32 & 1) * 16 + (c32 >> 1);
      const float f = beta * rk;
#pragma unroll
      for (int jj = 0; jj < 16; ++jj) {
        const int j = 2 * jj + half;
        const float e = hw_exp2((float)(cum - cums[w][j]));
        M[j * kM + pos] = j < c32 ? f * rlen[0][j] * prod[0][c32 * 33 + j] * e : 0.0f;
      }
    }
    // the query matrix, straight into operand order
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      const int row = 16 * rt + i16;
      const double cr = cums[w][row];
      const float fr = rlen[1][row] * q.scale;
      f32x4 x[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int col = (e < 4 ? 0 : 16) + 4 * g4 + (e & 3);
        if constexpr (kBwd) {             // transposed: this lane's row is a key, its columns queries
          const float d = hw_exp2((float)(cums[w][col] - cr));
          x[e >> 2][e & 3] = col >= row ? q.scale * rlen[1][col] * rlen[0][row] * prod[1][col * 33 + row] * d : 0.0f;
        } else {
          const float d = hw_exp2((float)(cr - cums[w][col]));
          x[e >> 2][e & 3] = col <= row ? fr * rlen[0][col] * prod[1][row * 33 + col] * d : 0.0f;
        }
      }
      if constexpr (kBwd) {
        bf16x8 f[3];
        gdr_split<3>(x[0], x[1], f);
#pragma unroll
        for (int s = 0; s < 3; ++s)
          *reinterpret_cast<bf16x8*>(planes + (6 + s) * kGdrPlane + rt * 512 + lane * 8) = f[s];
      } else if (p.p_parts == 2) {
        bf16x8 f[2];
        gdr_split<2>(x[0], x[1], f);
#pragma unroll
        for (int s = 0; s < 2; ++s)
          *reinterpret_cast<bf16x8*>(planes + (3 + s) * kGdrPlane + rt * 512 + lane * 8) = f[s];
      } else {
        bf16x8 f[3];
        gdr_split<3>(x[0], x[1], f);
#pragma unroll
        for (int s = 0; s < 3; ++s)
          *reinterpret_cast<bf16x8*>(planes + (3 + s) * kGdrPlane + rt * 512 + lane * 8) = f[s];
      }
    }
    wave_sync();
    // T = (1 + A)^-1: x[m] is row 2 m + half of column c32
    float x[16];
#pragma unroll
    for (int m = 0; m < 16; ++m) x[m] = (2 * m + half == c32) ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < 31; ++j) {
      // row j to both halves of the wave
      const auto sw = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x[j >> 1]),
                                                       __builtin_bit_cast(uint32_t, x[j >> 1]), false, false);
      const float xj = __builtin_bit_cast(float, (j & 1) ? sw[1] : sw[0]);
      const float* col = M + j * kM + half * 16;
#pragma unroll
      for (int m4 = (j + 1) / 2 & ~3; m4 < 16; m4 += 4) {
        const float4 a = *reinterpret_cast<const float4*>(col + m4);
        if (2 * m4 + 1 > j) x[m4] = __builtin_fmaf(-a.x, xj, x[m4]);
        if (2 * m4 + 3 > j) x[m4 + 1] = __builtin_fmaf(-a.y, xj, x[m4 + 1]);
        if (2 * m4 + 5 > j) x[m4 + 2] = __builtin_fmaf(-a.z, xj, x[m4 + 2]);
        if (2 * m4 + 7 > j) x[m4 + 3] = __builtin_fmaf(-a.w, xj, x[m4 + 3]);
      }
    }
    wave_sync();
#pragma unroll
    for (int m = 0; m < 16; ++m)     // (above the diagonal zero, also times a NaN)
      M[(2 * m + half) * 33 + c32] = 2 * m + half >= c32 ? x[m] * beta : 0.0f;
    wave_sync();
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      f32x4 y[2];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] = M[(16 * rt + i16) * 33 + (e < 4 ? 0 : 16) + 4 * g4 + (e & 3)];
      bf16x8 f[3];
      gdr_split<3>(y[0], y[1], f);
#pragma unroll
      for (int s = 0; s < 3; ++s) *reinterpret_cast<bf16x8*>(planes + s * kGdrPlane + rt * 512 + lane * 8) = f[s];
      if constexpr (kBwd) {
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e >> 2][e & 3] = M[((e < 4 ? 0 : 16) + 4 * g4 + (e & 3)) * 33 + 16 * rt + i16];
        gdr_split<3>(y[0], y[1], f);
#pragma unroll
        for (int s = 0; s < 3; ++s)
          *reinterpret_cast<bf16x8*>(planes + (3 + s) * kGdrPlane + rt * 512 + lane * 8) = f[s];
      }
    }
    wave_sync();
  }
}

// ----------------------------------------------------------------------------- the chain of chunks
// kStates (for the backward pass): no queries; keeps every chunk's U and the state
// entering every block of kGdrBlk chunks.
enum ChainMode { kFull = 0, kSummary = 1, kStates = 2 };

// Takes a channel's residuals R (parts rb) that are not finite out of a chunk: U = T R again
// with zeros from the first such token on, U itself zero from it on (so that the query matrix
// gives the tokens before it what is theirs), the factors of its queries and its state NaN.
template <int kNT>
__device__ __forceinline__ void gdr_from_first(const bf16x8 (&tf)[2][3], const bf16x8 (&rb)[3], f32x4 (&U)[2],
                                               f32x4 (&fq)[2], f32x4 (&S)[kNT], int g4) {
  const float nan = __builtin_nanf("");
  auto token = [&](int e) { return (e < 4 ? 0 : 16) + 4 * g4 + (e & 3); };
  const uint4 top = __builtin_bit_cast(uint4, rb[0]);
  const uint32_t tw[4] = {top.x, top.y, top.z, top.w};
  int first = kC;
#pragma unroll
  for (int e = 7; e >= 0; --e)
    if ((tw[e >> 1] >> (16 * (e & 1)) & 0x7f80u) == 0x7f80u) first = token(e);
  first = min(first, __shfl_xor(first, 16));
  first = min(first, __shfl_xor(first, 32));
  bf16x8 part[3];
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const uint4 x = __builtin_bit_cast(uint4, rb[s]);
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] &= (token(2 * j) < first ? 0xffffu : 0u) | (token(2 * j + 1) < first ? 0xffff0000u : 0u);
    part[s] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
  }
  U[0] = U[1] = f32x4{0.f, 0.f, 0.f, 0.f};
  gdr_mma_rows<3>(tf, part, U);
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const bool before = 16 * rt + 4 * g4 + r < first;
      U[rt][r] = before ? U[rt][r] : 0.0f;
      fq[rt][r] = before ? fq[rt][r] : nan;
    }
#pragma unroll
  for (int tn = 0; tn < kNT; ++tn)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[tn][r] = first < kC ? nan : S[tn][r];
}

template <typename T, typename O, int kN, int kMode>
__global__ __launch_bounds__(256, 2) void gdr_chain_kernel(GdrChunkParams p) {
  constexpr int kParts = GdrIn<T>::kParts;
  constexpr int kTile = kN * kGdrRow * kParts;
  constexpr int kNT = kN / 16, kNB = kN / 32;
  constexpr int kOut = sizeof(O) == 2 ? 2 : 3;            // parts of what only y sees
  constexpr int kBuf = kParts == 1 ? 2 : 1;               // fp32 tiles take three planes: one buffer
  __shared__ __align__(16) uint16_t Kt[kBuf][kTile];
  __shared__ __align__(16) uint16_t Qt[kMode == kFull ? kBuf : 1][kMode == kFull ? kTile : 8];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15, g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t vslices = (q.P + 63) / 64;
  const int64_t slices = kMode != kSummary ? vslices : vslices + (q.N + 63) / 64;
  const int64_t segs = kMode != kSummary ? p.S : p.S - 1;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);
  const int64_t slice = it % slices, h = (it / slices) % q.H, bs = it / (slices * q.H);
  const int64_t seg = bs % segs, b = bs / segs, bh = b * q.H + h, g = h / (q.H / q.G);
  const bool ident = kMode == kSummary && slice >= vslices;  // rows of the transition
  const int64_t ch0 = (ident ? slice - vslices : slice) * 64 + 16 * w, ch = ch0 + i16;
  const int64_t channels = ident ? q.N : q.P;
  const bool mine = ch < channels, some = ch0 < channels;
  const int64_t mch = mine ? ch : channels - 1;              // lanes past the last channel run along on it
  const int64_t len = gdr_length(q, b);
  const int64_t c0 = seg * p.seg_chunks, c1 = c0 + p.seg_chunks < p.n_chunks ? c0 + p.seg_chunks : p.n_chunks;
  const int64_t live = (len + kC - 1) / kC, ce = live < c1 ? live : c1;

  const T* krows = static_cast<const T*>(q.k) + b * q.k_stride + g * q.N * q.L;
  const T* qrows = static_cast<const T*>(q.q) + b * q.q_stride + g * q.N * q.L;
  const T* tail_k = static_cast<const T*>(p.tail_k) + (b * q.G + g) * q.N * kC;
  const T* tail_q = static_cast<const T*>(p.tail_q) + (b * q.G + g) * q.N * kC;
  const int64_t vch = ident ? 0 : mch;                       // the transition's rows read a value and drop it
  const T* vrow = static_cast<const T*>(q.v) + b * q.v_stride + (h * q.P + vch) * q.L + 4 * g4;
  const T* tail_v = static_cast<const T*>(p.tail_v) + (bh * q.P + vch) * kC + 4 * g4;
  O* yrow = static_cast<O*>(q.y) + (bh * q.P + vch) * q.L;
  const int64_t Pp = vslices * 64;
  (void)Pp;

  f32x4 S[kNT];
  {
    const float* src = nullptr;
    if (kMode != kSummary && p.S > 1) src = p.seg_start + ((bs * q.H + h) * q.P + mch) * q.N;
    else if (kMode != kSummary && q.init) src = q.init + (bh * q.P + mch) * q.N;
#pragma unroll
    for (int tn = 0; tn < kNT; ++tn) {
      S[tn] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (src) S[tn] = gdr_load_state(src, 16 * tn + 4 * g4, q.N, q.state_vec);
      if (ident) {
#pragma unroll
        for (int r = 0; r < 4; ++r) S[tn][r] = 16 * tn + 4 * g4 + r == mch ? 1.0f : 0.0f;
      }
    }
  }

  // What a wave needs of a chunk besides the shared tiles.  Each is reloaded for the
  // next chunk right after its last use, so that it has a whole chunk to arrive
  // without a second set of registers.
  bf16x8 tf[2][3], pf[2][kOut];
  typename GdrIn<T>::Four v[2];
  f32x4 fk[2], fq[2], fu[2];
  float dec = 0.0f;
  const int64_t blk0 = block_of(p, b, h, 0);
  const int64_t pstride = (int64_t)(kMode == kStates ? 9 : 3 + p.p_parts) * kGdrPlane, vstride = p.vec_stride;
  const uint16_t* planes = p.planes + blk0 * pstride;
  const float* vec = p.vec + blk0 * vstride;
  auto load_v = [&](int64_t c) {
    const T* src = (c + 1) * kC <= len ? vrow + c * kC : tail_v;
    v[0].load(src);
    v[1].load(src + 16);
  };
  auto load_vec = [&](int64_t c, int which, f32x4 (&f)[2]) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
      f[rt] = lane_load<f32x4>(vec + c * vstride + 32 * which + 16 * rt, g4 * 16);
  };
  auto load_t = [&](int64_t c) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int s = 0; s < 3; ++s)
        tf[rt][s] = lane_load<bf16x8>(planes + c * pstride + s * kGdrPlane + rt * 512, lane * 16);
  };
  auto load_p = [&](int64_t c) {
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int s = 0; s < kOut; ++s)
        pf[rt][s] = lane_load<bf16x8>(planes + c * pstride + (3 + s) * kGdrPlane + rt * 512, lane * 16);
  };
  GdrTile<T, kN> tk, tq;
  tk.init(q.N, tid);
  tq.init(q.N, tid);
  auto load_tiles = [&](int64_t c) {
    const GdrChunkSrc<T> sk(krows, q.L, tail_k, c, len);
    tk.load(sk.at, sk.stride, tid);
    if constexpr (kMode == kFull) {
      const GdrChunkSrc<T> sq(qrows, q.L, tail_q, c, len);
      tq.load(sq.at, sq.stride, tid);
    }
  };
  auto put = [&](int buf) {
    tk.put(Kt[buf], tid);
    if constexpr (kMode == kFull) tq.put(Qt[buf], tid);
  };

  if (c0 < ce) {
    load_tiles(c0);
    load_v(c0);
    load_vec(c0, 0, fk);
    load_t(c0);
    load_vec(c0, 2, fu);
    dec = vec[c0 * vstride + 96];
    if constexpr (kMode == kFull) {
      load_vec(c0, 1, fq);
      load_p(c0);
    }
    put(0);
    __syncthreads();
  }
  bf16x8 sb[kNB][3];                                       // the state's operand parts
#pragma unroll
  for (int kb = 0; kb < kNB; ++kb) gdr_split<3>(S[2 * kb], S[2 * kb + 1], sb[kb]);
  auto end_of = [&](int buf) {
    const int free = kBuf == 2 ? buf ^ 1 : 0;
    return reinterpret_cast<float*>(w & 2 ? &Qt[free][0] : &Kt[free][0]) + (w & 1) * 512 + lane * 8;
  };
  for (int64_t c = c0; c < ce; ++c) {
    const int buf = kBuf == 2 ? (int)((c - c0) & 1) : 0;
    const uint16_t* K = Kt[buf];
    const uint16_t* Qb = Qt[kMode == kFull ? buf : 0];
    const int64_t cn = c + 1 < ce ? c + 1 : c;             // the last chunk loads itself again
    load_tiles(cn);
    if constexpr (kMode == kStates) {
      if (c % kGdrBlk == 0) {
        float* dst = p.blk_S + ((bh * p.n_blks + c / kGdrBlk) * Pp + ch) * kN;
#pragma unroll
        for (int tn = 0; tn < kNT; ++tn)
          *reinterpret_cast<f32x4*>(dst + 16 * tn + 4 * g4) = mine ? S[tn] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    {
      // K S0 (and Q S0), the state already split: operands of one block of 32 state rows are
      // read while the one before is used
      constexpr int kA = kParts == 1 ? kNB : 1;              // bf16: all blocks' operands at once
      bf16x8 ka[kA][2][kParts], qa[kMode == kFull ? kA : 1][2][kParts];
      auto load_k = [&](int kb) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) gdr_frags_t<T, kN>(K, 32 * kb, 16 * rt, lane, ka[kb % kA][rt]);
      };
      auto load_q = [&](int kb) {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) gdr_frags_t<T, kN>(Qb, 32 * kb, 16 * rt, lane, qa[kb % kA][rt]);
      };
      f32x4 R[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}}, Y[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
#pragma unroll
      for (int kb = 0; kb < kA; ++kb) load_k(kb);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int kb = 0; kb < kNB; ++kb) {
        gdr_mma_rows<3>(ka[kb % kA], sb[kb], R);
        if (kb + kA < kNB) load_k(kb + kA);
        if constexpr (kMode == kFull) {
          if (kb + kA >= kNB) load_q(kb + kA - kNB);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      bf16x8 rb[3];
      const f32x4 v0 = ident ? f32x4{0.f, 0.f, 0.f, 0.f} : v[0].get(), v1 = ident ? f32x4{0.f, 0.f, 0.f, 0.f} : v[1].get();
      gdr_split<3>(v0 - fk[0] * R[0], v1 - fk[1] * R[1], rb);
      if constexpr (kMode == kFull) {
#pragma unroll
        for (int kb = 0; kb < kNB; ++kb) {
          gdr_mma_rows<kOut>(qa[kb % kA], sb[kb], Y);
          if (kb + kA < kNB) load_q(kb + kA);
        }
        // one product, then what the vector unit can do of the residual meanwhile
#pragma unroll
        for (int i = 0; i < 4 * kNB; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
          __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
        }
        pin(rb);
        __builtin_amdgcn_sched_barrier(0);
      }
      load_v(cn);
      load_vec(cn, 0, fk);
      f32x4 U[2] = {f32x4{0, 0, 0, 0}, f32x4{0, 0, 0, 0}};
      gdr_mma_rows<3>(tf, rb, U);
#pragma unroll
      for (int tn = 0; tn < kNT; ++tn) S[tn] *= dec;
#pragma unroll
      for (int i = 0; i < 12; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 3, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kMode == kFull) {
        // A residual that is not finite makes every update of its channel NaN, the tokens
        // before it included (T holds zeros for them, and 0 times it is NaN): rare, found in
        // any one of the updates.
        if (__builtin_expect(__ballot(U[0][0] != U[0][0]) != 0, 0)) gdr_from_first<kNT>(tf, rb, U, fq, S, g4);
      }
      load_t(cn);
      if constexpr (kMode == kStates) {
        float* dst = p.u + ((blk0 + c) * Pp + ch) * kC + 4 * g4;
        *reinterpret_cast<f32x4*>(dst) = mine ? U[0] : f32x4{0.f, 0.f, 0.f, 0.f};
        *reinterpret_cast<f32x4*>(dst + 16) = mine ? U[1] : f32x4{0.f, 0.f, 0.f, 0.f};
      }
      constexpr int kT = kParts == 1 ? kNB : 1;
      bf16x8 kt[kT][2][kParts];
      auto load_kt = [&](int t2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) gdr_frags<T, kN>(K, 16 * (2 * t2 + j), 0, lane, kt[t2 % kT][j]);
      };
#pragma unroll
      for (int t2 = 0; t2 < kT; ++t2) load_kt(t2);
      __builtin_amdgcn_sched_barrier(0);
      bf16x8 wb[3];
      gdr_split<3>(fu[0] * U[0], fu[1] * U[1], wb);
      load_vec(cn, 2, fu);
      dec = vec[cn * vstride + 96];
      __builtin_amdgcn_sched_barrier(0);
      // the state two tiles at a time; the tiles before are split meanwhile
#pragma unroll
      for (int t2 = 0; t2 < kNB; ++t2) {
        f32x4 s2[2] = {S[2 * t2], S[2 * t2 + 1]};
        gdr_mma_rows<3>(kt[t2 % kT], wb, s2);
        if (t2 + kT < kNB) load_kt(t2 + kT);
        S[2 * t2] = s2[0];
        S[2 * t2 + 1] = s2[1];
        if (t2 > 0) gdr_split<3>(S[2 * t2 - 2], S[2 * t2 - 1], sb[t2 - 1]);
      }
      if constexpr (kMode == kFull) {
        bf16x8 ub[kOut];
        gdr_split<kOut>(U[0], U[1], ub);
        Y[0] *= fq[0];
        Y[1] *= fq[1];
        gdr_mma_rows<kOut>(pf, ub, Y);
      }
      gdr_split<3>(S[kNT - 2], S[kNT - 1], sb[kNB - 1]);
#pragma unroll
      for (int i = 0; i < 6 * kNB + (kMode == kFull ? 6 : 0); ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x002, 7, 0);
      }
#pragma unroll
      for (int kb = 0; kb < kNB; ++kb) pin(sb[kb]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kMode == kFull) {
        load_vec(cn, 1, fq);
        load_p(cn);
        if (some && (c + 1) * kC <= len) {
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) gdr_store_whole4(yrow + c * kC + 16 * rt + 4 * g4, Y[rt]);
        }
      }
      if constexpr (kBuf == 1) __syncthreads();
      if constexpr (kMode == kFull) {
        if ((c + 1) * kC > len) {                            // the row's end: kept in a free tile, stored last
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) *reinterpret_cast<f32x4*>(end_of(buf) + 4 * rt) = Y[rt];
        }
      }
    }
    if (c + 1 < ce) {
      put(kBuf == 2 ? buf ^ 1 : 0);
      __syncthreads();
    }
  }

  if constexpr (kMode == kFull) {
    if (q.final_state && seg == p.S - 1)
      gdr_store_rows(q.final_state + (bh * q.P + ch0) * q.N, q.P - ch0, q.N, q.state_vec, S, lane);
    // tokens of this segment behind the row's end
    if (mine) {
      if (ce > c0 && ce * kC > len) {
        const float* kept = end_of(kBuf == 2 ? (int)((ce - 1 - c0) & 1) : 0);
        gdr_store_end(yrow, (ce - 1) * kC, len, q.L,
                      {*reinterpret_cast<const f32x4*>(kept), *reinterpret_cast<const f32x4*>(kept + 4)}, g4);
      }
      const int64_t from = (ce > c0 ? ce : c0) * kC, to = c1 * kC < q.L ? c1 * kC : q.L;
      for (int64_t t = from + 4 * g4; t < to; t += 16) gdr_store4(yrow, t, to, f32x4{0.f, 0.f, 0.f, 0.f});
    }
  } else if (kMode == kSummary) {
    float* dst = ident ? p.seg_M + ((bs * q.H + h) * q.N + ch0) * q.N : p.seg_h + ((bs * q.H + h) * q.P + ch0) * q.N;
    gdr_store_rows(dst, channels - ch0, q.N, q.state_vec, S, lane);
  }
}

// ----------------------------------------------------------------------------- carries
// start[0] = initial state, start[s + 1] = start[s] M_s + h_s.  The rows of the state
// are independent: one workgroup per 16 of them, one wave per 16 columns.  Exact fp32
// products (v_mfma_f32_16x16x4_f32).  The chain of segments is latency: a wave keeps its
// columns of the next segment's M in registers (a load per 32 keys where they are used
// cost 338 us at 16 heads, 128 x 128, 16 segments; so it is 46, and 21 at 8 segments).
template <int kN>
__global__ __launch_bounds__(kN * 4) void gdr_carry_kernel(GdrChunkParams p) {
  constexpr int kRow = kN + 4, kThreads = kN * 4, kB = kN / 4;
  __shared__ float A[2][16 * kRow];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6), i16 = lane & 15, g4 = lane >> 4;
  const GdrParams& q = p.g;
  const int64_t tiles = (q.P + 15) / 16;
  const int64_t it = gdr_xcd_item(blockIdx.x, gridDim.x);      // the tiles of a head share M in one L2
  const int64_t bh = it / tiles, b = bh / q.H, h = bh % q.H, p0 = (it % tiles) * 16;
  const int N = (int)q.N;
  const int64_t len = gdr_length(q, b);
  for (int e = tid; e < 16 * kN; e += kThreads) {
    const int row = e / kN, n = e % kN;
    float x = 0.0f;
    if (p0 + row < q.P && n < N) {
      if (q.init) x = q.init[(bh * q.P + p0 + row) * N + n];
      p.seg_start[(((b * p.S) * q.H + h) * q.P + p0 + row) * N + n] = x;
    }
    A[0][row * kRow + n] = x;
  }
  const int n = 16 * w + i16, nc = n < N ? n : N - 1;
  float m[kB], hs[4];
  // no branches around live registers: clamped addresses, and selects where they are used
  auto load = [&](int64_t s) {
    const int64_t sm = (b * (p.S - 1) + s) * q.H + h;
    const float* M = p.seg_M + sm * (int64_t)N * N;
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const int k = 4 * j + g4;
      m[j] = lane_load<float>(M, (uint32_t)((k < N ? k : N - 1) * N + nc) * 4u);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = p0 + 4 * g4 + r;
      hs[r] = p.seg_h[(sm * q.P + (row < q.P ? row : q.P - 1)) * N + nc];
    }
  };
  load(0);
  __syncthreads();
  for (int64_t s = 0; s + 1 < p.S; ++s) {
    const float* a = A[s & 1];
    float mc[kB], hc[4];
#pragma unroll
    for (int j = 0; j < kB; ++j) mc[j] = 4 * j + g4 < N && n < N ? m[j] : 0.0f;
#pragma unroll
    for (int r = 0; r < 4; ++r) hc[r] = n < N && p0 + 4 * g4 + r < q.P ? hs[r] : 0.0f;
    load(s + 2 < p.S ? s + 1 : s);                         // the last segment loads itself again
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kB; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i16 * kRow + 4 * j + g4], mc[j], acc, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 4 * g4 + r;
      // a segment without tokens hands the state on as it is (also what is not finite in it)
      const float x = s * p.seg_chunks * kC < len ? acc[r] + hc[r] : a[row * kRow + n];
      A[(s + 1) & 1][row * kRow + n] = x;                  // zero where n >= N: both terms are
      if (n < N && p0 + row < q.P) p.seg_start[(((b * p.S + s + 1) * q.H + h) * q.P + p0 + row) * N + n] = x;
    }
    __syncthreads();
  }
}

template <typename T, typename O, int kN, bool kBwd>
hipError_t prep_n(const GdrChunkParams& p, hipStream_t s) {
  hipLaunchKernelGGL((gdr_prep_kernel<T, O, kN, kBwd>), dim3((unsigned)(p.g.B * p.g.G * p.n_chunks)), dim3(256), 0, s,
                     p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t prep_t(const GdrChunkParams& p, bool bwd, hipStream_t s) {
  if (bwd) return p.g.N > 64 ? prep_n<T, O, 128, true>(p, s) : prep_n<T, O, 64, true>(p, s);
  return p.g.N > 64 ? prep_n<T, O, 128, false>(p, s) : prep_n<T, O, 64, false>(p, s);
}

template <typename T, typename O, int kN>
hipError_t chunk_n(const GdrChunkParams& p, hipStream_t s) {
  const GdrParams& q = p.g;
  hipError_t e;
  const int64_t vslices = (q.P + 63) / 64, islices = (q.N + 63) / 64;
  if (p.S > 1) {
    hipLaunchKernelGGL((gdr_chain_kernel<T, O, kN, kSummary>),
                       dim3((unsigned)(q.B * (p.S - 1) * q.H * (vslices + islices))), dim3(256), 0, s, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL(gdr_carry_kernel<kN>, dim3((unsigned)(q.B * q.H * ((q.P + 15) / 16))), dim3(kN * 4), 0, s, p);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }
  hipLaunchKernelGGL((gdr_chain_kernel<T, O, kN, kFull>), dim3((unsigned)(q.B * p.S * q.H * vslices)), dim3(256), 0,
                     s, p);
  return hipGetLastError();
}

template <typename T, typename O>
hipError_t chunk_t(const GdrChunkParams& p, hipStream_t s) {
  return p.g.N > 64 ? chunk_n<T, O, 128>(p, s) : chunk_n<T, O, 64>(p, s);
}

template <typename T>
hipError_t states_t(const GdrChunkParams& p, hipStream_t s) {
  const dim3 grid((unsigned)(p.g.B * p.S * p.g.H * ((p.g.P + 63) / 64)));
  if (p.g.N > 64)
    hipLaunchKernelGGL((gdr_chain_kernel<T, float, 128, kStates>), grid, dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((gdr_chain_kernel<T, float, 64, kStates>), grid, dim3(256), 0, s, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_prep(const GdrChunkParams& p, Dt in, Dt grad, bool bwd, hipStream_t s) {
  if (!bwd || in == grad) return in == Dt::BF16 ? prep_t<uint16_t, uint16_t>(p, bwd, s) : prep_t<float, float>(p, bwd, s);
  return in == Dt::BF16 ? prep_t<uint16_t, float>(p, bwd, s) : prep_t<float, uint16_t>(p, bwd, s);
}

hipError_t launch_gdr_states(const GdrChunkParams& p, Dt in, hipStream_t s) {
  return in == Dt::BF16 ? states_t<uint16_t>(p, s) : states_t<float>(p, s);
}

hipError_t launch_gdr_chunk(const GdrChunkParams& p, Dt in, Dt out, hipStream_t s) {
  const hipError_t e = launch_gdr_prep(p, in, in, false, s);
  if (e != hipSuccess) return e;
  if (in == Dt::BF16) return out == Dt::BF16 ? chunk_t<uint16_t, uint16_t>(p, s) : chunk_t<uint16_t, float>(p, s);
  return out == Dt::BF16 ? chunk_t<float, uint16_t>(p, s) : chunk_t<float, float>(p, s);
}

}  // namespace mamba
