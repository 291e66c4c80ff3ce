// abi_gdr.hip -- the C ABI declared in include/mamba_gdr.h and
// include/mamba_state_cache.h: argument checks, workspace plans and launches.
// Every check runs before any HIP call.
#include <atomic>

#include "kernels.hpp"
#include "mamba_gdr.h"
#include "mamba_state_cache.h"

namespace {

using mamba::Dt;

constexpr int64_t kMaxElems = int64_t(1) << 46;

bool aligned(const void* ptr, size_t a) { return (reinterpret_cast<uintptr_t>(ptr) % a) == 0; }
bool dtype_ok(int t) { return t == MAMBA_F32 || t == MAMBA_BF16; }
size_t width(int t) { return t == MAMBA_BF16 ? 2 : 4; }
Dt dt_of(int t) { return t == MAMBA_BF16 ? Dt::BF16 : Dt::F32; }

// a * b * c with every factor >= 1 and the product below kMaxElems
bool product_ok(int64_t a, int64_t b, int64_t c) {
  if (a < 1 || b < 1 || c < 1) return false;
  if (a > kMaxElems / b) return false;
  return a * b <= (kMaxElems - 1) / c;
}

bool gdr_sizes_ok(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L) {
  if (G < 1 || H < 1 || P < 1 || N < 1 || H > kMaxElems / P || G > kMaxElems / N) return false;
  if (!product_ok(B, H * P, L) || !product_ok(B, G * N, L)) return false;
  return H % G == 0 && product_ok(B, H * P, N);
}

// The checks shared by every call of the rule; `rows` are the arrays of
// in_dtype, `words` those of 4-byte elements.
int check_gdr(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L, int64_t qs, int64_t ks, int64_t vs,
              int in_dtype, int out_dtype, unsigned flags) {
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
  if (flags & ~MAMBA_FLAG_QK_NORM) return MAMBA_ERR_UNSUPPORTED;
  if (!gdr_sizes_ok(B, H, G, P, N, L)) return MAMBA_ERR_SHAPE;
  if (N > 128) return MAMBA_ERR_UNSUPPORTED;
  if (qs < G * N * L || ks < G * N * L || vs < H * P * L) return MAMBA_ERR_SHAPE;
  if (qs > kMaxElems / B || ks > kMaxElems / B || vs > kMaxElems / B) return MAMBA_ERR_SHAPE;
  return MAMBA_OK;
}

mamba::GdrParams gdr_params(const void* q, const void* k, const void* v, const void* delta, const void* beta,
                            const float* A, const float* bias, int64_t B, int64_t H, int64_t G, int64_t P, int64_t N,
                            int64_t L, int64_t qs, int64_t ks, int64_t vs, float scale, unsigned flags) {
  mamba::GdrParams p{};
  p.q = q; p.k = k; p.v = v; p.delta = delta; p.beta = beta; p.A = A; p.bias = bias;
  p.B = B; p.H = H; p.G = G; p.P = P; p.N = N; p.L = L; p.n_slots = B;
  p.q_stride = qs; p.k_stride = ks; p.v_stride = vs;
  p.scale = scale;
  p.norm = (flags & MAMBA_FLAG_QK_NORM) ? 1 : 0;
  return p;
}

// Test knobs (mamba_gdr_set_test_knobs), read once per call.
std::atomic<int> g_kernel{0};
std::atomic<int64_t> g_segments{0};

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct GdrPlan {
  bool chunk = false;
  int64_t n_chunks = 0, S = 1, seg_chunks = 0;
  size_t off_planes = 0, off_vec = 0, off_tk = 0, off_tq = 0, off_tv = 0, off_M = 0, off_h = 0, off_start = 0, bytes = 0;
};

// Sizes-only plan of the forward pass.
// Token by token (one launch) while the steps cost less than the chunks' launches, about 27 us
// up to L = 32.  Steps cost more the more rows of state there are beyond about 5000, which
// keep every CU busy, and 1.2 to 1.9 times their neighbours where L is a multiple of 4
// (gdr_step.hip).  The rule ends in front of the first such L that loses.  Measured, call to
// call, token against chunks, in us.  32 heads of 128 x 128: L = 11: 22.8, 27.3; 12: 29.1, 27.0;
// 13: 24.0, 28.5; 15: 26.8, 28.9; 16: 37.9, 27.1; 17: 29.6, 27.3; 24: 55.1, 27.2; 31: 51.7, 27.2.
// 4 heads of 64 x 64: L = 19: 22.8, 27.2; 20: 28.0, 27.2; 21: 23.6, 27.2; 23: 25.4, 27.3; 24: 33.0, 26.9;
// 25: 27.4, 27.3; 31: 32.8, 27.1.  160 heads of 128 x 128: L = 2: 23.5, 28.2; 3: 23.5, 27.7; 4: 38.6, 28.0.
// So it gives up 2 to 4 us at the odd lengths between 12 and 15, or 20 and 23.
// In chunks, L is cut into segments when the 16-channel waves of all heads would leave
// SIMDs idle (there are 1024).  The summary launch then adds the N transition rows to the
// P value rows of every head, so fewer than three segments do not pay, and the two launches
// cost what 16 chunks do.  One wave per SIMD is the aim, in segments of 8 chunks or more, 32
// at most.  128 x 128, one segment, the
// rule's and two or three times as many: 16 heads, L = 32768: 2112, 726 (8), 755 us (24);
// 16 heads, L = 2048: 140, 85 (8), 108 (16); 64 heads, L = 4096: 295 (1), 306 (4).  60 heads
// of 80 x 96, L = 1003: 99 (1), 116 (3).
GdrPlan make_gdr_plan(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L, size_t e) {
  GdrPlan q;
  const int kernel = g_kernel.load();
  const int64_t rows = B * H * P, steps = L * ((rows + 5119) / 5120);
  q.chunk = kernel == 2 || (kernel == 0 && steps > (N > 64 ? 11 : 19));
  if (!q.chunk) return q;
  q.n_chunks = (L + mamba::kGdrChunk - 1) / mamba::kGdrChunk;
  const int64_t waves = B * H * ((P + 15) / 16);
  int64_t S = (1024 + waves / 2) / waves;
  if (S > q.n_chunks / 8) S = q.n_chunks / 8;
  if (S > 32) S = 32;
  if (S < 3 || q.n_chunks - 2 * ((q.n_chunks + S - 1) / S) < 16) S = 1;
  const int64_t forced = g_segments.load();
  if (forced > 0) S = forced < q.n_chunks ? forced : q.n_chunks;
  q.seg_chunks = (q.n_chunks + S - 1) / S;
  q.S = (q.n_chunks + q.seg_chunks - 1) / q.seg_chunks;
  const size_t blocks = size_t(B) * H * q.n_chunks;
  size_t o = 0;
  q.off_planes = o; o += align256(blocks * 6 * mamba::kGdrPlane * sizeof(uint16_t));
  q.off_vec = o; o += align256(blocks * mamba::kGdrVec * sizeof(float));
  q.off_tk = o; o += align256(size_t(B) * G * N * mamba::kGdrChunk * e);
  q.off_tq = o; o += align256(size_t(B) * G * N * mamba::kGdrChunk * e);
  q.off_tv = o; o += align256(size_t(B) * H * P * mamba::kGdrChunk * e);
  if (q.S > 1) {
    const size_t heads = size_t(B) * H;
    q.off_M = o; o += align256(heads * (q.S - 1) * N * N * sizeof(float));
    q.off_h = o; o += align256(heads * (q.S - 1) * P * N * sizeof(float));
    q.off_start = o; o += align256(heads * q.S * P * N * sizeof(float));
  }
  q.bytes = o;
  return q;
}

struct GdrBwdPlan {
  int64_t n_chunks = 0, n_blks = 0;
  size_t off_planes = 0, off_vec = 0, off_tk = 0, off_tq = 0, off_tv = 0, off_tdy = 0, off_u = 0, off_dv = 0, off_S = 0,
         off_dS = 0, off_aq = 0, off_ak = 0, off_part = 0, bytes = 0;
};

GdrBwdPlan make_gdr_bwd_plan(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L, size_t e, size_t eg) {
  GdrBwdPlan q;
  q.n_chunks = (L + mamba::kGdrChunk - 1) / mamba::kGdrChunk;
  q.n_blks = (q.n_chunks + mamba::kGdrBlk - 1) / mamba::kGdrBlk;
  const size_t heads = size_t(B) * H, blocks = heads * q.n_chunks, C = mamba::kGdrChunk;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o += align256(bytes); return at; };
  q.off_planes = take(blocks * 9 * mamba::kGdrPlane * sizeof(uint16_t));
  q.off_vec = take(blocks * mamba::kGdrVecBwd * sizeof(float));
  q.off_tk = take(size_t(B) * G * N * C * e);
  q.off_tq = take(size_t(B) * G * N * C * e);
  q.off_tv = take(heads * P * C * e);
  q.off_tdy = take(heads * P * C * eg);
  const size_t Pp = (P + 63) / 64 * 64, Np = (N + 63) / 64 * 64;
  q.off_u = take(blocks * Pp * C * sizeof(float));
  q.off_dv = take(blocks * Pp * C * sizeof(float));
  q.off_S = take(heads * q.n_blks * Pp * Np * sizeof(float));
  q.off_dS = take(blocks * Pp * Np * sizeof(float));
  if (H > G || P > 64) {     // more than one turn of a key head's sums
    q.off_aq = take(size_t(B) * G * q.n_chunks * Np * C * sizeof(float));
    q.off_ak = take(size_t(B) * G * q.n_chunks * Np * C * sizeof(float));
  }
  q.off_part = take(heads * q.n_blks * 2 * sizeof(float));
  q.bytes = o;
  return q;
}

// Whether every launch of a pass in chunks is one: preparation, summaries and full chain, carries.
bool gdr_chunk_fits(const GdrPlan& q, int64_t B, int64_t H, int64_t G, int64_t P, int64_t N) {
  const int64_t vs = (P + 63) / 64, is = (N + 63) / 64;
  return mamba::launch_fits(B * G * q.n_chunks, 256) && mamba::launch_fits(B * q.S * H * vs, 256) &&
         (q.S == 1 || (mamba::launch_fits(B * (q.S - 1) * H * (vs + is), 256) &&
                       mamba::launch_fits(B * H * ((P + 15) / 16), N > 64 ? 512 : 256)));
}
// The same for the backward pass: preparation, chains, pairs, grads, sums.
bool gdr_bwd_fits(const GdrBwdPlan& q, int64_t B, int64_t H, int64_t G, int64_t P, int64_t N) {
  return mamba::launch_fits(B * G * q.n_chunks, 256) && mamba::launch_fits(B * H * ((P + 63) / 64), 256) &&
         mamba::launch_fits(B * H * q.n_chunks, 256) && mamba::launch_fits(B * G * q.n_blks, N > 64 ? 512 : 256) &&
         mamba::launch_fits(H, 64);
}

int check_cache(const mamba::CacheParams& p, int dtype) {
  if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
  if (!product_ok(p.rows, p.n, 1) || !product_ok(p.n_slots, p.n, 1)) return MAMBA_ERR_SHAPE;
  if (!p.slots && p.n_slots < p.rows) return MAMBA_ERR_SHAPE;
  if (!p.state || !p.codes || !p.exps) return MAMBA_ERR_NULL;
  if (!mamba::launch_fits(mamba::cache_workgroups(p), 256)) return MAMBA_ERR_SHAPE;
  if (!aligned(p.state, width(dtype)) || (p.slots && !aligned(p.slots, 4))) return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

mamba::CacheParams cache_params(void* state, const int32_t* slots, int8_t* codes, uint8_t* exps, int64_t rows,
                                int64_t n, int64_t n_slots, int dtype) {
  mamba::CacheParams p{};
  p.state = state; p.slots = slots; p.codes = codes; p.exps = exps;
  p.rows = rows; p.n = n; p.n_slots = n_slots;
  p.groups = n / 32 + (n % 32 > 0);
  p.vec = n % 4 == 0 && aligned(state, dtype == MAMBA_BF16 ? 8 : 16) && aligned(codes, 4);
  return p;
}

}  // namespace

extern "C" {

size_t mamba_gdr_workspace_size(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                                mamba_dtype_t in_dtype) {
  if (!dtype_ok(in_dtype) || !gdr_sizes_ok(B, H, G, P, N, L) || N > 128) return (size_t)-1;
  return make_gdr_plan(B, H, G, P, N, L, width(in_dtype)).bytes;
}

int mamba_gdr_fwd(const void* q, const void* k, const void* v, const void* delta, const void* beta, const float* A,
                  const float* delta_bias, const float* initial_state, const int32_t* lengths, void* y,
                  float* final_state, int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                  int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, mamba_dtype_t in_dtype,
                  mamba_dtype_t out_dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
  const int st = check_gdr(B, H, G, P, N, L, q_stride, k_stride, v_stride, in_dtype, out_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!q || !k || !v || !delta || !beta || !A || !y) return MAMBA_ERR_NULL;
  const GdrPlan plan = make_gdr_plan(B, H, G, P, N, L, width(in_dtype));
  mamba::GdrParams p = gdr_params(q, k, v, delta, beta, A, delta_bias, B, H, G, P, N, L, q_stride, k_stride, v_stride,
                                  scale, flags);
  p.init = initial_state; p.lengths = lengths; p.y = y; p.final_state = final_state;
  p.state_vec = N % 4 == 0 && (!initial_state || aligned(initial_state, 16)) && (!final_state || aligned(final_state, 16));
  if (plan.chunk ? !gdr_chunk_fits(plan, B, H, G, P, N) : !mamba::launch_fits(mamba::gdr_step_workgroups(p), 256))
    return MAMBA_ERR_SHAPE;
  for (const void* ptr : {q, k, v, delta, beta})
    if (!aligned(ptr, width(in_dtype))) return MAMBA_ERR_ALIGN;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {(const void*)A, (const void*)delta_bias, (const void*)initial_state, (const void*)lengths,
                          (const void*)final_state})
    if (ptr && !aligned(ptr, 4)) return MAMBA_ERR_ALIGN;
  if (plan.bytes && (!workspace || workspace_bytes < plan.bytes)) return MAMBA_ERR_WORKSPACE;
  if (plan.bytes && !aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  if (plan.chunk) {
    mamba::GdrChunkParams c{};
    c.g = p;
    char* ws = static_cast<char*>(workspace);
    c.planes = reinterpret_cast<uint16_t*>(ws + plan.off_planes);
    c.vec = reinterpret_cast<float*>(ws + plan.off_vec);
    c.tail_k = ws + plan.off_tk; c.tail_q = ws + plan.off_tq; c.tail_v = ws + plan.off_tv;
    c.n_chunks = plan.n_chunks; c.S = plan.S; c.seg_chunks = plan.seg_chunks;
    if (plan.S > 1) {
      c.seg_M = reinterpret_cast<float*>(ws + plan.off_M);
      c.seg_h = reinterpret_cast<float*>(ws + plan.off_h);
      c.seg_start = reinterpret_cast<float*>(ws + plan.off_start);
    }
    c.p_parts = out_dtype == MAMBA_BF16 ? 2 : 3;
    c.vec_stride = mamba::kGdrVec;
    return mamba::launch_gdr_chunk(c, dt_of(in_dtype), dt_of(out_dtype), stream) == hipSuccess ? MAMBA_OK
                                                                                              : MAMBA_ERR_HIP;
  }
  return mamba::launch_gdr_step(p, dt_of(in_dtype), dt_of(out_dtype), stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

size_t mamba_gdr_bwd_workspace_size(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                                    mamba_dtype_t in_dtype, mamba_dtype_t grad_dtype) {
  if (!dtype_ok(in_dtype) || !dtype_ok(grad_dtype) || !gdr_sizes_ok(B, H, G, P, N, L) || N > 128) return (size_t)-1;
  return make_gdr_bwd_plan(B, H, G, P, N, L, width(in_dtype), width(grad_dtype)).bytes;
}

int mamba_gdr_bwd(const void* q, const void* k, const void* v, const void* delta, const void* beta, const float* A,
                  const float* delta_bias, const float* initial_state, const int32_t* lengths, const void* dy,
                  const float* dfinal_state, void* dq, void* dk, void* dv, void* ddelta, void* dbeta, float* dA,
                  float* ddelta_bias, float* dinitial_state, int64_t B, int64_t H, int64_t G, int64_t P, int64_t N,
                  int64_t L, int64_t q_stride, int64_t k_stride, int64_t v_stride, float scale, mamba_dtype_t in_dtype,
                  mamba_dtype_t grad_dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
  const int st = check_gdr(B, H, G, P, N, L, q_stride, k_stride, v_stride, in_dtype, grad_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!q || !k || !v || !delta || !beta || !A || !dy || !dq || !dk || !dv || !ddelta || !dbeta || !dA || !ddelta_bias)
    return MAMBA_ERR_NULL;
  for (const void* ptr : {q, k, v, delta, beta})
    if (!aligned(ptr, width(in_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {dy, (const void*)dq, (const void*)dk, (const void*)dv, (const void*)ddelta, (const void*)dbeta})
    if (!aligned(ptr, width(grad_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {(const void*)A, (const void*)delta_bias, (const void*)initial_state, (const void*)lengths,
                          (const void*)dfinal_state, (const void*)dA, (const void*)ddelta_bias,
                          (const void*)dinitial_state})
    if (ptr && !aligned(ptr, 4)) return MAMBA_ERR_ALIGN;
  const GdrBwdPlan plan = make_gdr_bwd_plan(B, H, G, P, N, L, width(in_dtype), width(grad_dtype));
  if (!gdr_bwd_fits(plan, B, H, G, P, N)) return MAMBA_ERR_SHAPE;
  if (!workspace || workspace_bytes < plan.bytes) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  mamba::GdrChunkParams c{};
  c.g = gdr_params(q, k, v, delta, beta, A, delta_bias, B, H, G, P, N, L, q_stride, k_stride, v_stride, scale, flags);
  c.g.init = initial_state; c.g.lengths = lengths;
  c.g.state_vec = N % 4 == 0;
  for (const void* ptr : {(const void*)initial_state, (const void*)dfinal_state, (const void*)dinitial_state})
    if (ptr && !aligned(ptr, 16)) c.g.state_vec = 0;
  char* ws = static_cast<char*>(workspace);
  c.planes = reinterpret_cast<uint16_t*>(ws + plan.off_planes);
  c.vec = reinterpret_cast<float*>(ws + plan.off_vec);
  c.tail_k = ws + plan.off_tk; c.tail_q = ws + plan.off_tq; c.tail_v = ws + plan.off_tv; c.tail_dy = ws + plan.off_tdy;
  c.n_chunks = plan.n_chunks; c.S = 1; c.seg_chunks = plan.n_chunks;
  c.p_parts = 3;
  c.vec_stride = mamba::kGdrVecBwd;
  c.dy = dy; c.dfinal = dfinal_state;
  c.u = reinterpret_cast<float*>(ws + plan.off_u);
  c.dvw = reinterpret_cast<float*>(ws + plan.off_dv);
  c.blk_S = reinterpret_cast<float*>(ws + plan.off_S);
  c.chunk_dS = reinterpret_cast<float*>(ws + plan.off_dS);
  c.acc_dq = reinterpret_cast<float*>(ws + plan.off_aq);
  c.acc_dk = reinterpret_cast<float*>(ws + plan.off_ak);
  c.n_blks = plan.n_blks;
  c.dq = dq; c.dk = dk; c.dv = dv; c.ddelta = ddelta; c.dbeta = dbeta;
  c.dA = dA; c.dbias = ddelta_bias; c.dinit = dinitial_state;
  c.part = reinterpret_cast<float*>(ws + plan.off_part);
  return mamba::launch_gdr_bwd(c, dt_of(in_dtype), dt_of(grad_dtype), stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_gdr_update(float* state, const int32_t* slots, const void* q, const void* k, const void* v,
                     const void* delta, const void* beta, const float* A, const float* delta_bias, void* y, int64_t B,
                     int64_t H, int64_t G, int64_t P, int64_t N, int64_t n_slots, int64_t q_stride, int64_t k_stride,
                     int64_t v_stride, float scale, mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags,
                     hipStream_t stream) {
  const int st = check_gdr(B, H, G, P, N, 1, q_stride, k_stride, v_stride, in_dtype, out_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!product_ok(n_slots, H * P, N) || (!slots && n_slots < B)) return MAMBA_ERR_SHAPE;
  if (!state || !q || !k || !v || !delta || !beta || !A || !y) return MAMBA_ERR_NULL;
  mamba::GdrParams p = gdr_params(q, k, v, delta, beta, A, delta_bias, B, H, G, P, N, 1, q_stride, k_stride, v_stride,
                                  scale, flags);
  p.init = state; p.final_state = state; p.slots = slots; p.n_slots = n_slots; p.y = y;
  p.state_vec = N % 4 == 0 && aligned(state, 16);
  if (!mamba::launch_fits(mamba::gdr_step_workgroups(p), 256)) return MAMBA_ERR_SHAPE;
  for (const void* ptr : {q, k, v, delta, beta})
    if (!aligned(ptr, width(in_dtype))) return MAMBA_ERR_ALIGN;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {(const void*)A, (const void*)delta_bias, (const void*)state, (const void*)slots})
    if (ptr && !aligned(ptr, 4)) return MAMBA_ERR_ALIGN;
  return mamba::launch_gdr_step(p, dt_of(in_dtype), dt_of(out_dtype), stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_gdr_set_test_knobs(int kernel, int64_t segments) {
  if (kernel < 0 || kernel > 2 || segments < 0) return MAMBA_ERR_SHAPE;
  g_kernel.store(kernel);
  g_segments.store(segments);
  return MAMBA_OK;
}

int mamba_state_cache_write(const void* state, const int32_t* slots, int8_t* codes, uint8_t* exps, int64_t rows,
                            int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream) {
  const mamba::CacheParams p = cache_params(const_cast<void*>(state), slots, codes, exps, rows, n, n_slots, dtype);
  const int st = check_cache(p, dtype);
  if (st != MAMBA_OK) return st;
  return mamba::launch_state_cache(p, dt_of(dtype), true, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_state_cache_read(const int8_t* codes, const uint8_t* exps, const int32_t* slots, void* state, int64_t rows,
                           int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream) {
  const mamba::CacheParams p = cache_params(state, slots, const_cast<int8_t*>(codes), const_cast<uint8_t*>(exps), rows,
                                            n, n_slots, dtype);
  const int st = check_cache(p, dtype);
  if (st != MAMBA_OK) return st;
  return mamba::launch_state_cache(p, dt_of(dtype), false, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
