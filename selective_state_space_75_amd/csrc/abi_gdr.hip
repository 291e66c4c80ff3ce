// abi_gdr.hip -- the C ABI declared in include/mamba_gdr.h and
// include/mamba_state_cache.h: argument checks, workspace plans and launches.
// Every check runs before any HIP call.
#include "kernels.hpp"
#include "mamba_gdr.h"
#include "mamba_state_cache.h"

namespace {

using mamba::Dt;

constexpr int64_t kMaxElems = int64_t(1) << 46;
constexpr int64_t kMaxGrid = int64_t(1) << 31;

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

int check_cache(const void* state, const int32_t* slots, const void* codes, const void* exps, int64_t rows, int64_t n,
                int64_t n_slots, int dtype) {
  if (!dtype_ok(dtype)) return MAMBA_ERR_DTYPE;
  if (!product_ok(rows, n, 1) || !product_ok(n_slots, n, 1)) return MAMBA_ERR_SHAPE;
  if (!slots && n_slots < rows) return MAMBA_ERR_SHAPE;
  if (!state || !codes || !exps) return MAMBA_ERR_NULL;
  if (!aligned(state, width(dtype)) || (slots && !aligned(slots, 4))) return MAMBA_ERR_ALIGN;
  if (n > (kMaxGrid - 1) / rows * 1024 - 1024) return MAMBA_ERR_SHAPE;
  return MAMBA_OK;
}

mamba::CacheParams cache_params(void* state, const int32_t* slots, int8_t* codes, uint8_t* exps, int64_t rows,
                                int64_t n, int64_t n_slots, int dtype) {
  mamba::CacheParams p{};
  p.state = state; p.slots = slots; p.codes = codes; p.exps = exps;
  p.rows = rows; p.n = n; p.n_slots = n_slots;
  p.groups = (n + 31) / 32;
  p.vec = n % 4 == 0 && aligned(state, dtype == MAMBA_BF16 ? 8 : 16) && aligned(codes, 4);
  return p;
}

}  // namespace

extern "C" {

size_t mamba_gdr_workspace_size(int64_t B, int64_t H, int64_t G, int64_t P, int64_t N, int64_t L,
                                mamba_dtype_t in_dtype) {
  if (!dtype_ok(in_dtype) || !gdr_sizes_ok(B, H, G, P, N, L) || N > 128) return (size_t)-1;
  return 0;
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
  for (const void* ptr : {q, k, v, delta, beta})
    if (!aligned(ptr, width(in_dtype))) return MAMBA_ERR_ALIGN;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {(const void*)A, (const void*)delta_bias, (const void*)initial_state, (const void*)lengths,
                          (const void*)final_state})
    if (ptr && !aligned(ptr, 4)) return MAMBA_ERR_ALIGN;
  if (B * H * ((P + 3) / 4) / 4 + 1 >= kMaxGrid) return MAMBA_ERR_SHAPE;
  (void)workspace;
  (void)workspace_bytes;
  mamba::GdrParams p = gdr_params(q, k, v, delta, beta, A, delta_bias, B, H, G, P, N, L, q_stride, k_stride, v_stride,
                                  scale, flags);
  p.init = initial_state; p.lengths = lengths; p.y = y; p.final_state = final_state;
  p.state_vec = N % 4 == 0 && (!initial_state || aligned(initial_state, 16)) && (!final_state || aligned(final_state, 16));
  return mamba::launch_gdr_step(p, dt_of(in_dtype), dt_of(out_dtype), stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
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
  for (const void* ptr : {q, k, v, delta, beta})
    if (!aligned(ptr, width(in_dtype))) return MAMBA_ERR_ALIGN;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  for (const void* ptr : {(const void*)A, (const void*)delta_bias, (const void*)state, (const void*)slots})
    if (ptr && !aligned(ptr, 4)) return MAMBA_ERR_ALIGN;
  if (B * H * ((P + 3) / 4) / 4 + 1 >= kMaxGrid) return MAMBA_ERR_SHAPE;
  mamba::GdrParams p = gdr_params(q, k, v, delta, beta, A, delta_bias, B, H, G, P, N, 1, q_stride, k_stride, v_stride,
                                  scale, flags);
  p.init = state; p.final_state = state; p.slots = slots; p.n_slots = n_slots; p.y = y;
  p.state_vec = N % 4 == 0 && aligned(state, 16);
  return mamba::launch_gdr_step(p, dt_of(in_dtype), dt_of(out_dtype), stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_state_cache_write(const void* state, const int32_t* slots, int8_t* codes, uint8_t* exps, int64_t rows,
                            int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream) {
  const int st = check_cache(state, slots, codes, exps, rows, n, n_slots, dtype);
  if (st != MAMBA_OK) return st;
  const mamba::CacheParams p = cache_params(const_cast<void*>(state), slots, codes, exps, rows, n, n_slots, dtype);
  return mamba::launch_state_cache(p, dt_of(dtype), true, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

int mamba_state_cache_read(const int8_t* codes, const uint8_t* exps, const int32_t* slots, void* state, int64_t rows,
                           int64_t n, int64_t n_slots, mamba_dtype_t dtype, hipStream_t stream) {
  const int st = check_cache(state, slots, codes, exps, rows, n, n_slots, dtype);
  if (st != MAMBA_OK) return st;
  const mamba::CacheParams p = cache_params(state, slots, const_cast<int8_t*>(codes), const_cast<uint8_t*>(exps), rows,
                                            n, n_slots, dtype);
  return mamba::launch_state_cache(p, dt_of(dtype), false, stream) == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP;
}

}  // extern "C"
