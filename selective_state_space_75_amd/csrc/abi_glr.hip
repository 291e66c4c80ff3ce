// abi_glr.hip -- the C ABI declared in include/mamba_glr.h and include/mamba_norm.h:
// argument checks, plans and launches.  Every check runs before any HIP call.
#include <atomic>

#include "kernels.hpp"
#include "mamba_glr.h"
#include "mamba_norm.h"

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

bool stride_ok(int64_t s, int64_t B, int64_t row) { return s >= row && s <= kMaxElems / B; }
bool all_aligned(std::initializer_list<const void*> ptrs, size_t a) {
  for (const void* ptr : ptrs)
    if (ptr && !aligned(ptr, a)) return false;
  return true;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Test knobs (mamba_glr_set_test_knobs), read while a call's plan is made.
std::atomic<int> g_waves{0};
std::atomic<int64_t> g_segments{0};

struct GlrPlan {
  int64_t S = 1, seg_len = 0;
  int64_t group = 1, groups = 1;                // backward: segments of a workgroup, workgroups of a row
  int waves = 1;
  int lanes = 0;                                // short rows: lanes of a row, several rows a wave
};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// L in S segments of a multiple of 8 tokens each, as even as that allows.
void cut(GlrPlan& q, int64_t L, int64_t S) {
  q.seg_len = ceil_div(ceil_div(L, S), mamba::kGlrLane) * mamba::kGlrLane;
  q.S = ceil_div(L, q.seg_len);
}

// Short rows go several to a wave (unless a test asks for waves or segments).  32768 rows, bf16, forward and backward in us,
// with a wave a row before: 8 tokens 6 (30) and 10 (63), 64: 11 (30), 18 (62), 100: 15 (46), 28 (90), 256: 24 (30),
// 45 (62); with a row a wave, 512: 48 (36), 84 (66), so not past 256.
constexpr int64_t kShort = 256;
bool short_rows(GlrPlan& q, int64_t L) {
  if (L > kShort || g_waves.load() > 0 || g_segments.load() > 0) return false;
  cut(q, L, 1);
  for (q.lanes = 1; q.lanes * mamba::kGlrLane < L;) q.lanes *= 2;
  return true;
}

// Sizes-only plan of the forward pass: waves per row, and segments of L.
// A workgroup's waves lie one after the other on the row, so more of them read longer stretches at a time, and
// a row of up to 16 waves' tokens is one tile.  1, 2, 4, 8, 16 waves, in us: 20480 rows, L = 2048: 82.2, 80.3,
// 78.7; 4096 rows, L = 32768: 280, 280, 275, 267, 250; 1536 rows, L = 8192: 39.4, 35.4, 28.7, 28.4, 29.4; 16
// rows, L = 4096: 14.6, 10.5, 8.0, 7.0.  Rows of two tiles are the exception where there are rows enough for
// every wave slot: 7680 rows, L = 1000: 20.1, 21.2 (2000 rows, L = 2000: 15.6, 14.2).
// Few rows are cut into segments of a tile of 4 waves, in two launches, as many as make 1024 workgroups.
// One segment of 16 waves against that: 16 rows, L = 32768: 18.6, 10.6 (16 segments); 64 rows: 18.8, 15.1 (16);
// 512 rows: 38.3, 54.8 (4).
GlrPlan make_glr_plan(int64_t B, int64_t D, int64_t L) {
  GlrPlan q;
  if (short_rows(q, L)) return q;
  const int64_t rows = B * D, tiles = ceil_div(L, mamba::kGlrWave);
  int64_t waves = tiles <= 2 && rows >= 4096 ? 1 : 16, S = 1;
  if (rows <= 128 && tiles >= 16) {
    S = tiles / 4 < 1024 / rows ? tiles / 4 : 1024 / rows;
    waves = 4;
  }
  const int forced = g_waves.load();
  if (forced > 0) waves = forced;
  const int64_t forced_s = g_segments.load();
  if (forced_s > 0) S = forced_s;
  cut(q, L, S);
  const int64_t own = ceil_div(q.seg_len, mamba::kGlrWave);
  q.waves = (int)(waves < own ? waves : own);
  return q;
}

// The backward pass: a workgroup holds a segment on the chip, a row of up to 16 waves in one.  Longer rows are
// cut.  With 512 rows or more a workgroup takes all segments of a row, of 4 waves each (three such workgroups
// share a CU, of 8 waves one: 2560 rows, L = 16384, bf16: 213 us, 263), and the first launch reads three arrays
// instead of five; below that, a workgroup takes one segment of 8 waves.  One segment against all, bf16,
// L = 32768, in us: 128 rows: 45, 68; 256: 63, 73; 512: 116, 110; 900: 194, 183; 1300: 270, 241; L = 12000, 512 rows:
// 50, 49.
GlrPlan make_glr_bwd_plan(int64_t B, int64_t D, int64_t L) {
  GlrPlan q;
  if (short_rows(q, L)) return q;
  const int forced = g_waves.load();
  const bool many = B * D >= 512;
  const int64_t waves = forced > 0 ? forced : L <= 16 * mamba::kGlrWave ? 16 : many ? 4 : 8;
  int64_t S = ceil_div(L, waves * mamba::kGlrWave);
  const int64_t forced_s = g_segments.load();
  if (forced_s > S) S = forced_s;
  cut(q, L, S);
  q.waves = (int)ceil_div(q.seg_len, mamba::kGlrWave);
  if (many && q.waves <= 8) q.group = q.S;
  q.groups = ceil_div(q.S, q.group);
  return q;
}

bool glr_sizes_ok(int64_t B, int64_t D, int64_t L) { return product_ok(B, D, L); }

int check_glr(const mamba::GlrParams& p, int in_dtype, int out_dtype, unsigned flags) {
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
  if (flags & ~MAMBA_FLAG_BLEND) return MAMBA_ERR_UNSUPPORTED;
  if (!glr_sizes_ok(p.B, p.D, p.L)) return MAMBA_ERR_SHAPE;
  const int64_t row = p.D * p.L;
  if (!stride_ok(p.x_stride, p.B, row) || !stride_ok(p.r_stride, p.B, row)) return MAMBA_ERR_SHAPE;
  if ((p.i && !stride_ok(p.i_stride, p.B, row)) || (p.z && !stride_ok(p.z_stride, p.B, row))) return MAMBA_ERR_SHAPE;
  if (!p.x || !p.r || (!p.blend && !p.A)) return MAMBA_ERR_NULL;
  if (!all_aligned({p.x, p.r, p.i, p.z}, width(in_dtype))) return MAMBA_ERR_ALIGN;
  if (!all_aligned({p.A, p.r_bias, p.i_bias, p.init, p.lengths, p.slots, p.final_state}, 4)) return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

mamba::GlrParams glr_params(const void* x, const void* r, const void* i, const void* z, const float* A,
                            const float* r_bias, const float* i_bias, int64_t B, int64_t D, int64_t L, int64_t xs,
                            int64_t rs, int64_t is, int64_t zs, unsigned flags) {
  mamba::GlrParams p{};
  p.x = x; p.r = r; p.i = i; p.z = z;
  p.A = A; p.r_bias = r_bias; p.i_bias = i ? i_bias : nullptr;
  p.B = B; p.D = D; p.L = L; p.n_slots = B;
  p.x_stride = xs; p.r_stride = rs; p.i_stride = is; p.z_stride = zs;
  p.blend = (flags & MAMBA_FLAG_BLEND) ? 1 : 0;
  p.S = 1;
  return p;
}

size_t glr_bytes(const GlrPlan& q, int64_t B, int64_t D) {
  return q.S > 1 ? align256(size_t(B) * D * q.S * 2 * sizeof(float)) : 0;
}
size_t glr_bwd_sum_bytes(const GlrPlan& q, int64_t B, int64_t D) {
  return q.S > 1 ? align256(size_t(B) * D * q.S * (q.groups > 1 ? 3 : 2) * sizeof(float)) : 0;
}
size_t glr_bwd_bytes(const GlrPlan& q, int64_t B, int64_t D) {
  return glr_bwd_sum_bytes(q, B, D) + align256(size_t(B) * q.groups * 3 * D * sizeof(float));
}

bool norm_sizes_ok(int64_t B, int64_t D, int64_t L, int64_t G) {
  return product_ok(B, D, L) && G >= 1 && D % G == 0;
}

size_t norm_part_bytes(const mamba::NormPlan& q, int64_t D) { return align256(size_t(q.parts) * 2 * D * sizeof(float)); }
size_t norm_stat_bytes(const mamba::NormPlan& q, int64_t B, int64_t L, int64_t G, int numbers) {
  return q.kind == mamba::kNormColTwo ? size_t(B) * G * q.chunks * numbers * L * sizeof(float) : 0;
}

// The plan depends on the element widths and on z; the workspace is enough for all of them.
size_t norm_fwd_bytes(int64_t B, int64_t D, int64_t L, int64_t G) {
  size_t most = 0;
  for (int in : {2, 4}) {
    const size_t n = norm_stat_bytes(mamba::norm_plan(B, D, L, G, in, 0, false), B, L, G, 2);
    if (n > most) most = n;
  }
  return most;
}
size_t norm_bwd_bytes(int64_t B, int64_t D, int64_t L, int64_t G) {
  size_t most = 0;
  for (int grad : {2, 4}) {
    for (bool gate : {false, true}) {
      const mamba::NormPlan q = mamba::norm_plan(B, D, L, G, 2, grad, gate);
      const size_t n = norm_part_bytes(q, D) + norm_stat_bytes(q, B, L, G, 4);
      if (n > most) most = n;
    }
  }
  return most;
}

// Whether every launch is one; items: tokens and groups (forward) or parts and groups (backward).
bool norm_fits(const mamba::NormPlan& q, int64_t B, int64_t D, int64_t L, int64_t G, int64_t items) {
  if (q.kind == mamba::kNormColTwo)
    return mamba::launch_fits(B * G * q.chunks * q.tiles, q.threads) &&
           mamba::launch_fits(B * ceil_div(L, 8 * q.apply_lanes) * G * ceil_div(D / G, q.apply_chans), mamba::kNormApplyThreads);
  return mamba::launch_fits(items, q.threads);
}

int check_norm(const mamba::NormParams& p, int in_dtype, int out_dtype, unsigned flags) {
  if (!dtype_ok(in_dtype) || !dtype_ok(out_dtype)) return MAMBA_ERR_DTYPE;
  if (flags & ~MAMBA_FLAG_RMS) return MAMBA_ERR_UNSUPPORTED;
  if (!norm_sizes_ok(p.B, p.D, p.L, p.G)) return MAMBA_ERR_SHAPE;
  if (!stride_ok(p.x_stride, p.B, p.D * p.L) || (p.z && !stride_ok(p.z_stride, p.B, p.D * p.L))) return MAMBA_ERR_SHAPE;
  if (!(p.eps >= 0.0f)) return MAMBA_ERR_UNSUPPORTED;
  if (!p.x) return MAMBA_ERR_NULL;
  if (!all_aligned({p.x, p.z}, width(in_dtype)) || !all_aligned({p.weight, p.bias}, 4)) return MAMBA_ERR_ALIGN;
  return MAMBA_OK;
}

mamba::NormParams norm_params(const void* x, const void* z, const float* weight, const float* bias, int64_t B, int64_t D,
                              int64_t L, int64_t G, int64_t xs, int64_t zs, float eps, unsigned flags) {
  mamba::NormParams p{};
  p.x = x; p.z = z; p.weight = weight; p.bias = bias;
  p.B = B; p.D = D; p.L = L; p.G = G;
  p.x_stride = xs; p.z_stride = zs;
  p.eps = eps;
  p.rms = (flags & MAMBA_FLAG_RMS) ? 1 : 0;
  return p;
}

// After the checks: G >= 1.
void norm_set(mamba::NormParams& p, const mamba::NormPlan& q) {
  p.Dg = p.D / p.G;
  p.inv_dg = (float)(1.0 / (double)p.Dg);
  p.tiles = q.tiles;
  p.team = q.lanes;
  p.parts = q.parts;
  p.chunks = q.chunks; p.chunk = q.chunk; p.apply_chans = q.apply_chans;
}

int status_of(hipError_t e) { return e == hipSuccess ? MAMBA_OK : MAMBA_ERR_HIP; }

}  // namespace

extern "C" {

size_t mamba_glr_workspace_size(int64_t B, int64_t D, int64_t L) {
  if (!glr_sizes_ok(B, D, L)) return (size_t)-1;
  return glr_bytes(make_glr_plan(B, D, L), B, D);
}

int mamba_glr_fwd(const void* x, const void* r, const void* i, const void* z, const float* A, const float* r_bias,
                  const float* i_bias, const float* initial_state, const int32_t* lengths, void* y, float* final_state,
                  int64_t B, int64_t D, int64_t L, int64_t x_stride, int64_t r_stride, int64_t i_stride,
                  int64_t z_stride, mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags, void* workspace,
                  size_t workspace_bytes, hipStream_t stream) {
  mamba::GlrParams p = glr_params(x, r, i, z, A, r_bias, i_bias, B, D, L, x_stride, r_stride, i_stride, z_stride, flags);
  p.init = initial_state; p.lengths = lengths; p.y = y; p.final_state = final_state;
  const int st = check_glr(p, in_dtype, out_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!y) return MAMBA_ERR_NULL;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  const GlrPlan q = make_glr_plan(B, D, L);
  if (!mamba::launch_fits(B * D * q.S, 64 * q.waves)) return MAMBA_ERR_SHAPE;
  const size_t need = glr_bytes(q, B, D);
  if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  p.S = q.S; p.seg_len = q.seg_len; p.waves = q.waves; p.lanes = q.lanes;
  p.sum = static_cast<float*>(workspace);
  return status_of(mamba::launch_glr_fwd(p, dt_of(in_dtype), dt_of(out_dtype), stream));
}

int mamba_glr_update(float* state, const int32_t* slots, const void* x, const void* r, const void* i, const void* z,
                     const float* A, const float* r_bias, const float* i_bias, void* y, int64_t B, int64_t D,
                     int64_t n_slots, int64_t x_stride, int64_t r_stride, int64_t i_stride, int64_t z_stride,
                     mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags, hipStream_t stream) {
  mamba::GlrParams p = glr_params(x, r, i, z, A, r_bias, i_bias, B, D, 1, x_stride, r_stride, i_stride, z_stride, flags);
  p.final_state = state; p.slots = slots; p.n_slots = n_slots; p.y = y;
  const int st = check_glr(p, in_dtype, out_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!product_ok(n_slots, D, 1) || (!slots && n_slots < B)) return MAMBA_ERR_SHAPE;
  if (!state || !y) return MAMBA_ERR_NULL;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  if (!mamba::launch_fits(B * ceil_div(D, 256), 256)) return MAMBA_ERR_SHAPE;
  return status_of(mamba::launch_glr_update(p, dt_of(in_dtype), dt_of(out_dtype), stream));
}

size_t mamba_glr_bwd_workspace_size(int64_t B, int64_t D, int64_t L) {
  if (!glr_sizes_ok(B, D, L)) return (size_t)-1;
  return glr_bwd_bytes(make_glr_bwd_plan(B, D, L), B, D);
}

int mamba_glr_bwd(const void* x, const void* r, const void* i, const void* z, const float* A, const float* r_bias,
                  const float* i_bias, const float* initial_state, const int32_t* lengths, const void* dy,
                  const float* dfinal_state, void* dx, void* dr, void* di, void* dz, float* dA, float* dr_bias,
                  float* di_bias, float* dinitial_state, int64_t B, int64_t D, int64_t L, int64_t x_stride,
                  int64_t r_stride, int64_t i_stride, int64_t z_stride, mamba_dtype_t in_dtype,
                  mamba_dtype_t grad_dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                  hipStream_t stream) {
  mamba::GlrParams p = glr_params(x, r, i, z, A, r_bias, i_bias, B, D, L, x_stride, r_stride, i_stride, z_stride, flags);
  p.init = initial_state; p.lengths = lengths;
  const int st = check_glr(p, in_dtype, grad_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!dy || !dx || !dr || (i && !di) || (z && !dz) || (!p.blend && !dA) || !dr_bias || (i && !di_bias))
    return MAMBA_ERR_NULL;
  if (!all_aligned({dy, dx, dr, di, dz}, width(grad_dtype))) return MAMBA_ERR_ALIGN;
  if (!all_aligned({dfinal_state, dA, dr_bias, di_bias, dinitial_state}, 4)) return MAMBA_ERR_ALIGN;
  const GlrPlan q = make_glr_bwd_plan(B, D, L);
  if (B * D > kMaxElems / q.S || !mamba::launch_fits(B * D * q.S, 64 * q.waves)) return MAMBA_ERR_SHAPE;
  const size_t need = glr_bwd_bytes(q, B, D);
  if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  p.S = q.S; p.seg_len = q.seg_len; p.waves = q.waves; p.lanes = q.lanes; p.group = q.group; p.groups = q.groups;
  p.sum = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + glr_bwd_sum_bytes(q, B, D));
  p.dy = dy; p.dfinal = dfinal_state;
  p.dx = dx; p.dr = dr; p.di = i ? di : nullptr; p.dz = z ? dz : nullptr;
  p.dA = p.blend ? nullptr : dA; p.dr_bias = dr_bias; p.di_bias = i ? di_bias : nullptr;
  p.dinit = dinitial_state;
  return status_of(mamba::launch_glr_bwd(p, dt_of(in_dtype), dt_of(grad_dtype), stream));
}

int mamba_glr_set_test_knobs(int waves, int64_t segments) {
  if (waves < 0 || waves > 16 || segments < 0) return MAMBA_ERR_SHAPE;
  g_waves.store(waves);
  g_segments.store(segments);
  return MAMBA_OK;
}

size_t mamba_layer_norm_workspace_size(int64_t B, int64_t D, int64_t L, int64_t groups) {
  if (!norm_sizes_ok(B, D, L, groups)) return (size_t)-1;
  return norm_fwd_bytes(B, D, L, groups);
}

int mamba_layer_norm_fwd(const void* x, const void* z, const float* weight, const float* bias, void* y, int64_t B,
                         int64_t D, int64_t L, int64_t groups, int64_t x_stride, int64_t z_stride, float eps,
                         mamba_dtype_t in_dtype, mamba_dtype_t out_dtype, unsigned flags, void* workspace,
                         size_t workspace_bytes, hipStream_t stream) {
  mamba::NormParams p = norm_params(x, z, weight, bias, B, D, L, groups, x_stride, z_stride, eps, flags);
  p.y = y;
  const int st = check_norm(p, in_dtype, out_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!y) return MAMBA_ERR_NULL;
  if (!aligned(y, width(out_dtype))) return MAMBA_ERR_ALIGN;
  const mamba::NormPlan q = mamba::norm_plan(B, D, L, groups, (int)width(in_dtype), 0, z != nullptr);
  const bool by_part = q.kind == mamba::kNormRowBlock || q.kind == mamba::kNormRowWide;
  if (!norm_fits(q, B, D, L, groups, by_part ? q.parts * groups : B * groups * q.tiles)) return MAMBA_ERR_SHAPE;
  const size_t need = norm_fwd_bytes(B, D, L, groups);
  if (need && (!workspace || workspace_bytes < need)) return MAMBA_ERR_WORKSPACE;
  if (need && !aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  norm_set(p, q);
  p.stat = static_cast<float*>(workspace);
  return status_of(mamba::launch_norm_fwd(p, q, dt_of(in_dtype), dt_of(out_dtype), stream));
}

size_t mamba_layer_norm_bwd_workspace_size(int64_t B, int64_t D, int64_t L, int64_t groups) {
  if (!norm_sizes_ok(B, D, L, groups)) return (size_t)-1;
  return norm_bwd_bytes(B, D, L, groups);
}

int mamba_layer_norm_bwd(const void* x, const void* z, const float* weight, const float* bias, const void* dy, void* dx,
                         void* dz, float* dweight, float* dbias, int64_t B, int64_t D, int64_t L, int64_t groups,
                         int64_t x_stride, int64_t z_stride, float eps, mamba_dtype_t in_dtype,
                         mamba_dtype_t grad_dtype, unsigned flags, void* workspace, size_t workspace_bytes,
                         hipStream_t stream) {
  mamba::NormParams p = norm_params(x, z, weight, bias, B, D, L, groups, x_stride, z_stride, eps, flags);
  const int st = check_norm(p, in_dtype, grad_dtype, flags);
  if (st != MAMBA_OK) return st;
  if (!dy || !dx || (z && !dz) || !dweight || !dbias) return MAMBA_ERR_NULL;
  if (!all_aligned({dy, dx, dz}, width(grad_dtype)) || !all_aligned({dweight, dbias}, 4)) return MAMBA_ERR_ALIGN;
  const mamba::NormPlan q = mamba::norm_plan(B, D, L, groups, (int)width(in_dtype), (int)width(grad_dtype), z != nullptr);
  if (!norm_fits(q, B, D, L, groups, q.parts * groups) || !mamba::launch_fits(ceil_div(2 * D, 64), 1024))
    return MAMBA_ERR_SHAPE;
  norm_set(p, q);
  const size_t need = norm_bwd_bytes(B, D, L, groups);
  if (!workspace || workspace_bytes < need) return MAMBA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MAMBA_ERR_ALIGN;
  p.dy = dy; p.dx = dx; p.dz = z ? dz : nullptr; p.dweight = dweight; p.dbias = dbias;
  p.part = static_cast<float*>(workspace);
  p.stat = reinterpret_cast<float*>(static_cast<char*>(workspace) + norm_part_bytes(q, D));
  return status_of(mamba::launch_norm_bwd(p, q, dt_of(in_dtype), dt_of(grad_dtype), stream));
}

}  // extern "C"
