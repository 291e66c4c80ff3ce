// gdr_mfma.hpp -- matrix-core building blocks of the gated delta rule's chunk
// kernels (gfx950).
//
// Every product is v_mfma_f32_16x16x32_bf16 with fp32 accumulators.  Lane l of a
// wave (i = l & 15, g = l >> 4) holds
//   of A (16 x 32): row i, eight of the 32 contraction indices;
//   of B (32 x 16): column i, the same eight;
//   of the result (16 x 16): column i, rows 4 g .. 4 g + 3.
// Which eight is free as long as A and B agree.  All kernels here take, for lane
// group g, indices 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3: exactly the rows
// that a lane holds of two results stacked on each other.  A result therefore is
// the B operand of the next product as it lies in the registers, and the chain
// state -> residual -> update -> state of a chunk never moves between lanes.
//
// fp32 operands are split into bf16 parts that are multiplied separately.  Three
// parts hold an fp32 number exactly (8 bits each), so products of parts i and j with
// i + j < 3 leave out only terms below 2^-25 of the largest: fp32 accuracy at three
// products for a bf16 operand (exact in one part) times an fp32 one and six for two
// fp32 ones, on units 16 times as fast as the fp32 MFMA.  Each part is rounded to
// nearest, so that the left-out terms have either sign (truncated parts all have
// the number's sign: every product came out 2^-24 too small, and sums over tokens
// kept that).  Results that are rounded to bf16 at once take two parts (2^-17).
#pragma once

#include "gdr.hpp"

namespace mamba {

constexpr int kC = kGdrChunk;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 gdr_mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += sum over parts i, j with i + j < kOrd of a[i] b[j], small terms first
template <int kOrd, int kA, int kB>
__device__ __forceinline__ f32x4 gdr_mma(const bf16x8 (&a)[kA], const bf16x8 (&b)[kB], f32x4 c) {
#pragma unroll
  for (int o = kOrd - 1; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < kA; ++i)
      if (o - i >= 0 && o - i < kB) c = gdr_mfma(a[i], b[o - i], c);
  return c;
}

// The same for several results at once: the products of one result follow each other
// at a distance, so that none waits for the accumulator of the one before.
template <int kOrd, int kA, int kB, int kR>
__device__ __forceinline__ void gdr_mma_rows(const bf16x8 (&a)[kR][kA], const bf16x8 (&b)[kB], f32x4 (&c)[kR]) {
#pragma unroll
  for (int o = kOrd - 1; o >= 0; --o)
#pragma unroll
    for (int i = 0; i < kA; ++i)
      if (o - i >= 0 && o - i < kB) {
#pragma unroll
        for (int r = 0; r < kR; ++r) c[r] = gdr_mfma(a[r][i], b[o - i], c[r]);
      }
}

// a b + c, rounded once.
__device__ __forceinline__ f32x4 gdr_fma(f32x4 a, f32x4 b, f32x4 c) {
  f32x4 r;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = __builtin_fmaf(a[j], b[j], c[j]);
  return r;
}

// Two fp32 numbers rounded to bf16, as one v_cvt_pk_bf16_f32.
__device__ __forceinline__ uint32_t gdr_pack(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Eight fp32 numbers (the rows of two stacked results) -> kParts bf16 operands.
template <int kParts>
__device__ __forceinline__ void gdr_split(f32x4 x, f32x4 y, bf16x8 (&out)[kParts]) {
  float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
#pragma unroll
  for (int s = 0; s < kParts; ++s) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = gdr_pack(v[2 * j], v[2 * j + 1]);
      if (s + 1 < kParts) {
        v[2 * j] -= bf16_lo(w[j]);
        v[2 * j + 1] -= bf16_hi(w[j]);
      }
    }
    out[s] = __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
  }
}

// Keeps the computation of operands where it stands (the compiler moves it past the
// products it should overlap with otherwise).
template <int kParts>
__device__ __forceinline__ void pin(bf16x8 (&x)[kParts]) {
#pragma unroll
  for (int s = 0; s < kParts; ++s) asm volatile("" : "+v"(x[s]));
}

// Operand tiles in LDS: rows of 32 tokens, 36 apart.  72 bytes (18 banks of 64) spread both
// reads of a lane group, 16 rows at one token (gdr_frag) and 4 rows at 16 tokens (gdr_frag_t),
// over most of the banks; rows 7 apart still meet in two.  Measured on the layer (40 heads, L =
// 2048): bank conflicts are 0.38 of the LDS's access cycles in the forward chain, 0.25 in the
// adjoint, 0.27 in the grads and 0.45 in the pairs, which is 0.06, 0.02, 0.07 and 0.13 of their time.
constexpr int kGdrRow = 36;

// A or B operand whose row (column) index runs along the stored row: lane i takes
// column col0 + i of rows row0 + 4 g .. + 3 and row0 + 16 + 4 g .. + 3.  The
// transposing read hands lane i of a 16-lane group column i of the 4 x 16 block
// that the group's addresses cover, row r at lanes 4 r .. 4 r + 3.
template <int kStride>
__device__ __forceinline__ bf16x8 gdr_frag_t(const uint16_t* tile, int row0, int col0, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const uint16_t* p = tile + (row0 + 4 * g + (i >> 2)) * kStride + col0 + 4 * (i & 3);
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 16 * kStride));
  const uint2 x = __builtin_bit_cast(uint2, a), y = __builtin_bit_cast(uint2, b);
  return __builtin_bit_cast(bf16x8, make_uint4(x.x, x.y, y.x, y.y));
}

// A or B operand whose contraction index runs along the stored row: lane i takes
// row row0 + i, numbers col0 + 4 g .. + 3 and col0 + 16 + 4 g .. + 3.
template <int kStride>
__device__ __forceinline__ bf16x8 gdr_frag(const uint16_t* tile, int row0, int col0, int lane) {
  const int g = lane >> 4, i = lane & 15;
  const uint16_t* p = tile + (row0 + i) * kStride + col0 + 4 * g;
  const uint2 x = *reinterpret_cast<const uint2*>(p), y = *reinterpret_cast<const uint2*>(p + 16);
  return __builtin_bit_cast(bf16x8, make_uint4(x.x, x.y, y.x, y.y));
}

// Vectors at any element-aligned global address (the hardware takes unaligned
// dword accesses; rows of odd length start anywhere).
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(2)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

// 16 bytes into a tile row (8-byte aligned)
__device__ __forceinline__ void gdr_put16(uint16_t* dst, uint4 v) {
  reinterpret_cast<uint2*>(dst)[0] = make_uint2(v.x, v.y);
  reinterpret_cast<uint2*>(dst)[1] = make_uint2(v.z, v.w);
}

// Eight consecutive numbers of a row from token t: all of them (whole), or zeros from
// token `end` on.  The two are separate calls so that whole chunks load without
// branches: a load in a divergent branch is waited for where the branch ends.
struct GdrRaw16 {
  uint4 v;
  __device__ __forceinline__ void whole(const uint16_t* p) {
    const u32x4_u x = *reinterpret_cast<const u32x4_u*>(p);
    v = make_uint4(x[0], x[1], x[2], x[3]);
  }
  __device__ __forceinline__ void part(const uint16_t* p, int64_t valid) {
    uint32_t h[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = j < valid ? (uint32_t)p[j] : 0u;
    v = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
  __device__ __forceinline__ void save(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  // into the plane(s) of a tile, as zeros where mask is 0 (else all ones)
  template <int kPlaneStride>
  __device__ __forceinline__ void put(uint16_t* dst, uint32_t mask = ~0u) const {
    gdr_put16(dst, make_uint4(v.x & mask, v.y & mask, v.z & mask, v.w & mask));
  }
};

struct GdrRaw32 {
  f32x4 a, b;
  __device__ __forceinline__ void whole(const float* p) {
    a = *reinterpret_cast<const f32x4_u*>(p);
    b = *reinterpret_cast<const f32x4_u*>(p + 4);
  }
  __device__ __forceinline__ void part(const float* p, int64_t valid) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      a[j] = j < valid ? p[j] : 0.0f;
      b[j] = 4 + j < valid ? p[4 + j] : 0.0f;
    }
  }
  __device__ __forceinline__ void save(float* p) const {
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 4) = b;
  }
  template <int kPlaneStride>
  __device__ __forceinline__ void put(uint16_t* dst, uint32_t mask = ~0u) const {
    bf16x8 part[3];
    gdr_split<3>(a, b, part);
#pragma unroll
    for (int s = 0; s < 3; ++s) {
      const uint4 w = __builtin_bit_cast(uint4, part[s]);
      gdr_put16(dst + s * kPlaneStride, make_uint4(w.x & mask, w.y & mask, w.z & mask, w.w & mask));
    }
  }
};


// A vector at a byte offset of this lane from a base that all lanes share (scalar base
// plus 32-bit offset: no 64-bit address arithmetic per lane).
template <typename V, typename T>
__device__ __forceinline__ V lane_load(const T* base, uint32_t off) {
  return *reinterpret_cast<const V*>(reinterpret_cast<const char*>(base) + off);
}

template <typename V, typename T>
__device__ __forceinline__ void lane_store(T* base, uint32_t off, V x) {
  *reinterpret_cast<V*>(reinterpret_cast<char*>(base) + off) = x;
}

// Four consecutive numbers of a row, kept as they are stored until they are used (a
// conversion would be waited for at the load).
struct GdrFour16 {
  u32x2_u x;
  __device__ __forceinline__ void load(const uint16_t* p) { x = *reinterpret_cast<const u32x2_u*>(p); }
  __device__ __forceinline__ f32x4 get() const { return f32x4{bf16_lo(x[0]), bf16_hi(x[0]), bf16_lo(x[1]), bf16_hi(x[1])}; }
};
struct GdrFour32 {
  f32x4 x;
  __device__ __forceinline__ void load(const float* p) { x = *reinterpret_cast<const f32x4_u*>(p); }
  __device__ __forceinline__ f32x4 get() const { return x; }
};

template <typename T> struct GdrIn;
template <> struct GdrIn<uint16_t> { using Raw = GdrRaw16; using Four = GdrFour16; static constexpr int kParts = 1; };
template <> struct GdrIn<float> { using Raw = GdrRaw32; using Four = GdrFour32; static constexpr int kParts = 3; };

__device__ __forceinline__ void gdr_store_whole4(uint16_t* p, f32x4 x) {
  *reinterpret_cast<u32x2_u*>(p) = u32x2_u{gdr_pack(x[0], x[1]), gdr_pack(x[2], x[3])};
}
__device__ __forceinline__ void gdr_store_whole4(float* p, f32x4 x) { *reinterpret_cast<f32x4_u*>(p) = x; }
__device__ __forceinline__ void gdr_store4(uint16_t* row, int64_t t, int64_t end, f32x4 x) {
  if (t + 4 <= end) {
    *reinterpret_cast<u32x2_u*>(row + t) = u32x2_u{gdr_pack(x[0], x[1]), gdr_pack(x[2], x[3])};
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (t + j < end) row[t + j] = f32_to_bf16(x[j]);
}
__device__ __forceinline__ void gdr_store4(float* row, int64_t t, int64_t end, f32x4 x) {
  if (t + 4 <= end) {
    *reinterpret_cast<f32x4_u*>(row + t) = x;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (t + j < end) row[t + j] = x[j];
}

// A chunk's results x (lane group g: tokens 16 rt + 4 g .. + 3) of the chunk from token t that
// the row of `len` tokens ends in: zeros from `len` on, nothing from L on.
template <typename O>
__device__ __forceinline__ void gdr_store_end(O* row, int64_t t, int64_t len, int64_t L, const f32x4 (&x)[2], int g) {
#pragma unroll
  for (int rt = 0; rt < 2; ++rt) {
    const int64_t at = t + 16 * rt + 4 * g;
    f32x4 v;
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = at + r < len ? x[rt][r] : 0.0f;
    gdr_store4(row, at, L, v);
  }
}

// Between the first and the last product of the chain, adjoint, pair and grad kernels no branch
// is taken by some lanes of a wave only: at such a branch's end the compiler, out of registers
// (only the pairs have some left), may copy some before it re-enables the other lanes.  Lanes
// with nothing of their own read clamped addresses and write what another lane writes, or are
// dropped by the bounds of a buffer.  tests/test_gdr_codegen.py looks at the compiled code.

// Four numbers n .. n + 3 of a state row of N (zeros behind it).
__device__ __forceinline__ f32x4 gdr_load_state(const float* row, int64_t n, int64_t N, bool vec) {
  f32x4 r;
  if (vec) {
    r = *reinterpret_cast<const f32x4*>(row + (n < N ? n : 0));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = row[n + j < N ? n + j : N - 1];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = n + j < N ? r[j] : 0.0f;
  return r;
}

// Number i of `count` consecutive ones at `row`; i >= count is dropped.
__device__ __forceinline__ void gdr_store_within(float* row, int64_t count, int i, float x) {
  const auto buf = __builtin_amdgcn_make_buffer_rsrc(row, 0, (int)(count < kC ? count : kC) * 4, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, x), buf, 4 * i, 0, 0);
}
__device__ __forceinline__ void gdr_store_within(uint16_t* row, int64_t count, int i, float x) {
  const auto buf = __builtin_amdgcn_make_buffer_rsrc(row, 0, (int)(count < kC ? count : kC) * 2, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(x), buf, 2 * i, 0, 0);
}

// A wave's 16 rows of state (kNT tiles of 16 numbers), the first `count` of which are there
// (0 or less: none), to consecutive rows of N at `rows`.
template <int kNT>
__device__ __forceinline__ void gdr_store_rows(float* rows, int64_t count, int64_t N, bool vec, const f32x4 (&S)[kNT],
                                               int lane) {
  constexpr uint32_t kDrop = 0x80000000u;                  // past the buffer's end: not written
  const int bytes = (int)((count < 0 ? 0 : count < 16 ? count : 16) * N * 4);
  const auto buf = __builtin_amdgcn_make_buffer_rsrc(rows, 0, bytes, 0x00020000);
  const int i = lane & 15, g = lane >> 4, width = (int)N;
#pragma unroll
  for (int tn = 0; tn < kNT; ++tn) {
    const int n = 16 * tn + 4 * g;
    const uint32_t at = (uint32_t)(i * width + n) * 4u;
    if (vec) {
      typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[tn]), buf, n < width ? at : kDrop, 0, 0);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (float)S[tn][j]), buf,
                                              n + j < width ? at + 4u * j : kDrop, 0, 0);
    }
  }
}

// The chunk of 32 tokens of a key head, staged by a 256-thread workgroup: kN rows
// (numbers of the head, zeros past N) of 32 tokens in LDS, one plane per part.  Piece
// j of thread t is eight tokens of row t / 4 + 64 j.
template <typename T, int kN>
struct GdrTile {
  static constexpr int kParts = GdrIn<T>::kParts;
  static constexpr int kPlane = kN * kGdrRow;
  static constexpr int kSize = kPlane * kParts;
  static constexpr int kPieces = kN / 64;
  using Raw = typename GdrIn<T>::Raw;
  int64_t row[kPieces];
  Raw raw[kPieces];
  bool ok[kPieces];            // false for rows past N: put as zeros
  __device__ __forceinline__ void init(int64_t N, int tid) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
      const int64_t n = (tid >> 2) + 64 * j;
      ok[j] = n < N;
      row[j] = n < N ? n : N - 1;
    }
  }
  // all 32 tokens from `rows`, whose rows are `stride` apart
  __device__ __forceinline__ void load(const T* rows, int64_t stride, int tid) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) raw[j].whole(rows + row[j] * stride + 8 * (tid & 3));
  }
  // the first `valid` of them, zeros behind
  __device__ __forceinline__ void load_part(const T* rows, int64_t stride, int64_t valid, int tid) {
#pragma unroll
    for (int j = 0; j < kPieces; ++j) raw[j].part(rows + row[j] * stride + 8 * (tid & 3), valid - 8 * (tid & 3));
  }
  __device__ __forceinline__ void put(uint16_t* tile, int tid) const {
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
      raw[j].template put<kPlane>(tile + ((tid >> 2) + 64 * j) * kGdrRow + 8 * (tid & 3), ok[j] ? ~0u : 0u);
  }
  // as they were loaded, into dense rows of 32 (row N - 1 again for rows past it)
  __device__ __forceinline__ void save(T* rows, int tid) const {
#pragma unroll
    for (int j = 0; j < kPieces; ++j)
      raw[j].save(rows + row[j] * kGdrChunk + 8 * (tid & 3));
  }
};

// Where chunk c of the rows at `rows` (stride L) is read: in place, or, when the row
// ends inside it, from its zero-padded copy (stride 32) that the preparation left.
template <typename T>
struct GdrChunkSrc {
  const T* at;
  int64_t stride;
  __device__ __forceinline__ GdrChunkSrc(const T* rows, int64_t L, const T* tail, int64_t c, int64_t len) {
    const bool whole = (c + 1) * kGdrChunk <= len;
    at = whole ? rows + c * kGdrChunk : tail;
    stride = whole ? L : kGdrChunk;
  }
};

template <typename T, int kN>
__device__ __forceinline__ void gdr_frags_t(const uint16_t* tile, int row0, int col0, int lane,
                                            bf16x8 (&f)[GdrIn<T>::kParts]) {
#pragma unroll
  for (int s = 0; s < GdrIn<T>::kParts; ++s) f[s] = gdr_frag_t<kGdrRow>(tile + s * kN * kGdrRow, row0, col0, lane);
}
template <typename T, int kN>
__device__ __forceinline__ void gdr_frags(const uint16_t* tile, int row0, int col0, int lane,
                                          bf16x8 (&f)[GdrIn<T>::kParts]) {
#pragma unroll
  for (int s = 0; s < GdrIn<T>::kParts; ++s) f[s] = gdr_frag<kGdrRow>(tile + s * kN * kGdrRow, row0, col0, lane);
}

// Block (b, h, c) of the preparation's outputs; kBwd: nine planes, else 3 + p_parts.
__device__ __forceinline__ int64_t block_of(const GdrChunkParams& p, int64_t b, int64_t h, int64_t c) {
  return (b * p.g.H + h) * p.n_chunks + c;
}

// Orders a wave's LDS accesses across its lanes (no other wave is involved).
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Work item of workgroup `id` of `n` so that each of the 8 XCDs (workgroups go
// round them) gets a contiguous range: workgroups of one head, which read the
// same keys, then share an L2.
__device__ __forceinline__ int64_t gdr_xcd_item(int64_t id, int64_t n) {
  const int64_t per = n / 8;
  return id >= 8 * per ? id : (id % 8) * per + id / 8;
}

}  // namespace mamba
