// state_cache.hip -- rows of fp32 or bf16 state kept in 8 bits (gfx950).
//
// A row is any fixed-size per-request state laid out flat (a scan state (D, N),
// a conv state (D, K), an SSD or delta-rule state (H P, N)).  Every 32
// consecutive numbers of a row share one power of two 2^e, the smallest with
// 127 2^e >= max|x| (e >= -126), stored as the byte e + 127; each number is the
// signed byte rint(x / 2^e).  The division by a power of two is exact, so the
// code is one rounding of x whatever carries it out: the error of a number is
// at most 2^(e-1), i.e. between max|x|/254 and max|x|/127 of its group (e stops at
// 121, so that every code stands for a finite number: numbers beyond 127 2^121
// are held to it).  A power
// of two rather than max|x|/127 costs up to one of the 8 bits, and makes the
// stored values independent of any division's rounding and exact in bf16.
// A group that holds an infinity or a NaN gets byte 255 and codes 0 and reads
// back as NaN (0 times the infinity whose pattern 255 << 23 is).
//
// Both kernels stream: 4 (2) bytes and 1.03 bytes per number, one way each, and
// nothing else; HBM-bound.  A thread takes four consecutive numbers, so that
// eight neighbouring lanes hold one group and its maximum is three lane
// exchanges; a wave's reads are 1 KB contiguous.  kU independent pieces per
// thread keep several loads in flight once there is enough work to fill the
// GPU with fewer, longer workgroups.  Measured: 64 rows of 2 MB read in 24 us; call to
// call 24 states of 2.6 MB are parked in 33 us (158 MB, a large copy's rate) and a
// single row takes 12 to 24 us, the launch and the call around it.
#include "device_math.hpp"
#include "kernels.hpp"

namespace mamba {
namespace {

constexpr int kGroup = 32;

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = f32_to_bf16(x); }

__device__ __forceinline__ void load4(const float* p, float (&x)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
}
__device__ __forceinline__ void store4(float* p, const float (&x)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float (&x)[4]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// Slot of row r, or -1 when the row has none (a negative or too large index).
__device__ __forceinline__ int64_t slot_of(const int32_t* slots, int64_t r, int64_t n_slots) {
  const int64_t s = slots ? (int64_t)slots[r] : r;
  return s >= 0 && s < n_slots ? s : -1;
}

// kVec: n % 4 == 0 and every array aligned for four numbers at a time.
template <typename T, bool kVec, int kU>
__global__ __launch_bounds__(256) void cache_write_kernel(CacheParams p) {
  const int64_t per_row = (p.n + 1024 * kU - 1) / (1024 * kU);
  const int64_t r = blockIdx.x / per_row;
  const int64_t slot = slot_of(p.slots, r, p.n_slots);
  if (slot < 0) return;                                  // the whole workgroup: no row to keep
  const T* src = static_cast<const T*>(p.state) + r * p.n;
  int8_t* dst = p.codes + slot * p.n;
  uint8_t* ex = p.exps + slot * p.groups;
  const int64_t base = (blockIdx.x % per_row) * (1024 * kU) + 4 * (int64_t)threadIdx.x;
  float x[kU][4];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = base + 1024 * u;
    if constexpr (kVec) {
      x[u][0] = x[u][1] = x[u][2] = x[u][3] = 0.0f;
      if (i < p.n) load4(src + i, x[u]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[u][j] = i + j < p.n ? load1(src + i + j) : 0.0f;
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = base + 1024 * u;
    // patterns of |x| order like the values, infinities and NaN above all of them
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t a = __builtin_bit_cast(uint32_t, x[u][j]) & 0x7fffffffu;
      top = top > a ? top : a;
    }
#pragma unroll
    for (int m = 1; m < 8; m *= 2) {
      const uint32_t o = (uint32_t)__shfl_xor((int)top, m);
      top = top > o ? top : o;
    }
    // max|x| = 1.M 2^(E - 127), and 127 = 1.111111b 2^6: 2^(E - 133) reaches it
    // unless M is above 111111b in its first six bits
    const int E = (int)(top >> 23);
    int eb = E - 6 + ((top & 0x7fffffu) > 0x7e0000u ? 1 : 0);
    eb = eb < 1 ? 1 : eb > 248 ? 248 : eb;       // above 248 a code of 64 would stand for 2^128
    const bool finite = E < 255;
    const float inv = __builtin_bit_cast(float, (uint32_t)(254 - eb) << 23);   // 2^-(eb - 127)
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      int q = finite ? (int)__builtin_rintf(x[u][j] * inv) : 0;
      q = q > 127 ? 127 : q < -127 ? -127 : q;   // only at eb = 248
      c |= (uint32_t)(q & 0xff) << (8 * j);
    }
    if constexpr (kVec) {
      if (i < p.n) *reinterpret_cast<uint32_t*>(dst + i) = c;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < p.n) dst[i + j] = (int8_t)(c >> (8 * j));
    }
    if ((threadIdx.x & 7) == 0 && i < p.n) ex[i / kGroup] = finite ? (uint8_t)eb : (uint8_t)255;
  }
}

template <typename T, bool kVec, int kU>
__global__ __launch_bounds__(256) void cache_read_kernel(CacheParams p) {
  const int64_t per_row = (p.n + 1024 * kU - 1) / (1024 * kU);
  const int64_t r = blockIdx.x / per_row;
  const int64_t slot = slot_of(p.slots, r, p.n_slots);
  T* dst = static_cast<T*>(p.state) + r * p.n;
  const int8_t* src = p.codes + (slot < 0 ? 0 : slot) * p.n;
  const uint8_t* ex = p.exps + (slot < 0 ? 0 : slot) * p.groups;
  const int64_t base = (blockIdx.x % per_row) * (1024 * kU) + 4 * (int64_t)threadIdx.x;
  uint32_t c[kU], e[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = base + 1024 * u;
    c[u] = e[u] = 0;
    if (slot >= 0 && i < p.n) {                          // a row without a slot reads as zeros
      e[u] = ex[i / kGroup];
      if constexpr (kVec) {
        c[u] = *reinterpret_cast<const uint32_t*>(src + i);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (i + j < p.n) c[u] |= (uint32_t)(uint8_t)src[i + j] << (8 * j);
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kU; ++u) {
    const int64_t i = base + 1024 * u;
    const float step = __builtin_bit_cast(float, e[u] << 23);
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = (float)(int8_t)(c[u] >> (8 * j)) * step;
    if constexpr (kVec) {
      if (i < p.n) store4(dst + i, x);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < p.n) store1(dst + i + j, x[j]);
    }
  }
}

template <typename T, bool kVec, int kU>
hipError_t launch_u(const CacheParams& p, bool write, hipStream_t s) {
  const int64_t wgs = cache_workgroups(p);
  if (write)
    hipLaunchKernelGGL((cache_write_kernel<T, kVec, kU>), dim3((unsigned)wgs), dim3(256), 0, s, p);
  else
    hipLaunchKernelGGL((cache_read_kernel<T, kVec, kU>), dim3((unsigned)wgs), dim3(256), 0, s, p);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_t(const CacheParams& p, bool write, hipStream_t s) {
  if (p.vec) return cache_pieces(p) == 4 ? launch_u<T, true, 4>(p, write, s) : launch_u<T, true, 1>(p, write, s);
  return launch_u<T, false, 1>(p, write, s);
}

}  // namespace

hipError_t launch_state_cache(const CacheParams& p, Dt dt, bool write, hipStream_t s) {
  return dt == Dt::BF16 ? launch_t<uint16_t>(p, write, s) : launch_t<float>(p, write, s);
}

}  // namespace mamba
