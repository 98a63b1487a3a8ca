// fp8.hpp -- e4m3 codes, vectors of eight activations at any alignment, and the
// power-of-two block scale shared by the serving kernels (norm.hip,
// kv_append.hip, attn_paged.hip).
#pragma once

#include "common.hpp"

namespace hyena {

constexpr float FP8_MAX = 448.0f;            // largest finite e4m3 value
constexpr float FP8_MIN_SCALE = 0x1p-96f;    // smallest scale of a cache block
constexpr uint32_t FP8_NAN = 0x7Fu;          // a code that reads as NaN

typedef unsigned u32x4_t __attribute__((ext_vector_type(4)));

// Four floats to four e4m3 codes (round to nearest even; the caller keeps
// |x| <= 448, NaN stays NaN), element 0 in the low byte.
__device__ __forceinline__ uint32_t fp8x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// Codes times a factor, rounded to codes again.
__device__ __forceinline__ uint32_t fp8x4_scale(uint32_t w, float f) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
  return fp8x4(lo[0] * f, lo[1] * f, hi[0] * f, hi[1] * f);
}

// Eight consecutive activations as fp32.  The rows of a strided or odd-length
// tensor need no alignment beyond their element's: global memory takes 16-byte
// accesses at any such address, so one form serves every row.
template <typename IO> struct Vec8;
template <> struct Vec8<bf16_t> {
  u32x4_t w;
  __device__ __forceinline__ void load(const bf16_t* p) { __builtin_memcpy(&w, p, 16); }
  __device__ __forceinline__ float get(int e) const {
    const uint32_t x = w[e >> 1];
    return __uint_as_float((e & 1) ? (x & 0xFFFF0000u) : (x << 16));
  }
  static __device__ __forceinline__ void store(bf16_t* p, const float (&x)[8]) {
    u32x4_t o;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      o[e] = static_cast<uint32_t>(f32_to_bf16(x[2 * e])) |
             (static_cast<uint32_t>(f32_to_bf16(x[2 * e + 1])) << 16);
    __builtin_memcpy(p, &o, 16);
  }
};
template <> struct Vec8<float> {
  u32x4_t a, b;
  __device__ __forceinline__ void load(const float* p) {
    __builtin_memcpy(&a, p, 16);
    __builtin_memcpy(&b, p + 4, 16);
  }
  __device__ __forceinline__ float get(int e) const {
    return __uint_as_float(e < 4 ? a[e] : b[e - 4]);
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    __builtin_memcpy(p, x, 16);
    __builtin_memcpy(p + 4, x + 4, 16);
  }
};

// Elements [0, n) of the eight at p, zero beyond (n >= 8: all of them).
template <typename IO>
__device__ __forceinline__ void load8(const IO* p, int64_t n, float (&x)[8]) {
  if (n >= 8) {
    Vec8<IO> v;
    v.load(p);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = v.get(e);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = e < n ? Io<IO>::ld(p, e) : 0.0f;
  }
}

template <typename IO>
__device__ __forceinline__ void store8(IO* p, int64_t n, const float (&x)[8]) {
  if (n >= 8) {
    Vec8<IO>::store(p, x);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) Io<IO>::st(p, e, x[e]);
  }
}

// |x| as an integer: the order of the magnitudes, NaN above infinity, so an
// integer maximum carries a NaN where a float maximum would drop it.
__device__ __forceinline__ uint32_t mag_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Largest x over the 16 lanes of a row of the wave, in each of them.
__device__ __forceinline__ uint32_t max16(uint32_t x) {
  auto up = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  x = up(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0xB1, 0xF, 0xF, true)));
  x = up(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x4E, 0xF, 0xF, true)));
  x = up(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x141, 0xF, 0xF, true)));
  x = up(x, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(x), 0x140, 0xF, 0xF, true)));
  return x;
}
// and over the wave.
__device__ __forceinline__ uint32_t max64(uint32_t x) {
  x = max16(x);
  const int l = static_cast<int>(threadIdx.x);
  uint32_t o = __float_as_uint(xor16(__uint_as_float(x), l));
  x = x > o ? x : o;
  o = __float_as_uint(xor32(__uint_as_float(x), (l >> 5) & 1));
  return x > o ? x : o;
}

// The smallest power of two s with top / s <= 448 = 1.75 * 2^8, at least
// FP8_MIN_SCALE; top a finite magnitude's bits.  Exact: exponent and mantissa
// are compared as integers.
__device__ __forceinline__ float block_scale(uint32_t top) {
  int e = static_cast<int>(top >> 23) - 8;                 // biased exponent of s
  if ((top & 0x7FFFFFu) > 0x600000u) ++e;                  // mantissa above 1.75
  const int lo = static_cast<int>(__float_as_uint(FP8_MIN_SCALE) >> 23);
  return __uint_as_float(static_cast<uint32_t>(e > lo ? e : lo) << 23);
}

}  // namespace hyena
