// linear_common.hpp -- device pieces of the block-scaled e4m3 products
// (linear_tile.hip, linear_few.hip).
#pragma once

#include "fp8.hpp"
#include "projection.hpp"

namespace hyena {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int RUN = 128;      // columns of K that share a scale

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// One operand of a 16 x 16 tile of a run: lane l holds 32 codes of row l % 16;
// which 32 of the run's 128 columns is free as long as both operands agree.  The
// product gives the lane rows 4 (l / 16) .. + 3 of a (weights) by column l % 16 (tokens).
//
// The matrix unit adds the products of e4m3 codes in groups of eight columns, cut
// below 2^-13 of the group's largest (measured: 2^16 + 2^2 gives 2^16 where both stand
// in one group, and all of it where they do not, on every e4m3 instruction);
// at most 2^-10 of the summed magnitudes, and 1.5e-5 of the sums' norm for normally distributed
// codes, whatever K, against the 1.7e-3 of outputs rounded to bf16.  The caller has a choice: for
// fp32 outputs, and for the scales of 8-bit ones, which are fp32 too, the codes are widened to bf16
// (exact), whose products the unit adds without loss in fp32, at half the rate.
template <bool WIDE> struct Frag;
template <> struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(i32x8 codes) { v = codes; }
};
template <> struct Frag<true> {
  bf16x8 v[4];
  __device__ __forceinline__ void set(i32x8 codes) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = static_cast<uint32_t>(codes[2 * i]), hi = static_cast<uint32_t>(codes[2 * i + 1]);
      const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
      const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
      const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
      const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
      v[i] = bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    }
  }
};
__device__ __forceinline__ f32x4 mfma_run(const Frag<false>& a, const Frag<false>& b) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a.v, b.v, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_run(const Frag<true>& a, const Frag<true>& b) {
  f32x4 c = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v[i], b.v[i], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ i32x8 pair16(i32x4 lo, i32x4 hi) {
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 16 codes at p, of which n (at most 16, maybe none) exist; zero beyond.
__device__ __forceinline__ i32x4 codes16(const uint8_t* p, int n) {
  i32x4 v = {0, 0, 0, 0};
  if (n >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else {
    for (int e = 0; e < n; ++e) v[e >> 2] |= static_cast<int>(p[e]) << (8 * (e & 3));
  }
  return v;
}

// act(g) * u, in forms without a difference of near equals.
//
// The gelu is g Phi(g), Phi(-|g|) = exp(-g^2 / 2) erfcx(|g| / sqrt 2) / 2, where erfcx(z) =
// exp(z^2) erfc(z) = t q(t), t = 1 / (1 + 0.35 z), with a polynomial q fitted over all z >= 0
// (least squares at Chebyshev points, reweighted towards the largest error): with the coefficients as
// they stand here, in fp32, within a relative 3.5e-8 of it, taken in 64 bits.  About 20
// instructions; the device library's erfc, ten times that, took a fifth of the time of a gated
// product of 8192 x 4096 to 11008.
template <int ACT>
__device__ __forceinline__ float gate(float g, float u) {
  if constexpr (ACT == ACT_GELU) {
    const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(g), 0.24748737341529164f, 1.0f));
    float q = 0.007330488879233599f;
    q = fmaf(q, t, 0.005140664987266064f);
    q = fmaf(q, t, -0.10037992149591446f);
    q = fmaf(q, t, 0.13765418529510498f);
    q = fmaf(q, t, -0.02970522828400135f);
    q = fmaf(q, t, 0.11713682115077972f);
    q = fmaf(q, t, 0.12056729942560196f);
    q = fmaf(q, t, 0.16200152039527893f);
    q = fmaf(q, t, 0.18532025814056396f);
    q = fmaf(q, t, 0.19746758043766022f);
    q = fmaf(q, t, 0.19746634364128113f);
    const float h = 0.5f * __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f) * (q * t);
    g *= g < 0.0f ? h : 1.0f - h;
  } else if constexpr (ACT == ACT_GELU_TANH) {           // g / (1 + exp(-2 z)); 2 sqrt(2 / pi) log2 e
    g *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-2.3022081982148305f * fmaf(0.044715f * g * g, g, g)));
  } else if constexpr (ACT == ACT_SILU) {
    g *= __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
  }
  return g * u;
}
// f(act as a constant)
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == ACT_GELU) f(std::integral_constant<int, ACT_GELU>{});
  else if (act == ACT_GELU_TANH) f(std::integral_constant<int, ACT_GELU_TANH>{});
  else if (act == ACT_SILU) f(std::integral_constant<int, ACT_SILU>{});
  else f(std::integral_constant<int, ACT_NONE>{});
}

// The scale of a run whose largest magnitude has the bits `top`, and codes of
// its values, by the rules of hyena_add_rmsnorm_fp8.
__device__ __forceinline__ float run_scale(uint32_t top) {
  const float a = __uint_as_float(top);
  return a > 0.0f ? fmaxf(a / FP8_MAX, 0x1p-140f) : 1.0f;
}
template <int N>
__device__ __forceinline__ void to_codes(const float (&x)[N], float scale, uint32_t (&w)[N / 4]) {
  float z[N];
  if (scale >= 0x1p-100f) {
    const float is = 1.0f / scale;
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = x[e] * is;
  } else {                              // 1 / scale may overflow
#pragma unroll
    for (int e = 0; e < N; ++e) z[e] = x[e] / scale;
  }
#pragma unroll
  for (int e = 0; e < N; e += 4) w[e / 4] = fp8x4(z[e], z[e + 1], z[e + 2], z[e + 3]);
}

// LDS place of 16-byte chunk c of row r: any 8 and any 16 consecutive rows have
// their chunks c in different banks.
__device__ __forceinline__ int slot(int r, int c) {
  return r * 8 + (c ^ (r & 7) ^ ((r >> 3) & 1));
}

// A lane's two chunks of row lane % 16 of a tile of 16 rows.
__device__ __forceinline__ i32x8 tile_codes(const uint8_t* tile, int lane) {
  const int r = lane & 15, c = (lane >> 4) * 2, swz = (r & 7) ^ (r >> 3);
  return pair16(*reinterpret_cast<const i32x4*>(tile + r * RUN + (c ^ swz) * 16),
                *reinterpret_cast<const i32x4*>(tile + r * RUN + ((c + 1) ^ swz) * 16));
}

typedef __attribute__((address_space(3))) void lds_ptr;

// A wave's value where the compiler has not seen that it is one.
__device__ __forceinline__ uint64_t scalar(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(u >> 32));
  return lo | (static_cast<uint64_t>(hi) << 32);
}
// 16 bytes (4) per lane from base + off straight into LDS, lane l at dst + 16 l (4 l);
// base and dst are the wave's.  Written as assembly so that the compiler, which cannot tell
// the halves of the LDS buffer apart, does not make every LDS read of one half wait for the
// loads into the other; the kernels wait for them themselves.  They write no vector
// registers.  A load that reads m0 needs one wait state after its write, one whose base a
// v_readfirstlane (or a restored spill's v_readlane) wrote needs five; the compiler adds none
// in front of assembly: the move and the s_nop are five.  They cost 0 to 3 % (64 x 4096 to 12288
// 21.6 -> 22.3 us).
// m0 is named as written, though the compiler keeps no value there (hence its warning): a write of
// its own is not moved across.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(dst)),
               "v"(off), "s"(scalar(base))
               : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dword %1, %2" ::"s"(
                   __builtin_amdgcn_readfirstlane(dst)),
               "v"(off), "s"(scalar(base))
               : "memory", "m0");
}
#pragma clang diagnostic pop
// All but N of this wave's loads have arrived.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace hyena
