// norm.hip -- residual addition and root-mean-square norm, with an output in
// the activations' type or in e4m3 with scales.
//
// The block's pre / post norms sit between the residual stream and the 8-bit
// in_proj (evo2_flash README, layer_names table: 'blocks.N.pre_norm',
// 'blocks.N.projections').  Per row of D columns
//     s = x + r,   y = s / sqrt(mean(s^2) + eps) * w,   r' = round(s)
// and for the 8-bit output, over the row or over runs of `group` columns,
//     scale = max(max|y| / 448, 2^-140) (1 where y is 0),   q = e4m3(y / scale).
// The norm reads the unrounded sum: y is rounded once.
//
// Every element is read once and written once, ~10 vector operations each:
// HBM bound for many rows, the latency of one load, two reductions and one
// store for few.  A row lives in the registers of W waves, eight consecutive
// columns per lane and step, so x and r are read with 16-byte loads and the
// second reduction (the largest |y|) needs no second read.
//
// 32768 x 4096 bf16 with residual, e4m3 per 128 columns: 166 us, 5.7 TB/s of the
// 944 MB it cannot do without (a 4 GiB copy: 4.75 TB/s counting both ways; three
// of five bytes here are reads).  5000 x 1001 fp32: 17.7 us, 4.5 TB/s.  16 x
// 4096: 4.5 us, a launch and the chain above.
#include "fp8.hpp"
#include "serving.hpp"

namespace hyena {

// Sum (or maximum of magnitude bits) over the W waves of a row, or its LR lanes.
template <int W, int LR>
__device__ __forceinline__ float row_sum(float x, float* sh, int wave) {
  if constexpr (LR < 64) {
#pragma unroll
    for (int o = 1; o < LR; o <<= 1) x += __shfl_xor(x, o);
    return x;
  }
  x = wave_sum(x);
  if constexpr (W == 1) return x;
  if ((threadIdx.x & 63) == 0) sh[wave] = x;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < W; ++i) t += sh[i];
  __syncthreads();
  return t;
}
template <int W, int LR>
__device__ __forceinline__ uint32_t row_max(uint32_t x, float* sh, int wave) {
  if constexpr (LR < 64) {
#pragma unroll
    for (int o = 1; o < LR; o <<= 1) x = max(x, static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), o)));
    return x;
  }
  x = max64(x);
  if constexpr (W == 1) return x;
  if ((threadIdx.x & 63) == 0) sh[wave] = __uint_as_float(x);
  __syncthreads();
  uint32_t t = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t o = __float_as_uint(sh[i]);
    t = t > o ? t : o;
  }
  __syncthreads();
  return t;
}

// W waves of LR = 64 lanes per row, or (W = NV = 1) 64 / LR rows per wave: rows of
// 64 to 256 columns, such as a head's queries, would leave most of a wave idle
// (262144 x 64 bf16 with residual, to bf16 87 and to e4m3 101 us that way, 22 and
// 20 us with eight rows per wave; 262144 x 250 196 and 187, 119 and 113 with two).
// OUT 0: y in the activations' type; 1: e4m3, one scale per row; 2: e4m3, one
// scale per 128 columns (16 lanes).
template <typename IO, int W, int NV, int LR, int OUT>
__global__ __launch_bounds__(W == 1 ? 256 : W * 64) void add_rmsnorm_kernel(
    const IO* x, int64_t x_stride, const IO* residual, int64_t residual_stride,
    const float* __restrict__ weight, float eps, IO* y, int64_t y_stride,
    uint8_t* __restrict__ q, float* __restrict__ q_scale, IO* residual_out,
    int64_t residual_out_stride, int64_t T, int D) {
  __shared__ float sh[W];
  static_assert(LR == 64 || (W == 1 && NV == 1), "several rows per wave: one step");
  const int lane = threadIdx.x & (LR - 1);
  const int wave = W == 1 ? 0 : static_cast<int>(threadIdx.x >> 6);
  const int64_t row = W == 1 ? static_cast<int64_t>(blockIdx.x) * (256 / LR) + threadIdx.x / LR
                             : static_cast<int64_t>(blockIdx.x);
  if (row >= T) return;                 // W == 1 only; it has no barrier
  const IO* xr = x + row * x_stride;

  float s[NV][8];
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = ((v * W + wave) * 64 + lane) * 8;
    load8(xr + c, static_cast<int64_t>(D) - c, s[v]);
  }
  if (residual) {
    const IO* rr = residual + row * residual_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = ((v * W + wave) * 64 + lane) * 8;
      float r[8];
      load8(rr + c, static_cast<int64_t>(D) - c, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] += r[e];
    }
  }
  float ss = 0.0f;
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(s[v][e], s[v][e], ss);
  ss = row_sum<W, LR>(ss, sh, wave);
  // Where the squares or eps leave fp32 (|s| around 1e18 and more), or the squares
  // fall below its normal range (|s| around 1e-17 and less) and eps does not cover
  // them: the same with the row scaled.  By 2^-96 every finite row's squares stay
  // below 2^64 each, by 2^96 those of the smallest values above 2^-106.
  float unit = 1.0f, eps_in = eps;
  if (!(fmaxf(ss, eps) < 0x1p126f)) unit = 0x1p-96f;
  else if (ss < 0x1p-100f && eps < 0x1p-64f) unit = 0x1p96f;
  if (unit != 1.0f) {
    ss = 0.0f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float z = s[v][e] * unit;
        ss = fmaf(z, z, ss);
      }
    ss = row_sum<W, LR>(ss, sh, wave);
    eps_in = eps * unit * unit;
  }
  const float inv = rsqrtf(ss / static_cast<float>(D) + eps_in);

  if (residual_out) {
    IO* ro = residual_out + row * residual_out_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = ((v * W + wave) * 64 + lane) * 8;
      store8(ro + c, static_cast<int64_t>(D) - c, s[v]);
    }
  }
  if (unit != 1.0f) {                   // (not into inv, which would leave the normal range)
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] *= unit;
  }
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int c = ((v * W + wave) * 64 + lane) * 8;
    float w[8];
    if (weight) {
      load8(weight + c, static_cast<int64_t>(D) - c, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] = s[v][e] * inv * w[e];
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) s[v][e] *= inv;
    }
  }

  if constexpr (OUT == 0) {
    IO* yr = y + row * y_stride;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = ((v * W + wave) * 64 + lane) * 8;
      store8(yr + c, static_cast<int64_t>(D) - c, s[v]);
    }
  } else {
    uint32_t top[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      top[v] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t m = mag_bits(s[v][e]);
        top[v] = m > top[v] ? m : top[v];
      }
    }
    if constexpr (OUT == 1) {
#pragma unroll
      for (int v = 1; v < NV; ++v) top[0] = top[v] > top[0] ? top[v] : top[0];
      top[0] = row_max<W, LR>(top[0], sh, wave);
#pragma unroll
      for (int v = 1; v < NV; ++v) top[v] = top[0];
    } else if constexpr (LR < 16) {
      top[0] = row_max<W, LR>(top[0], sh, wave);           // the row is shorter than a group
    } else {
#pragma unroll
      for (int v = 0; v < NV; ++v) top[v] = max16(top[v]);
    }
    const int groups = (D + 127) >> 7;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int c = ((v * W + wave) * 64 + lane) * 8;
      const float a = __uint_as_float(top[v]);
      // NaN: 1, its codes say NaN.  Not below 2^-140: a smaller quotient has too few
      // bits, and y / scale could pass 464, e4m3's end, or be x / 0
      const float scale = a > 0.0f ? fmaxf(a / FP8_MAX, 0x1p-140f) : 1.0f;
      if constexpr (OUT == 1) {
        if (v == 0 && lane == 0 && wave == 0) q_scale[row] = scale;
      } else {
        if ((lane & 15) == 0 && c < D) q_scale[row * groups + (c >> 7)] = scale;
      }
      // codes from the product with 1 / scale; below 2^-100 the reciprocal
      // may overflow and the quotient is taken
      float z[8];
      const float is = 1.0f / scale;
      if (scale >= 0x1p-100f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = s[v][e] * is;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = s[v][e] / scale;
      }
      const uint32_t lo = fp8x4(z[0], z[1], z[2], z[3]), hi = fp8x4(z[4], z[5], z[6], z[7]);
      uint8_t* qp = q + row * D + c;
      if (c + 8 <= D) {
        const uint32_t w[2] = {lo, hi};
        __builtin_memcpy(qp, w, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < D) qp[e] = static_cast<uint8_t>((e < 4 ? lo >> (8 * e) : hi >> (8 * e - 32)) & 0xFFu);
      }
    }
  }
}

template <typename IO, int W, int NV, int LR = 64>
static void norm_out(const NormArgs& a) {
  const unsigned grid = static_cast<unsigned>(W == 1 ? (a.T + 256 / LR - 1) / (256 / LR) : a.T);
  const unsigned block = W == 1 ? 256 : W * 64;
  auto go = [&](auto kernel) {
    kernel<<<grid, block, 0, a.stream>>>(
        static_cast<const IO*>(a.x), a.x_stride, static_cast<const IO*>(a.residual), a.residual_stride,
        a.weight, a.eps, static_cast<IO*>(a.y), a.y_stride, a.q, a.q_scale,
        static_cast<IO*>(a.residual_out), a.residual_out_stride, a.T, a.D);
  };
  if (!a.q) go(add_rmsnorm_kernel<IO, W, NV, LR, 0>);
  else if (a.group == 0) go(add_rmsnorm_kernel<IO, W, NV, LR, 1>);
  else go(add_rmsnorm_kernel<IO, W, NV, LR, 2>);
}

template <typename IO>
static void norm_rows(const NormArgs& a) {
  const int D = a.D;
  if (D <= 64) norm_out<IO, 1, 1, 8>(a);
  else if (D <= 128) norm_out<IO, 1, 1, 16>(a);
  else if (D <= 256) norm_out<IO, 1, 1, 32>(a);
  else if (D <= 512) norm_out<IO, 1, 1>(a);
  else if (D <= 1024) norm_out<IO, 1, 2>(a);
  else if (D <= 2048) norm_out<IO, 4, 1>(a);
  else if (D <= 4096) norm_out<IO, 4, 2>(a);
  else if (D <= 8192) norm_out<IO, 4, 4>(a);
  else norm_out<IO, 16, 4>(a);
}

hipError_t launch_add_rmsnorm(const NormArgs& a) {
  // a grid holds less than 2^32 threads, 1024 per row at most
  constexpr int64_t MOST = 1 << 21;
  const int64_t size = a.bf16 ? 2 : 4;
  auto at = [&](const void* p, int64_t n) {
    return p ? static_cast<const void*>(static_cast<const char*>(p) + n * size) : nullptr;
  };
  for (int64_t t = 0; t < a.T; t += MOST) {
    NormArgs b = a;
    b.T = a.T - t < MOST ? a.T - t : MOST;
    b.x = at(a.x, t * a.x_stride);
    b.residual = at(a.residual, t * a.residual_stride);
    b.y = const_cast<void*>(at(a.y, t * a.y_stride));
    b.residual_out = const_cast<void*>(at(a.residual_out, t * a.residual_out_stride));
    if (a.q) {
      b.q = a.q + t * a.D;
      b.q_scale = a.q_scale + t * (a.group ? (a.D + a.group - 1) / a.group : 1);
    }
    if (a.bf16) norm_rows<bf16_t>(b);
    else norm_rows<float>(b);
  }
  return hipGetLastError();
}

}  // namespace hyena
