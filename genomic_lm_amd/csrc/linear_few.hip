// linear_few.hip -- block-scaled e4m3 products of up to 16 rows (decode steps).
#include "linear_common.hpp"

namespace hyena {

// WN groups of WK waves; a group has NI tiles of 16 columns (of each weight),
// its waves take turns at the runs of K and add their sums in LDS.
template <int WN, int WK, int NI, bool GATED, int OUT>
__global__ __launch_bounds__(WN * WK * 64) void linear_few_kernel(LinearArgs a) {
  constexpr int CN = WN * NI * 16;                 // columns of the workgroup
  constexpr int M = GATED ? 2 * NI : NI;
  __shared__ f32x4 part[WN * WK * M * 64];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wn = wave / WK, wk = wave % WK;
  const int n0 = static_cast<int>(blockIdx.x) * CN + wn * NI * 16;
  const int K = a.K, N = a.N, T = static_cast<int>(a.T);
  const int blocks = (K + RUN - 1) / RUN, full = K / RUN;
  const int row = lane & 15, at = (lane >> 4) * 32;
  const bool token = row < T;
  const uint8_t* px = a.x + (token ? row : 0) * a.x_stride + at;
  const float* psx = a.x_scale + (token ? row : 0) * a.xs_row;
  const uint8_t* pw[M];
  const float* ps[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int c = n0 + (i % NI) * 16;
    const int n = c + row < N ? c + row : N - 1;
    pw[i] = (GATED && i >= NI ? a.w1 : a.w0) + static_cast<int64_t>(n) * K + at;
    ps[i] = (GATED && i >= NI ? a.s1 : a.s0) + static_cast<int64_t>((c < N ? c : N - 1) / RUN) * blocks;
  }
  f32x4 acc[M];
#pragma unroll
  for (int i = 0; i < M; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll 4
  for (int kb = wk; kb < full; kb += WK) {
    const int k = kb * RUN;
    i32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
    if (token) {
      __builtin_memcpy(&lo, px + k, 16);
      __builtin_memcpy(&hi, px + k + 16, 16);
    }
    Frag<true> fx, fw;
    fx.set(pair16(lo, hi));
    const float sx = psx[static_cast<int64_t>(kb) * a.xs_run];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      i32x8 w;
      __builtin_memcpy(&w, pw[i] + k, 32);
      fw.set(w);
      const f32x4 p = mfma_run(fw, fx);
      const float s = sx * ps[i][kb];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], s, acc[i][e]);
    }
  }
  if (full < blocks && wk == full % WK) {           // the last, shorter run
    const int k = full * RUN, left = K - k - at;
    Frag<true> fx, fw;
    fx.set(pair16(codes16(px + k, token ? left : 0), codes16(px + k + 16, token ? left - 16 : 0)));
    const float sx = psx[static_cast<int64_t>(full) * a.xs_run];
#pragma unroll
    for (int i = 0; i < M; ++i) {
      fw.set(pair16(codes16(pw[i] + k, left), codes16(pw[i] + k + 16, left - 16)));
      const f32x4 p = mfma_run(fw, fx);
      const float s = sx * ps[i][full];
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][e] = fmaf(p[e], s, acc[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < M; ++i) part[(wave * M + i) * 64 + lane] = acc[i];
  __syncthreads();

  // wave wk of a group adds the tiles wk, wk + WK, ... of its columns
  float* top = reinterpret_cast<float*>(part);      // codes: magnitudes, after a barrier
  f32x4 h[(NI + WK - 1) / WK];
#pragma unroll
  for (int v = 0; v < (NI + WK - 1) / WK; ++v) {
    const int i = v * WK + wk;
    if (i >= NI) continue;
    f32x4 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      s0 += part[((wn * WK + w) * M + i) * 64 + lane];
      if constexpr (GATED) s1 += part[((wn * WK + w) * M + NI + i) * 64 + lane];
    }
    const int n = n0 + i * 16 + 4 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (GATED) h[v][e] = n + e < N ? gate(s0[e], s1[e], a.act) : 0.0f;
      else h[v][e] = s0[e] + (a.bias && n + e < N ? a.bias[n + e] : 0.0f);
    }
    if constexpr (OUT != OUT_FP8) {
      using O = typename std::conditional<OUT == OUT_BF16, bf16_t, float>::type;
      if (token) {
        O* yr = static_cast<O*>(a.y) + row * a.y_stride;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) Io<O>::st(yr, n + e, h[v][e]);
      }
    }
  }
  if constexpr (OUT == OUT_FP8) {
    static_assert(CN == RUN, "a workgroup has one run of columns");
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int v = 0; v < (NI + WK - 1) / WK; ++v) {
      if (v * WK + wk >= NI) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t b = mag_bits(h[v][e]);
        m = b > m ? b : m;
      }
    }
    uint32_t o = __float_as_uint(xor16(__uint_as_float(m), lane));
    m = o > m ? o : m;
    o = __float_as_uint(xor32(__uint_as_float(m), lane >> 5));
    m = o > m ? o : m;
    if (lane < 16) top[wave * 16 + lane] = __uint_as_float(m);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WN * WK; ++w) {
      const uint32_t b = __float_as_uint(top[w * 16 + row]);
      m = b > m ? b : m;
    }
    const float scale = run_scale(m);
    if (token) {
      if (wave == 0 && lane < 16)
        a.q_scale[static_cast<int64_t>(row) * ((N + RUN - 1) / RUN) + blockIdx.x] = scale;
      uint8_t* yr = static_cast<uint8_t*>(a.y) + row * a.y_stride;
#pragma unroll
      for (int v = 0; v < (NI + WK - 1) / WK; ++v) {
        const int i = v * WK + wk;
        if (i >= NI) continue;
        const float z[4] = {h[v][0], h[v][1], h[v][2], h[v][3]};
        uint32_t w[1];
        to_codes<4>(z, scale, w);
        const int n = n0 + i * 16 + 4 * (lane >> 4);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (n + e < N) yr[n + e] = static_cast<uint8_t>(w[0] >> (8 * e));
      }
    }
  }
}

template <int WN, int WK, int NI, bool GATED, int OUT>
static void few_go(const LinearArgs& a) {
  constexpr int CN = WN * NI * 16;
  linear_few_kernel<WN, WK, NI, GATED, OUT>
      <<<static_cast<unsigned>((a.N + CN - 1) / CN), WN * WK * 64, 0, a.stream>>>(a);
}

hipError_t launch_linear_few(const LinearArgs& a) {
  if (a.out == OUT_FP8) few_go<4, 4, 2, true, OUT_FP8>(a);
  else if (a.w1) {
    if (a.out == OUT_BF16) few_go<1, 8, 1, true, OUT_BF16>(a);
    else few_go<1, 8, 1, true, OUT_F32>(a);
  } else {
    if (a.out == OUT_BF16) few_go<1, 8, 1, false, OUT_BF16>(a);
    else few_go<1, 8, 1, false, OUT_F32>(a);
  }
  return hipGetLastError();
}

// less than 2^32 threads in a grid of the smallest tiles (64 x 64, 256 threads)
bool linear_fits(int64_t T, int64_t N) { return (T + 63) / 64 * ((N + 63) / 64) < (int64_t(1) << 24); }

hipError_t launch_linear(const LinearArgs& a) {
  if (a.T <= LINEAR_FEW_ROWS) return launch_linear_few(a);
  return linear_dma_takes(a) ? launch_linear_dma(a) : launch_linear_tile(a);
}

}  // namespace hyena
