// linear_few.hip -- block-scaled e4m3 products of few rows (decode steps) or few outputs, and the
// choice among the products.
//
// Bound by reading the weights up to about 32 rows: 16 x 11008 to 4096 10.5 to 11.5 us by card, 4.0 to 4.3
// TB/s; 1 x 4096 to 12288 9.6 us, 5.2 TB/s from the last-level cache; gated 4 x 4096 to 11008 18 us,
// 5.0 TB/s.  Beyond, by the tokens that every workgroup loads for its 16 or 32 columns: 64 x 4096
// to 4096 9.0 to 9.6 us, 1.9 TB/s.
#include "linear_common.hpp"

namespace hyena {

// The waves' sums to the output: each wave leaves its part, MT x M tiles, in LDS, at part + STRIDE
// wave, where no other wave reads or writes before; then the waves add the parts of
// different tiles.  NI tiles of columns at n0.
template <int WK, int MT, int NI, int STRIDE, bool GATED, int OUT>
__device__ __forceinline__ void few_join(const LinearArgs& a, const f32x4 (&acc)[GATED ? 2 * NI : NI][MT],
                                         f32x4* part, int n0, int wave, int lane) {
  constexpr int M = GATED ? 2 * NI : NI;
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) part[wave * STRIDE + (i * MT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  using O = typename std::conditional<OUT == OUT_BF16, bf16_t, float>::type;
  for (int v = wave; v < NI * MT; v += WK) {
    const int i = v / MT, j = v % MT;
    f32x4 s0 = {0.0f, 0.0f, 0.0f, 0.0f}, s1 = s0;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      s0 += part[w * STRIDE + v * 64 + lane];
      if constexpr (GATED) s1 += part[w * STRIDE + (NI * MT + v) * 64 + lane];
    }
    const int row = j * 16 + (lane & 15);
    if (row >= a.T) continue;
    O* const yr = static_cast<O*>(a.y) + row * a.y_stride;
    const int n = n0 + i * 16 + 4 * (lane >> 4);
    if constexpr (GATED)
      with_act(a.act, [&](auto act) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s0[e] = gate<decltype(act)::value>(s0[e], s1[e]);
      });
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (n + e >= a.N) continue;
      if constexpr (GATED) Io<O>::st(yr, n + e, s0[e]);
      else Io<O>::st(yr, n + e, s0[e] + (a.bias ? a.bias[n + e] : 0.0f));
    }
  }
}

// The rows of the workgroup: R of them from R blockIdx.y on.
template <int R, int OUT>
__device__ __forceinline__ void few_rows(LinearArgs& a) {
  const int64_t t0 = static_cast<int64_t>(blockIdx.y) * R;
  a.x += t0 * a.x_stride;
  a.x_scale += t0 * a.xs_row;
  a.y = static_cast<uint8_t*>(a.y) + t0 * a.y_stride * (OUT == OUT_BF16 ? 2 : 4);
  a.T = a.T - t0 < R ? a.T - t0 : R;
}

// For rows of whole 16-byte chunks.  A wave has NI tiles of 16 columns (of each weight) and up to
// 16 MT tokens, and takes every WK-th run of K, through a ring of two runs in LDS of its own,
// filled straight from memory: loads of operands to registers, 16 rows in one instruction, pass
// the address unit at a quarter of its 64 bytes per cycle (16 x 11008 to 4096 14.0 us that way,
// 11 this).  No wave waits for another before the end, where their sums are added.
template <int WK, int MT, int NI, bool GATED, int OUT>
__global__ __launch_bounds__(WK * 64) void linear_few_dma_kernel(LinearArgs a) {
  constexpr int M = GATED ? 2 * NI : NI, W = GATED ? 2 : 1;
  constexpr int TILE = 16 * RUN;
  constexpr int SB = TILE * (MT + M), BUF = SB + 256 * (1 + W);    // tokens, weights, their scales
  constexpr int LOADS = 2 * (MT + M) + 1 + W;
  static_assert(BUF * 2 >= MT * M * 1024, "the wave's part fits its ring");
  __shared__ __attribute__((aligned(16))) uint8_t sh[WK * 2 * BUF];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  few_rows<16 * MT, OUT>(a);
  uint8_t* const ring = sh + wave * (2 * BUF);
  const uint32_t ring0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr*)(ring)));
  const int n0 = static_cast<int>(blockIdx.x) * (NI * 16);
  const int K = a.K, N = a.N, T = static_cast<int>(a.T);
  const int blocks = (K + RUN - 1) / RUN;
  const int mine = blocks > wave ? (blocks - wave + WK - 1) / WK : 0;    // runs of this wave
  // a load fills eight rows of 128 bytes, lane l place l % 8 of row l / 8 (slot: rows 8 .. 15 of a
  // tile have their chunks swapped in pairs)
  const int lrow = lane >> 3;
  const int chunk = ((lane & 7) ^ lrow) * 16;
  uint32_t ox[2 * MT], ow[2 * NI];
#pragma unroll
  for (int h = 0; h < 2 * MT; ++h) {
    const int r = h * 8 + lrow;
    ox[h] = static_cast<uint32_t>(r < T ? r : T - 1) * static_cast<uint32_t>(a.x_stride) + (chunk ^ ((h & 1) << 4));
  }
#pragma unroll
  for (int h = 0; h < 2 * NI; ++h) {
    const int r = h * 8 + lrow;
    ow[h] = static_cast<uint32_t>(n0 + r < N ? r : N - 1 - n0) * static_cast<uint32_t>(K) + (chunk ^ ((h & 1) << 4));
  }
  const uint8_t* const w0 = a.w0 + static_cast<int64_t>(n0) * K;
  const uint8_t* const w1 = GATED ? a.w1 + static_cast<int64_t>(n0) * K : nullptr;
  const int tok = lane % (16 * MT);
  const uint32_t os = static_cast<uint32_t>(tok < T ? tok : T - 1) * static_cast<uint32_t>(a.xs_row) * 4u;
  static_assert(RUN % (NI * 16) == 0, "a workgroup's columns lie in one block of the scales");
  const int64_t sbase = static_cast<int64_t>(n0 / RUN) * blocks;
  auto ask = [&](int r) __attribute__((always_inline)) {
    const int kb = wave + r * WK, k = kb * RUN;
    const uint32_t to = ring0 + (r & 1) * BUF;
    dma4(a.x_scale + static_cast<int64_t>(kb) * a.xs_run, os, to + SB);
    dma4(a.s0 + sbase + kb, 0, to + SB + 256);
    if constexpr (GATED) dma4(a.s1 + sbase + kb, 0, to + SB + 512);
    const i32x4 zero = {0, 0, 0, 0};
    i32x4* const z = reinterpret_cast<i32x4*>(ring + (r & 1) * BUF) + lane;
#pragma unroll
    for (int p = 0; p < 2; ++p) {                // even loads, odd loads: one chunk each
      if (k + (chunk ^ (p << 4)) < K) {
#pragma unroll
        for (int h = p; h < 2 * MT; h += 2) dma16(a.x + k, ox[h], to + h * 1024);
#pragma unroll
        for (int h = p; h < 2 * NI; h += 2) {
          dma16(w0 + k, ow[h], to + MT * TILE + h * 1024);
          if constexpr (GATED) dma16(w1 + k, ow[h], to + (MT + NI) * TILE + h * 1024);
        }
      } else {                                   // beyond K, a multiple of 16: zeros
#pragma unroll
        for (int h = p; h < 2 * (MT + M); h += 2) z[h * 64] = zero;
      }
    }
  };

  f32x4 acc[M][MT];
#pragma unroll
  for (int i = 0; i < M; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (mine > 0) ask(0);
  if (mine > 1) ask(1);
  for (int r = 0; r < mine; ++r) {
    if (r + 1 < mine) wait_loads<LOADS>();       // the next run's may be on their way
    else wait_loads<0>();
    const uint8_t* const b = ring + (r & 1) * BUF;
    Frag<true> fx[MT], fw;
    float sx[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      fx[j].set(tile_codes(b + j * TILE, lane));
      sx[j] = reinterpret_cast<const float*>(b + SB)[j * 16 + (lane & 15)];
    }
#pragma unroll
    for (int i = 0; i < M; ++i) {
      fw.set(tile_codes(b + (MT + i) * TILE, lane));
      const float s = *reinterpret_cast<const float*>(b + SB + (GATED && i >= NI ? 512 : 256));
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const f32x4 p = mfma_run(fw, fx[j]);
        const float f = sx[j] * s;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], f, acc[i][j][e]);
      }
    }
    if (r + 2 < mine) {
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");     // read, before it is overwritten
      ask(r + 2);
    }
  }
  few_join<WK, MT, NI, 2 * BUF / 16, GATED, OUT>(a, acc, reinterpret_cast<f32x4*>(sh), n0, wave, lane);
}

// WK waves share NI tiles of 16 columns (of each weight): they take turns at U runs of K each,
// whose loads are all under way before the first product, and add their sums in LDS.
template <int WK, int NI, int U, bool GATED, int OUT>
__global__ __launch_bounds__(WK * 64) void linear_few_kernel(LinearArgs a) {
  constexpr int M = GATED ? 2 * NI : NI;
  __shared__ f32x4 part[WK * M * 64];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  few_rows<16, OUT>(a);
  const int n0 = static_cast<int>(blockIdx.x) * (NI * 16);
  const int K = a.K, N = a.N, T = static_cast<int>(a.T);
  const int blocks = (K + RUN - 1) / RUN, full = K / RUN;
  const int row = lane & 15, at = (lane >> 4) * 32;
  const bool token = row < T;
  const uint8_t* const px = a.x + (token ? row : 0) * a.x_stride + at;
  const float* const psx = a.x_scale + (token ? row : 0) * a.xs_row;
  // the tiles of a workgroup lie in one block of the scales
  static_assert(RUN % (NI * 16) == 0, "one block of the scales");
  typedef const __attribute__((address_space(4))) float* cptr;
  const int64_t sbase = static_cast<int64_t>(n0 / RUN) * blocks;
  const cptr ps0 = (cptr)(a.s0 + sbase), ps1 = (cptr)(GATED ? a.s1 + sbase : a.s0);
  const uint8_t* pw[M];
#pragma unroll
  for (int i = 0; i < M; ++i) {
    const int c = n0 + (i % NI) * 16 + row;
    pw[i] = (GATED && i >= NI ? a.w1 : a.w0) + static_cast<int64_t>(c < N ? c : N - 1) * K + at;
  }
  f32x4 acc[M][1];
#pragma unroll
  for (int i = 0; i < M; ++i) acc[i][0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  auto add = [&](i32x8 x, const i32x8 (&w)[M], float sx, float w0, float w1) __attribute__((always_inline)) {
    Frag<true> fx, fw;
    fx.set(x);
#pragma unroll
    for (int i = 0; i < M; ++i) {
      fw.set(w[i]);
      const f32x4 p = mfma_run(fw, fx);
      const float s = sx * (GATED && i >= NI ? w1 : w0);
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][0][e] = fmaf(p[e], s, acc[i][0][e]);
    }
  };

  for (int k0 = wave * U; k0 < full; k0 += WK * U) {
    i32x8 x[U], w[U][M];
    float sx[U], w0[U], w1[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u < full ? k0 + u : full - 1;        // past the end: loaded, not added
      const int k = kb * RUN;
#pragma unroll
      for (int i = 0; i < M; ++i) __builtin_memcpy(&w[u][i], pw[i] + k, 32);
      x[u] = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
      if (token) __builtin_memcpy(&x[u], px + k, 32);
      sx[u] = psx[static_cast<int64_t>(kb) * a.xs_run];
      w0[u] = ps0[kb];
      w1[u] = GATED ? ps1[kb] : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k0 + u < full) add(x[u], w[u], sx[u], w0[u], w1[u]);
  }
  if (full < blocks && wave == full / U % WK) {                // the last, shorter run
    const int k = full * RUN, left = K - k - at;
    const i32x8 x = pair16(codes16(px + k, token ? left : 0), codes16(px + k + 16, token ? left - 16 : 0));
    i32x8 w[M];
#pragma unroll
    for (int i = 0; i < M; ++i) w[i] = pair16(codes16(pw[i] + k, left), codes16(pw[i] + k + 16, left - 16));
    add(x, w, psx[static_cast<int64_t>(full) * a.xs_run], ps0[full], GATED ? ps1[full] : 0.0f);
  }
  few_join<WK, 1, NI, M * 64, GATED, OUT>(a, acc, part, n0, wave, lane);
}

template <int WK, int MT, int NI, bool GATED, int OUT>
static void few_dma_go(const LinearArgs& a) {
  const dim3 grid(static_cast<unsigned>((a.N + NI * 16 - 1) / (NI * 16)),
                  static_cast<unsigned>((a.T + MT * 16 - 1) / (MT * 16)));
  linear_few_dma_kernel<WK, MT, NI, GATED, OUT><<<grid, WK * 64, 0, a.stream>>>(a);
}
// Eight waves to a workgroup where there are few; four, with more workgroups to a CU, and two
// tiles of columns for each reading of the tokens, where there are many.  Measured (us, weights
// from the last-level cache unless said): 16 x 11008 to 4096 (256 workgroups)
// 11.5 with eight waves, 12.8 with four; 1 x 4096 to 12288 9.6 with two tiles, 9.9 with one, 11.2
// with eight waves (from HBM 12.9, 13.0, 14.0); gated 4 x 4096 to 11008 19.9 with eight waves, 18.0 with
// four; 32 x 4096 to 12288 14.0 with one tile of columns, 13.6 with two, to 4096 7.7, 8.8; 64 x 4096 to
// 12288 23.3, 21.9, to 4096 9.6, 12.0.
template <bool GATED, int OUT>
static void few_pick(const LinearArgs& a) {
  const bool many = a.N > 16 * 512;
  if (!linear_dma_takes(a)) {
    const dim3 grid(static_cast<unsigned>((a.N + 15) / 16), static_cast<unsigned>((a.T + 15) / 16));
    linear_few_kernel<8, 1, 4, GATED, OUT><<<grid, 512, 0, a.stream>>>(a);
  } else if (a.T <= 16) {
    if (!many) few_dma_go<8, 1, 1, GATED, OUT>(a);
    else if constexpr (GATED) few_dma_go<4, 1, 1, true, OUT>(a);
    else few_dma_go<4, 1, 2, false, OUT>(a);
  } else if (a.T <= 32) {
    if (!GATED && many) few_dma_go<4, 2, 2, false, OUT>(a);
    else few_dma_go<4, 2, 1, GATED, OUT>(a);
  } else {
    if (!GATED && many) few_dma_go<4, 4, 2, false, OUT>(a);
    else few_dma_go<4, 4, 1, GATED, OUT>(a);
  }
}

hipError_t launch_linear_few(const LinearArgs& a) {
  if (a.gated) {
    if (a.out == OUT_BF16) few_pick<true, OUT_BF16>(a);
    else few_pick<true, OUT_F32>(a);
  } else {
    if (a.out == OUT_BF16) few_pick<false, OUT_BF16>(a);
    else few_pick<false, OUT_F32>(a);
  }
  return hipGetLastError();
}

// less than 2^32 threads in a grid of the smallest tiles (64 x 64, 256 threads)
bool linear_fits(int64_t T, int64_t N) { return (T + 63) / 64 * ((N + 63) / 64) < (int64_t(1) << 24); }

// Up to 64 rows (16 without the loads straight to LDS), and more of them as further workgroups up to
// 512, 256 without those loads: their waves split K finer than the tiles' do.  The rings of 33 rows or
// more take 84 to 102 KB, so one workgroup goes to a CU and more than 256 make a second round.  Measured
// (us, few-row kernel, then tiles; bf16 outputs): 128 x 4096 to 512 (64 workgroups) 9.1, 10.4; to 2048
// (256) 9.3, 10.4; 192 x 4096 to 4096 (768) 23, 11; 256 30, 12; K = 4097: 48 rows to 1024 (192) 18.0, 19.1; 128 to
// 512 (256) 18.2, 19.7; 65 to 1024 (320) 25, 19.  Between 256 and 512 the rule is older than the tiles'
// present ends, with which they are the faster: 128 x 4096 to 4096 (512) 16.9, 10.8 (fp32 16.9, 15.6); 512 x
// 11008 to 1024 (512) 34, 29.
static bool few_takes(const LinearArgs& a, bool dma) {
  const int64_t parts = dma ? (a.T + 63) / 64 : (a.T + 15) / 16;
  return parts == 1 || parts * ((a.N + 15) / 16) <= (dma ? 512 : 256);
}

// A workgroup that makes e4m3 codes has runs of 128 columns whole.  Where that leaves CUs idle, less
// than 300 tiles of 256 x 128, h goes through memory in fp32 and its codes are made in a second
// launch.  Measured (us, one launch, then two): 4 x 4096 to 11008 109, 21; 128 109, 43; 400 115, 112; 600
// (258 tiles) 213, 141; 1000 x 2048 to 5504 (172) 70, 66.  A little above 300, where one launch is a round and a
// part, two are the faster as well (1000 x 4096 to 11008, 344 tiles: 221, 184), for a workspace of 4 T N bytes.
size_t linear_workspace(int64_t T, int64_t N) {
  return (T + 255) / 256 * ((N + 127) / 128) < 300 ? static_cast<size_t>(T) * static_cast<size_t>(N) * 4 : 0;
}

hipError_t launch_linear(const LinearArgs& a) {
  if (a.out == OUT_FP8 && linear_workspace(a.T, a.N)) {
    LinearArgs b = a;
    b.out = OUT_F32;
    b.y = a.workspace;
    b.y_stride = a.N;
    const hipError_t e = launch_linear(b);
    if (e != hipSuccess) return e;
    return launch_quantize(QuantArgs{a.workspace, a.N, static_cast<uint8_t*>(a.y), a.q_scale, RUN, 1, a.T, a.N,
                                     false, a.stream});
  }
  const bool dma = linear_dma_takes(a);
  if (a.out != OUT_FP8 && few_takes(a, dma)) return launch_linear_few(a);
  return dma ? launch_linear_dma(a) : launch_linear_tile(a);
}

}  // namespace hyena
