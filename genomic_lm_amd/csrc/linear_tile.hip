// linear_tile.hip -- block-scaled e4m3 products of many rows at any alignment, on LDS
// tiles that pass through registers.
//
// K that is no multiple of 16 puts rows at odd addresses, which loads straight into LDS do
// not take.  333 x 1001 to 1000, fp32: 12.5 to 13.1 us, a chain of four runs per group, one of them on its way
// at a time, and the launch; 8192 x 4097 to 12288, bf16: 830 us, 1.0 PFLOP/s.
#include "linear_tile.hpp"

namespace hyena {

// KG groups of WT x WN waves, each wave with MT x MN tiles of 16 tokens by 16 columns.  The groups share
// the tile and take turns at the runs of K.
template <int WT, int WN, int MT, int MN, int KG, bool GATED, int OUT>
__global__ __launch_bounds__(WT * WN * KG * 64) void linear_tile_kernel(LinearArgs a, int tiles_t, int tiles_n) {
  constexpr int NW = WT * WN, NT = NW * 64;
  constexpr int BT = WT * MT * 16, BN = WN * MN * 16;    // rows of the two staged tiles
  constexpr int CN = GATED ? BN / 2 : BN;                // columns of the output tile
  constexpr int MC = GATED ? MN / 2 : MN;
  constexpr bool WIDE = OUT != OUT_BF16;                 // Frag says why
  constexpr int STEP = NT / 8;
  constexpr int RX = BT / STEP, RW = BN / STEP;
  static_assert(BT % STEP == 0 && BN % STEP == 0, "whole rows per pass");
  static_assert(RUN % (MC * 16) == 0, "a wave's columns lie in one block of the scales");
  constexpr int BUF = (BT + BN) * 8;                     // 16-byte slots
  constexpr int JOIN = (KG - 1) * NW * MN * MT * 1024;   // the other groups' sums
  constexpr int TOPS = OUT == OUT_FP8 ? WN * BT * 4 : 0;
  __shared__ __attribute__((aligned(16)))
  uint8_t sh[2 * KG * BUF * 16 > JOIN + TOPS ? 2 * KG * BUF * 16 : JOIN + TOPS];

  const int tid = static_cast<int>(threadIdx.x) % NT;    // within the group
  const int lane = tid & 63;
  const int kg = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / NT);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  i32x4* const lds = reinterpret_cast<i32x4*>(sh) + kg * 2 * BUF;
  const int wt = wave / WN, wn = wave % WN;

  int ti, ni;
  tile_of(tiles_t, tiles_n, ti, ni);
  const int64_t t0 = static_cast<int64_t>(ti) * BT;
  const int n0 = ni * CN;

  const int K = a.K, N = a.N;
  const int blocks = (K + RUN - 1) / RUN;

  // what this thread stages: chunk `sc` of rows srow, srow + STEP, ...
  const int srow = tid >> 3, sc = tid & 7;
  const uint8_t* px[RX];
  const uint8_t* pw[RW];
#pragma unroll
  for (int i = 0; i < RX; ++i) {
    int64_t t = t0 + srow + i * STEP;
    t = t < a.T ? t : a.T - 1;                           // rows past the end repeat the last one
    px[i] = a.x + t * a.x_stride + sc * 16;
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = srow + i * STEP;
    int n;
    const uint8_t* w = a.w0;
    if constexpr (GATED) {
      const int rr = r % (MN * 16);
      n = n0 + r / (MN * 16) * (MC * 16) + rr % (MC * 16);
      if (rr >= MC * 16) w = a.w1;
    } else {
      n = n0 + r;
    }
    n = n < N ? n : N - 1;
    pw[i] = w + static_cast<int64_t>(n) * K + sc * 16;
  }
  i32x4 rx[RX], rw[RW];
  auto fetch = [&](int kb) {
    const int k = kb * RUN;
    if (k + RUN <= K) {
#pragma unroll
      for (int i = 0; i < RX; ++i) __builtin_memcpy(&rx[i], px[i] + k, 16);
#pragma unroll
      for (int i = 0; i < RW; ++i) __builtin_memcpy(&rw[i], pw[i] + k, 16);
    } else {
      const int left = K - k - sc * 16;
#pragma unroll
      for (int i = 0; i < RX; ++i) rx[i] = codes16(px[i] + k, left);
#pragma unroll
      for (int i = 0; i < RW; ++i) rw[i] = codes16(pw[i] + k, left);
    }
  };
  auto put = [&](int buf) {
    i32x4* b = lds + buf * BUF;
#pragma unroll
    for (int i = 0; i < RX; ++i) b[slot(srow + i * STEP, sc)] = rx[i];
#pragma unroll
    for (int i = 0; i < RW; ++i) b[BT * 8 + slot(srow + i * STEP, sc)] = rw[i];
  };

  // scales: one per token and run, one per block of the weights
  const float* psx[MT];
#pragma unroll
  for (int j = 0; j < MT; ++j) {
    int64_t t = t0 + (wt * MT + j) * 16 + (lane & 15);
    t = t < a.T ? t : a.T - 1;
    psx[j] = a.x_scale + t * a.xs_row;
  }
  const int ncol = n0 + wn * (MC * 16);
  const int64_t sbase = static_cast<int64_t>((ncol < N ? ncol : N - 1) / RUN) * blocks;
  const float* ps0 = a.s0 + sbase;
  const float* ps1 = GATED ? a.s1 + sbase : nullptr;

  f32x4 acc[MN][MT];
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (kg < blocks) {
    fetch(kg);
    put(0);
  }
  if (kg + KG < blocks) fetch(kg + KG);
  tile_sync();
  const int fr = lane & 15, fc = (lane >> 4) * 2;
  int buf = 0;
  for (int k0 = 0; k0 < blocks; k0 += KG, buf ^= 1) {
    const int kb = k0 + kg;
    if (KG > 1 && kb >= blocks) {                        // nothing left for this group
      tile_sync();
      continue;
    }
    const i32x4* bx = lds + buf * BUF;
    const i32x4* bw = bx + BT * 8;
    float sx[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) sx[j] = psx[j][static_cast<int64_t>(kb) * a.xs_run];
    const float w0 = ps0[kb], w1 = GATED ? ps1[kb] : 0.0f;
    Frag<WIDE> fx[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int r = (wt * MT + j) * 16 + fr;
      fx[j].set(pair16(bx[slot(r, fc)], bx[slot(r, fc + 1)]));
    }
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      const int r = (wn * MN + i) * 16 + fr;
      Frag<WIDE> fw;
      fw.set(pair16(bw[slot(r, fc)], bw[slot(r, fc + 1)]));
      const float sw = GATED && i >= MC ? w1 : w0;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const f32x4 p = mfma_run(fw, fx[j]);
        const float s = sx[j] * sw;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s, acc[i][j][e]);
      }
    }
    if (kb + KG < blocks) put(buf ^ 1);
    if (kb + 2 * KG < blocks) fetch(kb + 2 * KG);
    tile_sync();
  }
  if constexpr (KG > 1) join_groups<KG, NW, MT, MN>(acc, sh, kg, wave, lane);
  if (kg > 0) return;

  tile_epilogue<WT, WN, MT, MN, GATED, OUT>(a, acc, t0, ncol, wt, wn, lane, sh + JOIN);
}

template <int WT, int WN, int MT, int MN, int KG, bool GATED>
static void tile_go(const LinearArgs& a) {
  constexpr int BT = WT * MT * 16, CN = WN * MN * 16 / (GATED ? 2 : 1);
  const int64_t tt = (a.T + BT - 1) / BT, tn = (a.N + CN - 1) / CN;
  const unsigned grid = static_cast<unsigned>(tt * tn);
  auto go = [&](auto kernel) {
    kernel<<<grid, WT * WN * KG * 64, 0, a.stream>>>(a, static_cast<int>(tt), static_cast<int>(tn));
  };
  if constexpr (GATED && CN % RUN == 0) go(linear_tile_kernel<WT, WN, MT, MN, KG, GATED, OUT_FP8>);
  else if (a.out == OUT_F32) go(linear_tile_kernel<WT, WN, MT, MN, KG, GATED, OUT_F32>);
  else go(linear_tile_kernel<WT, WN, MT, MN, KG, GATED, OUT_BF16>);
}

// Smaller tiles, whose K two groups of waves share, where those of 128 x 128 leave CUs idle.  Measured
// (us, tiles of 64 x 64 by one group, two, four): fp32 30 x 9662 to 384 60, 49, 45; 333 x 1001 to 1000
// 14.2, 13.5, 14.1; 500 x 1001 to 4000 20, 25, 27; 700 x 301 to 2000 15, 21, 22; bf16 47, 40, 40; 12.8,
// 12.8, 13.2; 18.1, 18.4, 24; 13.7, 14.2, 20: two gain where K is long for the number of tiles, one where
// several tiles share a CU.
hipError_t launch_linear_tile(const LinearArgs& a) {
  const int64_t n128 = (a.T + 127) / 128 * ((a.N + 127) / 128) * (a.gated ? 2 : 1);
  if (a.out == OUT_FP8 && !a.gated) return hipErrorInvalidValue;
  if (a.out == OUT_FP8) tile_go<4, 2, 2, 8, 1, true>(a);
  else if (a.gated) {
    if (n128 >= 256) tile_go<2, 2, 4, 4, 1, true>(a);
    else tile_go<2, 2, 2, 4, 2, true>(a);
  } else {
    if (n128 >= 256) tile_go<2, 2, 4, 4, 1, false>(a);
    else tile_go<2, 2, 2, 2, 2, false>(a);
  }
  return hipGetLastError();
}

}  // namespace hyena
