// linear_dma.hip -- block-scaled e4m3 products of many rows whose rows are
// 16-byte aligned: LDS tiles filled straight from memory.
#include "linear_tile.hpp"

namespace hyena {

typedef __attribute__((address_space(3))) void lds_ptr;

// 16 bytes (4) per lane from base + off straight into LDS, lane l at dst + 16 l (4 l).
// Written as assembly so that the compiler, which cannot tell the two halves of the LDS
// buffer apart, does not make every LDS read of one half wait for the loads into the
// other; the kernel waits for them itself (dma_sync).  They write no vector registers;
// m0 is the compiler's only where it sets it itself, just before the use.
__device__ __forceinline__ void dma16(const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(dst), "v"(off), "s"(base)
               : "memory");
}
__device__ __forceinline__ void dma4(const void* base, uint32_t off, uint32_t dst) {
  asm volatile("s_mov_b32 m0, %0\n\tglobal_load_lds_dword %1, %2" ::"s"(dst), "v"(off), "s"(base)
               : "memory");
}
// This wave's loads have arrived; then every wave is here.
__device__ __forceinline__ void dma_sync() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// WT x WN waves, each with MT x MN tiles of 16 tokens by 16 columns.
template <int WT, int WN, int MT, int MN, bool GATED, int OUT>
__global__ __launch_bounds__(WT * WN * 64) void linear_dma_kernel(LinearArgs a, int tiles_t, int tiles_n) {
  constexpr int NW = WT * WN;
  constexpr int BT = WT * MT * 16, BN = WN * MN * 16;
  constexpr int CN = GATED ? BN / 2 : BN;
  constexpr int MC = GATED ? MN / 2 : MN;
  constexpr bool WIDE = OUT != OUT_BF16;                 // Frag says why
  constexpr int RX = BT / (NW * 8), RW = BN / (NW * 8);  // loads of a wave, eight rows each
  static_assert(BT % (NW * 8) == 0 && BN % (NW * 8) == 0 && BT % 64 == 0 && BT / 64 <= NW, "whole loads");
  static_assert(RUN % (MC * 16) == 0, "a wave's columns lie in one block of the scales");
  constexpr int XB = BT * RUN, WB = BN * RUN, BUF = XB + WB + BT * 4;   // codes, codes, scales
  __shared__ __attribute__((aligned(16))) uint8_t sh[2 * BUF];
  const uint32_t sh0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr*)(sh)));

  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WN, wn = wave % WN;
  int ti, ni;
  tile_of(tiles_t, tiles_n, ti, ni);
  const int64_t t0 = static_cast<int64_t>(ti) * BT;
  const int n0 = ni * CN;
  const int K = a.K, N = a.N;
  const int blocks = (K + RUN - 1) / RUN;

  // A load of a wave fills eight rows of 128 bytes, lane l place l % 8 of row l / 8;
  // the chunk that belongs there (slot) is the same for all of a lane's loads.
  static_assert(NW % 2 == 0, "a wave's eight rows are all even or all odd ones");
  const int lrow = lane >> 3;
  const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ lrow ^ (wave & 1)) * 16;
  const int64_t rows = a.T - t0;                          // rows past the end repeat the last one
  const uint8_t* const bx = a.x + t0 * a.x_stride;
  const uint8_t* bw[RW];
  uint32_t ox[RX], ow[RW];
#pragma unroll
  for (int i = 0; i < RX; ++i) {
    const int r = (i * NW + wave) * 8 + lrow;
    ox[i] = static_cast<uint32_t>(r < rows ? r : rows - 1) * static_cast<uint32_t>(a.x_stride) + chunk;
  }
#pragma unroll
  for (int i = 0; i < RW; ++i) {
    const int r = (i * NW + wave) * 8;                   // first of the eight
    int n = r;
    bw[i] = a.w0;
    if constexpr (GATED) {
      const int rr = r % (MN * 16);
      n = r / (MN * 16) * (MC * 16) + rr % (MC * 16);
      if (rr >= MC * 16) bw[i] = a.w1;
    }
    bw[i] += static_cast<int64_t>(n0) * K;
    n += lrow;
    ow[i] = static_cast<uint32_t>(n < N - n0 ? n : N - n0 - 1) * static_cast<uint32_t>(K) + chunk;
  }
  const int sr = wave * 64 + lane;                       // scales: the first BT / 64 waves
  const uint32_t os = static_cast<uint32_t>(sr < rows ? sr : rows - 1) * static_cast<uint32_t>(a.xs_row) * 4u;
  const float* const bs = a.x_scale + t0 * a.xs_row;

  auto stage = [&](int kb, int buf) {
    const int k = kb * RUN;
    const uint32_t to = sh0 + buf * BUF + wave * 1024;
    if (wave < BT / 64) dma4(bs + static_cast<int64_t>(kb) * a.xs_run, os, sh0 + buf * BUF + XB + WB + wave * 256);
    if (k + static_cast<int>(chunk) < K) {               // K is a multiple of 16
#pragma unroll
      for (int i = 0; i < RX; ++i) dma16(bx + k, ox[i], to + i * (NW * 1024));
#pragma unroll
      for (int i = 0; i < RW; ++i) dma16(bw[i] + k, ow[i], to + XB + i * (NW * 1024));
    } else {                                             // the last, shorter run: zeros beyond K
      const i32x4 zero = {0, 0, 0, 0};
      i32x4* const z = reinterpret_cast<i32x4*>(sh + buf * BUF + wave * 1024) + lane;
#pragma unroll
      for (int i = 0; i < RX + RW; ++i) z[i * NW * 64] = zero;
    }
  };

  const int fr = lane & 15, fc = lane >> 4;
  const int swz = (fr & 7) ^ (fr >> 3);
  // byte places of the lane's two chunks in a tile of 16 rows
  const int f0 = fr * RUN + ((2 * fc) ^ swz) * 16, f1 = fr * RUN + ((2 * fc + 1) ^ swz) * 16;
  const int ncol = n0 + wn * (MC * 16);
  const int64_t sbase = static_cast<int64_t>((ncol < N ? ncol : N - 1) / RUN) * blocks;
  typedef const __attribute__((address_space(4))) float* cptr;
  const cptr ps0 = (cptr)(a.s0 + sbase);
  const cptr ps1 = (cptr)(GATED ? a.s1 + sbase : a.s0);

  f32x4 acc[MN][MT];
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (blocks > 0) stage(0, 0);
  dma_sync();
  for (int kb = 0; kb < blocks; ++kb) {
    if (kb + 1 < blocks) stage(kb + 1, (kb + 1) & 1);
    const uint8_t* const b = sh + (kb & 1) * BUF;
    const uint8_t* const xt = b + wt * MT * 2048;
    const uint8_t* const wp = b + XB + wn * MN * 2048;
    const float* const st = reinterpret_cast<const float*>(b + XB + WB) + wt * MT * 16 + fr;
    const float w0 = ps0[kb], w1 = GATED ? ps1[kb] : 0.0f;
    Frag<WIDE> fx[MT];
    float sx[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      fx[j].set(pair16(*reinterpret_cast<const i32x4*>(xt + j * 2048 + f0),
                       *reinterpret_cast<const i32x4*>(xt + j * 2048 + f1)));
      sx[j] = st[j * 16];
    }
#pragma unroll
    for (int i = 0; i < MN; ++i) {
      Frag<WIDE> fw;
      fw.set(pair16(*reinterpret_cast<const i32x4*>(wp + i * 2048 + f0),
                    *reinterpret_cast<const i32x4*>(wp + i * 2048 + f1)));
      const float sw = GATED && i >= MC ? w1 : w0;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const f32x4 p = mfma_run(fw, fx[j]);
        const float s = sx[j] * sw;
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], s, acc[i][j][e]);
      }
    }
    dma_sync();
  }
  tile_epilogue<WT, WN, MT, MN, GATED, OUT>(a, acc, t0, ncol, wt, wn, lane, sh);
}

template <int WT, int WN, int MT, int MN, bool GATED, int OUT>
static void dma_go(const LinearArgs& a) {
  constexpr int BT = WT * MT * 16, CN = WN * MN * 16 / (GATED ? 2 : 1);
  const int64_t tt = (a.T + BT - 1) / BT, tn = (a.N + CN - 1) / CN;
  linear_dma_kernel<WT, WN, MT, MN, GATED, OUT><<<static_cast<unsigned>(tt * tn), WT * WN * 64, 0, a.stream>>>(
      a, static_cast<int>(tt), static_cast<int>(tn));
}

// whole 16-byte chunks, and 32-bit offsets within a tile
bool linear_dma_takes(const LinearArgs& a) {
  auto whole = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return a.K % 16 == 0 && a.x_stride % 16 == 0 && whole(a.x) && whole(a.w0) && whole(a.w1) &&
         a.x_stride < (1 << 23) && a.xs_row < (1 << 21);
}

hipError_t launch_linear_dma(const LinearArgs& a) {
  if (a.w1) {
    if (a.out == OUT_BF16) dma_go<4, 2, 4, 8, true, OUT_BF16>(a);
    else if (a.out == OUT_F32) dma_go<4, 2, 4, 4, true, OUT_F32>(a);
    else dma_go<2, 4, 4, 4, true, OUT_FP8>(a);
  } else {
    if (a.out == OUT_BF16) dma_go<4, 2, 4, 8, false, OUT_BF16>(a);
    else dma_go<4, 2, 4, 4, false, OUT_F32>(a);
  }
  return hipGetLastError();
}

}  // namespace hyena
