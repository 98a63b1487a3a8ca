// linear_dma.hip -- block-scaled e4m3 products of many rows whose rows are
// 16-byte aligned: LDS tiles filled straight from memory.
//
// Bound by the matrix cores and the scales' FMAs beside them, at 1.9 to 2.05 GHz: 8192 x 4096 to 12288,
// bf16 outputs, 368 to 388 us by card, 2.1 to 2.2 PFLOP/s, fp32 ones, on the bf16 instructions, 690, 1.2;
// gated to 11008 with e4m3 outputs 1197 to 1235, 1.20 to 1.23 PFLOP/s; the matrix pipes are busy half of the
// cycles.  A load to LDS moves 1 KB in 16 cycles and needs no registers, which hold the sums (256 x
// 256 fp32 in eight waves); a tile staged through registers spilled 210 of them.
#include "linear_tile.hpp"

namespace hyena {

// All but N of this wave's loads have arrived, and its LDS reads; then every wave is here.
template <int N>
__device__ __forceinline__ void dma_sync() {
  static_assert(N < 64, "vmcnt range");
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// What a wave of WT x WN, each with MT x MN tiles of 16 x 16, loads of each run of K: codes of
// the tokens and of the weights (a gated wave's first MN / 2 tiles from w0, the others from w1),
// the tokens' scales, those of w0 and of w1, in this order in LDS.
template <int WT, int WN, int MT, int MN, bool GATED>
struct Loads {
  static constexpr int NW = WT * WN;
  static constexpr int BT = WT * MT * 16, BN = WN * MN * 16;
  static constexpr int CN = GATED ? BN / 2 : BN, MC = GATED ? MN / 2 : MN;   // columns of the output
  static constexpr int RX = BT / (NW * 8), RW = BN / (NW * 8);               // loads of eight rows each
  static constexpr int XW = BT / 64;                                         // waves for the tokens' scales
  static constexpr int LOADS = RX + RW + 1;                                  // of a wave and run
  static_assert(BT % (NW * 8) == 0 && BN % (NW * 8) == 0 && BT % 64 == 0, "whole loads");
  static_assert(NW > XW + (GATED ? 1 : 0), "waves for all scales");
  static_assert(RUN % (MC * 16) == 0, "a wave's columns lie in one block of the scales");
  static_assert(NW % 2 == 0, "a wave's eight rows are all even or all odd ones");
  static constexpr int XB = BT * RUN, SB = XB + BN * RUN, BUF = SB + XW * 256 + 512;

  const uint8_t* bx;
  const uint8_t* bw[RW];
  const float* bs;
  uint32_t ox[RX], ow[RW], os, ds;
  int step, wave;
  int chunk;        // a load's lane l fills place l % 8 of row l / 8: the chunk that belongs there (slot)

  __device__ __forceinline__ Loads(const LinearArgs& a, int64_t t0, int n0, int wave, int lane) : wave(wave) {
    const int lrow = lane >> 3;
    chunk = ((lane & 7) ^ lrow ^ (wave & 1)) * 16;
    const int64_t rows = a.T - t0;                       // rows past the end repeat the last one
    bx = a.x + t0 * a.x_stride;
#pragma unroll
    for (int i = 0; i < RX; ++i) {
      const int r = (i * NW + wave) * 8 + lrow;
      ox[i] = static_cast<uint32_t>(r < rows ? r : rows - 1) * static_cast<uint32_t>(a.x_stride) + chunk;
      asm volatile("" : "+v"(ox[i]));                    // 32 bits, not the 64 of the product
    }
#pragma unroll
    for (int i = 0; i < RW; ++i) {
      const int r = (i * NW + wave) * 8;                 // first of the eight
      int n = r;
      bw[i] = a.w0;
      if constexpr (GATED) {
        const int rr = r % (MN * 16);
        n = r / (MN * 16) * (MC * 16) + rr % (MC * 16);
        if (rr >= MC * 16) bw[i] = a.w1;
      }
      bw[i] += static_cast<int64_t>(n0) * a.K;
      n += lrow;
      ow[i] = static_cast<uint32_t>(n < a.N - n0 ? n : a.N - n0 - 1) * static_cast<uint32_t>(a.K) + chunk;
      asm volatile("" : "+v"(ow[i]));
    }
    // Scales come through LDS too: a scalar load in the loop would be waited for with every
    // LDS read (both count in lgkmcnt, scalar ones out of order).
    if (wave < XW) {
      const int r = wave * 64 + lane;
      bs = a.x_scale + t0 * a.xs_row;
      os = static_cast<uint32_t>(r < rows ? r : rows - 1) * static_cast<uint32_t>(a.xs_row) * 4u;
      step = a.xs_run;
      ds = SB + wave * 256;
    } else {                                             // of the block of each wave column
      const int which = GATED ? (wave - XW) & 1 : 0;
      const int c = n0 + lane % WN * (MC * 16);
      bs = which ? a.s1 : a.s0;
      os = static_cast<uint32_t>((c < a.N ? c : a.N - 1) / RUN) *
           static_cast<uint32_t>((a.K + RUN - 1) / RUN) * 4u;
      step = 1;
      ds = SB + (XW + which) * 256;
    }
  }
  __device__ __forceinline__ void scales(int kb, uint32_t to) const {
    dma4(bs + static_cast<int64_t>(kb) * step, os, to + ds);
  }
  __device__ __forceinline__ void tokens(int kb, uint32_t to) const {
#pragma unroll
    for (int i = 0; i < RX; ++i) dma16(bx + kb * RUN, ox[i], to + (i * NW + wave) * 1024);
  }
  template <int FIRST, int EVERY>
  __device__ __forceinline__ void weights(int kb, uint32_t to) const {
#pragma unroll
    for (int i = FIRST; i < RW; i += EVERY) dma16(bw[i] + kb * RUN, ow[i], to + XB + (i * NW + wave) * 1024);
  }
  // the lane's chunks of a run that K does not reach (it is a multiple of 16): zeros
  __device__ __forceinline__ void clear(uint8_t* buf, int lane) const {
    const i32x4 zero = {0, 0, 0, 0};
    i32x4* const z = reinterpret_cast<i32x4*>(buf + wave * 1024) + lane;
#pragma unroll
    for (int i = 0; i < RX + RW; ++i) z[i * NW * 64] = zero;
  }
};

// KG groups of WT x WN waves share a tile and take turns at the runs of K.
template <int WT, int WN, int MT, int MN, int KG, bool GATED, int OUT>
__global__ __launch_bounds__(WT * WN * KG * 64) void linear_dma_kernel(LinearArgs a, int tiles_t, int tiles_n) {
  using L = Loads<WT, WN, MT, MN, GATED>;
  constexpr int NW = L::NW, MC = L::MC, BUF = L::BUF;
  constexpr bool WIDE = OUT != OUT_BF16;                 // Frag says why
  constexpr int JOIN = (KG - 1) * NW * MN * MT * 1024;   // the other groups' sums
  constexpr int TOPS = OUT == OUT_FP8 ? WN * L::BT * 4 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t sh[2 * KG * BUF > JOIN + TOPS ? 2 * KG * BUF : JOIN + TOPS];

  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave_of_all = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int kg = wave_of_all / NW, wave = wave_of_all % NW;
  const int wt = wave / WN, wn = wave % WN;
  uint8_t* const mine = sh + kg * 2 * BUF;
  const uint32_t mine0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr*)(mine)));
  int ti, ni;
  tile_of(tiles_t, tiles_n, ti, ni);
  const int64_t t0 = static_cast<int64_t>(ti) * L::BT;
  const int n0 = ni * L::CN;
  const int K = a.K;
  const int blocks = (K + RUN - 1) / RUN;
  const L from(a, t0, n0, wave, lane);
  auto stage = [&](int kb, int buf) __attribute__((always_inline)) {
    const uint32_t to = mine0 + buf * BUF;
    from.scales(kb, to);
    if (kb * RUN + from.chunk < K) {
      from.tokens(kb, to);
      from.template weights<0, 1>(kb, to);
    } else {
      from.clear(mine + buf * BUF, lane);
    }
  };

  f32x4 acc[MN][MT];
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  if (kg < blocks) stage(kg, 0);
  dma_sync<0>();
  int buf = 0;
  for (int k0 = 0; k0 < blocks; k0 += KG) {
    const int kb = k0 + kg;
    if (kb + KG < blocks) stage(kb + KG, buf ^ 1);
    if (KG == 1 || kb < blocks) {
      const uint8_t* const b = mine + buf * BUF;
      const float* const st = reinterpret_cast<const float*>(b + L::SB) + wt * MT * 16 + (lane & 15);
      const float* const sw = reinterpret_cast<const float*>(b + L::SB + L::XW * 256) + wn;
      const float w0 = sw[0], w1 = GATED ? sw[64] : 0.0f;
      Frag<WIDE> fx[MT];
      float sx[MT];
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        fx[j].set(tile_codes(b + (wt * MT + j) * 2048, lane));
        sx[j] = st[j * 16];
      }
#pragma unroll
      for (int i = 0; i < MN; ++i) {
        Frag<WIDE> fw;
        fw.set(tile_codes(b + L::XB + (wn * MN + i) * 2048, lane));
        const float s = GATED && i >= MC ? w1 : w0;
        // keeps the compiler from widening several operands ahead, for which no registers are left
        if constexpr (WIDE) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const f32x4 p = mfma_run(fw, fx[j]);
          const float f = sx[j] * s;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(p[e], f, acc[i][j][e]);
        }
      }
    }
    buf ^= 1;
    dma_sync<0>();
  }
  if constexpr (KG > 1) join_groups<KG, NW, MT, MN>(acc, sh, kg, wave, lane);
  if (kg > 0) return;
  tile_epilogue<WT, WN, MT, MN, GATED, OUT>(a, acc, t0, n0 + wn * (MC * 16), wt, wn, lane, sh + JOIN);
}

// The largest products with bf16 outputs: 256 x 256 tiles, eight waves of 64 x 128 in two halves
// that take turns, one reading its operands of half a run while the other multiplies (the
// two waves of a SIMD belong to different halves).  Time goes by in slots that end with a barrier;
// of run r the first half reads in slots 4r and 4r + 2 and multiplies in 4r + 1 and 4r + 3, the
// second does the same a slot later.  A read slot also asks for what it may overwrite: in its
// first the other columns of the next run, in its second the tokens and first columns of the run
// after; so a run's worth of loads (FLY) stays on its way, each for about six slots.
// A shorter last run goes first, where its zeros can be written in peace.
template <bool GATED>
__global__ __launch_bounds__(512) void linear_turns_kernel(LinearArgs a, int tiles_t, int tiles_n) {
  constexpr int WT = 4, WN = 2, MT = 4, MN = 8;
  using L = Loads<WT, WN, MT, MN, GATED>;
  constexpr int BUF = L::BUF, FLY = L::LOADS;
  static_assert(L::NW == 8 && L::RW == 4, "the even loads are the waves' first halves");
  __shared__ __attribute__((aligned(16))) uint8_t sh[2 * BUF];
  const uint32_t sh0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_ptr*)(sh)));
  const int lane = static_cast<int>(threadIdx.x) & 63;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
  const int wt = wave / WN, wn = wave % WN;
  const bool second = wave >= 4;
  int ti, ni;
  tile_of(tiles_t, tiles_n, ti, ni);
  const int64_t t0 = static_cast<int64_t>(ti) * L::BT;
  const int n0 = ni * L::CN;
  const int full = a.K / RUN, tail = a.K % RUN ? 1 : 0, blocks = full + tail;   // full >= 1
  const L from(a, t0, n0, wave, lane);
  // Step `it` takes run it - tail, the first of a tail run `full`.  Past the end the last full run
  // is loaded again, so that every step has as many loads on their way.
  auto run_of = [&](int it) {
    const int kb = it - tail < full ? it - tail : full - 1;
    return kb < 0 ? full : kb;
  };
  auto ask0 = [&](int it) __attribute__((always_inline)) {
    const int kb = run_of(it);
    const uint32_t to = sh0 + (it & 1) * BUF;
    from.scales(kb, to);
    from.tokens(kb, to);
    from.template weights<0, 2>(kb, to);
  };
  auto ask1 = [&](int it) __attribute__((always_inline)) {
    from.template weights<1, 2>(run_of(it), sh0 + (it & 1) * BUF);
  };
  // nothing but the loads and reads moves from one slot to another
  auto slot_end = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_barrier" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  auto read_end = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    dma_sync<FLY>();
    __builtin_amdgcn_sched_barrier(0);
  };

  f32x4 acc[MN][MT];
#pragma unroll
  for (int i = 0; i < MN; ++i)
#pragma unroll
    for (int j = 0; j < MT; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  Frag<false> fx[MT], fw[MN / 2];
  float sx[MT];
  // products of half H's columns; each is scaled and added two products later, when it is there
  auto multiply = [&](auto half, float sw) __attribute__((always_inline)) {
    constexpr int H = decltype(half)::value, Q = MN / 2 * MT;
    float s[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) s[j] = sx[j] * sw;
    f32x4 p[3];
    auto add = [&](int q) __attribute__((always_inline)) {
      f32x4& c = acc[H * MN / 2 + q / MT][q % MT];
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = fmaf(p[q % 3][e], s[q % MT], c[e]);
    };
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      p[q % 3] = mfma_run(fw[q / MT], fx[q % MT]);
      __builtin_amdgcn_sched_barrier(0);
      if (q > 1) add(q - 2);
      __builtin_amdgcn_sched_barrier(0);
    }
    add(Q - 2);
    add(Q - 1);
  };

  {
    const int first = run_of(0);
    const bool on = first * RUN + from.chunk < a.K;
    if (on) {
      ask0(0);
      ask1(0);
    } else {
      from.scales(first, sh0);
      from.clear(sh, lane);
    }
    ask0(1);
  }
  // (the scales of lanes that are not `on` were asked for in a branch of their own, so fewer
  // loads than FLY may follow the first run's: all of them are waited for)
  dma_sync<0>();
  if (second) slot_end();
  for (int it = 0; it < blocks; ++it) {
    const uint8_t* const b = sh + (it & 1) * BUF;
    const uint8_t* const xt = b + wt * MT * 2048;
    const uint8_t* const wp = b + L::XB + wn * MN * 2048;
    const float* const st = reinterpret_cast<const float*>(b + L::SB) + wt * MT * 16 + (lane & 15);
    const float* const sw = reinterpret_cast<const float*>(b + L::SB + L::XW * 256) + wn;
    const float w0 = sw[0], w1 = GATED ? sw[64] : w0;
    ask1(it + 1);
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      fx[j].set(tile_codes(xt + j * 2048, lane));
      sx[j] = st[j * 16];
    }
#pragma unroll
    for (int i = 0; i < MN / 2; ++i) fw[i].set(tile_codes(wp + i * 2048, lane));
    read_end();
    multiply(std::integral_constant<int, 0>{}, w0);
    slot_end();
    ask0(it + 2);
#pragma unroll
    for (int i = 0; i < MN / 2; ++i) fw[i].set(tile_codes(wp + (MN / 2 + i) * 2048, lane));
    read_end();
    multiply(std::integral_constant<int, 1>{}, w1);
    slot_end();
  }
  if (!second) slot_end();
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // no load outlives its workgroup's LDS
  tile_epilogue<WT, WN, MT, MN, GATED, OUT_BF16>(a, acc, t0, n0 + wn * (L::MC * 16), wt, wn, lane, sh);
}

template <int BT, int CN>
static int64_t tiles(const LinearArgs& a) {
  return (a.T + BT - 1) / BT * ((a.N + CN - 1) / CN);
}

template <int WT, int WN, int MT, int MN, int KG, bool GATED, int OUT>
static void dma_go(const LinearArgs& a) {
  constexpr int BT = WT * MT * 16, CN = WN * MN * 16 / (GATED ? 2 : 1);
  linear_dma_kernel<WT, WN, MT, MN, KG, GATED, OUT>
      <<<static_cast<unsigned>(tiles<BT, CN>(a)), WT * WN * KG * 64, 0, a.stream>>>(
          a, static_cast<int>((a.T + BT - 1) / BT), static_cast<int>((a.N + CN - 1) / CN));
}

// whole 16-byte chunks, and 32-bit offsets within a tile
bool linear_dma_takes(const LinearArgs& a) {
  auto whole = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return a.K % 16 == 0 && a.x_stride % 16 == 0 && whole(a.x) && whole(a.w0) && whole(a.w1) &&
         a.x_stride < (1 << 23) && a.xs_row < (1 << 21);
}

// Tiles by the rounds of workgroups that they make on 256 CUs: one of 256 x 256 to a CU, two of 128 x
// 128, whose round takes 0.7 to 0.8 of the time of one of the former.  Where there is less than a
// round, two or four groups of waves share the K of a tile.  Measured (us, bf16 outputs, the tile
// that is taken, then the next): 8192 x 4096 to 12288 256 x 256 368, 128 x 128 471; 512 to 12288 (96 tiles
// of 256 x 256, 384 of 128 x 128) 128 x 128 38, 52; 512 to 16384 (128, 512) 41, 54; 512 to 4096 (128 of
// 128 x 128) by two groups 23, by one 33.  Up to 100 tiles that whole rounds leave go into a launch
// of smaller ones: 4096 to 4352 (272 tiles) 74, in one launch 108; 1500 to 12288 (288) 84, 108;
// gated 1000 to 10928 (344) 100, 114; but 3000 x 2048 to 8192 (384) 67, 66.
template <bool GATED, int OUT>
static void dma_pick(const LinearArgs& a) {
  constexpr int CN = GATED ? 128 : 256;                  // columns of a tile of 256 rows
  const int64_t n256 = tiles<256, CN>(a), n128 = tiles<128, CN / 2>(a);
  const int64_t tt = (a.T + 255) / 256, whole = n256 / 256 * 256 / tt, rest = n256 - whole * tt;
  if constexpr (OUT == OUT_FP8) {
    dma_go<4, 2, 4, 8, 1, GATED, OUT>(a);
  } else if (whole > 0 && rest > 0 && rest <= 100) {
    // the columns that would be little of a last round, in a launch of smaller tiles
    const int at = static_cast<int>(whole) * CN;
    LinearArgs b = a, c = a;
    b.N = at;
    dma_pick<GATED, OUT>(b);
    const int64_t block = static_cast<int64_t>(at / RUN) * ((a.K + RUN - 1) / RUN);
    c.N = a.N - at;
    c.w0 += static_cast<int64_t>(at) * a.K;
    c.s0 += block;
    if (GATED) {
      c.w1 += static_cast<int64_t>(at) * a.K;
      c.s1 += block;
    }
    if (a.bias) c.bias += at;
    c.y = static_cast<uint8_t*>(a.y) + at * (OUT == OUT_BF16 ? 2 : 4);
    dma_pick<GATED, OUT>(c);
  } else if (n128 > 256 && 100 * ((n256 + 255) / 256) <= 68 * ((n128 + 511) / 512) &&
             (OUT != OUT_BF16 || a.K >= RUN)) {
    if constexpr (OUT == OUT_BF16)
      linear_turns_kernel<GATED><<<static_cast<unsigned>(n256), 512, 0, a.stream>>>(
          a, static_cast<int>((a.T + 255) / 256), static_cast<int>(n256 / ((a.T + 255) / 256)));
    else dma_go<4, 2, 4, 8, 1, GATED, OUT>(a);
  } else if (n128 > 256) {
    dma_go<2, 2, 4, 4, 1, GATED, OUT>(a);
  } else if (n128 >= 90) {
    dma_go<2, 2, 4, 4, 2, GATED, OUT>(a);
  } else if constexpr (GATED) {
    dma_go<2, 2, 2, 4, 2, GATED, OUT>(a);
  } else {
    dma_go<2, 2, 2, 2, 4, GATED, OUT>(a);
  }
}

hipError_t launch_linear_dma(const LinearArgs& a) {
  if (a.out == OUT_FP8 && !a.gated) return hipErrorInvalidValue;
  if (a.gated) {
    if (a.out == OUT_BF16) dma_pick<true, OUT_BF16>(a);
    else if (a.out == OUT_F32) dma_pick<true, OUT_F32>(a);
    else dma_pick<true, OUT_FP8>(a);
  } else {
    if (a.out == OUT_BF16) dma_pick<false, OUT_BF16>(a);
    else dma_pick<false, OUT_F32>(a);
  }
  return hipGetLastError();
}

}  // namespace hyena
