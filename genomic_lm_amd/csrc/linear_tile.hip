// linear_tile.hip -- block-scaled e4m3 products of many rows, on LDS tiles.
#include "linear_common.hpp"

namespace hyena {

// The workgroup's LDS operations are complete and every wave is here; loads
// into registers stay in flight.
__device__ __forceinline__ void tile_sync() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// LDS place of 16-byte chunk c of row r: any 8 and any 16 consecutive rows have
// their chunks c in different banks.
__device__ __forceinline__ int slot(int r, int c) {
  return r * 8 + (c ^ (r & 7) ^ ((r >> 3) & 1));
}

// WT x WN waves, each with MT x MN tiles of 16 tokens by 16 columns.
template <int WT, int WN, int MT, int MN, bool GATED, int OUT>
__global__ __launch_bounds__(WT * WN * 64) void linear_tile_kernel(LinearArgs a, int tiles_t, int tiles_n) {
  constexpr int NT = WT * WN * 64;
  constexpr int BT = WT * MT * 16, BN = WN * MN * 16;    // rows of the two staged tiles
  constexpr int CN = GATED ? BN / 2 : BN;                // columns of the output tile
  constexpr int MC = GATED ? MN / 2 : MN;
  constexpr bool WIDE = OUT != OUT_BF16;                 // Frag says why
  constexpr int STEP = NT / 8;
  constexpr int RX = BT / STEP, RW = BN / STEP;
  static_assert(BT % STEP == 0 && BN % STEP == 0, "whole rows per pass");
  static_assert(RUN % (MC * 16) == 0, "a wave's columns lie in one block of the scales");
  __shared__ __attribute__((aligned(16))) uint8_t sh[2 * (BT + BN) * RUN];
  constexpr int BUF = (BT + BN) * 8;                     // 16-byte slots
  i32x4* lds = reinterpret_cast<i32x4*>(sh);

  const int tid = static_cast<int>(threadIdx.x);
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wt = wave / WN, wn = wave % WN;

  // workgroups of one XCD (every eighth) take neighbouring tiles, in groups of
  // up to 8 tile rows, so that they share operands in its L2
  const int64_t total = static_cast<int64_t>(tiles_t) * tiles_n;
  int64_t id = blockIdx.x;
  {
    const int64_t per = total / 8, rest = total % 8, xcd = id % 8, k = id / 8;
    id = xcd * per + (xcd < rest ? xcd : rest) + k;
  }
  const int64_t band = id / (8LL * tiles_n);
  const int bt0 = static_cast<int>(band) * 8;
  const int high = tiles_t - bt0 < 8 ? tiles_t - bt0 : 8;
  const int in = static_cast<int>(id - band * 8LL * tiles_n);
  const int64_t t0 = static_cast<int64_t>(bt0 + in % high) * BT;
  const int n0 = in / high * CN;

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

  fetch(0);
  put(0);
  if (blocks > 1) fetch(1);
  tile_sync();
  const int fr = lane & 15, fc = (lane >> 4) * 2;
  for (int kb = 0; kb < blocks; ++kb) {
    const i32x4* bx = lds + (kb & 1) * BUF;
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
    if (kb + 1 < blocks) put((kb + 1) & 1);
    if (kb + 2 < blocks) fetch(kb + 2);
    tile_sync();
  }

  // epilogue: lane holds columns cn .. cn + 3 of its tokens
  const int cg = 4 * (lane >> 4);
  if constexpr (OUT == OUT_FP8) {
    static_assert(GATED, "codes come from the gated product");
    float* top = reinterpret_cast<float*>(sh);          // [WN][BT]
    constexpr int GW = RUN / (MC * 16);                 // waves that share a run of columns
    float h[MC][MT][4];
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = ncol + i * 16 + cg + e;
          h[i][j][e] = n < N ? gate(acc[i][j][e], acc[i + MC][j][e], a.act) : 0.0f;
          const uint32_t b = mag_bits(h[i][j][e]);
          m = b > m ? b : m;
        }
      uint32_t o = __float_as_uint(xor16(__uint_as_float(m), lane));
      m = o > m ? o : m;
      o = __float_as_uint(xor32(__uint_as_float(m), lane >> 5));
      m = o > m ? o : m;
      if (lane < 16) top[wn * BT + (wt * MT + j) * 16 + lane] = __uint_as_float(m);
    }
    tile_sync();
    const int runs = (N + RUN - 1) / RUN;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int tr = (wt * MT + j) * 16 + (lane & 15);
      const int64_t t = t0 + tr;
      uint32_t m = 0;
#pragma unroll
      for (int g = 0; g < GW; ++g) {
        const uint32_t o = __float_as_uint(top[(wn / GW * GW + g) * BT + tr]);
        m = o > m ? o : m;
      }
      const float scale = run_scale(m);
      if (t >= a.T) continue;
      if (wn % GW == 0 && lane < 16 && ncol < N) a.q_scale[t * runs + ncol / RUN] = scale;
      uint8_t* row = static_cast<uint8_t*>(a.y) + t * a.y_stride;
#pragma unroll
      for (int i = 0; i < MC; ++i) {
        uint32_t w[1];
        to_codes<4>(h[i][j], scale, w);
        const int n = ncol + i * 16 + cg;
        if (n + 4 <= N) __builtin_memcpy(row + n, w, 4);
        else
          for (int e = 0; e < 4; ++e)
            if (n + e < N) row[n + e] = static_cast<uint8_t>(w[0] >> (8 * e));
      }
    }
  } else {
    using O = typename std::conditional<OUT == OUT_BF16, bf16_t, float>::type;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      const int64_t t = t0 + (wt * MT + j) * 16 + (lane & 15);
      if (t >= a.T) continue;
      O* row = static_cast<O*>(a.y) + t * a.y_stride;
#pragma unroll
      for (int i = 0; i < MC; ++i) {
        const int n = ncol + i * 16 + cg;
        float o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (GATED) o[e] = gate(acc[i][j][e], acc[i + MC][j][e], a.act);
          else o[e] = acc[i][j][e] + (a.bias && n + e < N ? a.bias[n + e] : 0.0f);
        }
        if (n + 4 <= N) {
          if constexpr (OUT == OUT_BF16) {
            const uint32_t w[2] = {
                static_cast<uint32_t>(f32_to_bf16(o[0])) | (static_cast<uint32_t>(f32_to_bf16(o[1])) << 16),
                static_cast<uint32_t>(f32_to_bf16(o[2])) | (static_cast<uint32_t>(f32_to_bf16(o[3])) << 16)};
            __builtin_memcpy(row + n, w, 8);
          } else {
            __builtin_memcpy(row + n, o, 16);
          }
        } else {
          for (int e = 0; e < 4; ++e)
            if (n + e < N) Io<O>::st(row, n + e, o[e]);
        }
      }
    }
  }
}

template <int WT, int WN, int MT, int MN, bool GATED>
static void tile_go(const LinearArgs& a) {
  constexpr int BT = WT * MT * 16, CN = WN * MN * 16 / (GATED ? 2 : 1);
  const int64_t tt = (a.T + BT - 1) / BT, tn = (a.N + CN - 1) / CN;
  const unsigned grid = static_cast<unsigned>(tt * tn);
  auto go = [&](auto kernel) {
    kernel<<<grid, WT * WN * 64, 0, a.stream>>>(a, static_cast<int>(tt), static_cast<int>(tn));
  };
  if (a.out == OUT_F32) go(linear_tile_kernel<WT, WN, MT, MN, GATED, OUT_F32>);
  else if (a.out == OUT_BF16) go(linear_tile_kernel<WT, WN, MT, MN, GATED, OUT_BF16>);
  else if constexpr (GATED && CN % RUN == 0) go(linear_tile_kernel<WT, WN, MT, MN, GATED, OUT_FP8>);
}

hipError_t launch_linear_tile(const LinearArgs& a) {
  if (a.w1) tile_go<2, 4, 4, 4, true>(a);
  else tile_go<2, 2, 4, 4, false>(a);
  return hipGetLastError();
}

}  // namespace hyena
