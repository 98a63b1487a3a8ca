// linear_tile.hpp -- what the kernels on LDS tiles share (linear_tile.hip,
// linear_dma.hip): the order of the tiles, the places in LDS and the epilogue.
#pragma once

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

// Tile (row, column) of this workgroup.  Workgroups of one XCD (every eighth)
// take neighbouring tiles, in groups of up to 8 tile rows, so that they share
// operands in its L2.
__device__ __forceinline__ void tile_of(int tiles_t, int tiles_n, int& ti, int& ni) {
  const int64_t total = static_cast<int64_t>(tiles_t) * tiles_n;
  const int64_t per = total / 8, rest = total % 8, xcd = blockIdx.x % 8, k = blockIdx.x / 8;
  const int64_t id = xcd * per + (xcd < rest ? xcd : rest) + k;
  const int64_t band = id / (8LL * tiles_n);
  const int bt0 = static_cast<int>(band) * 8;
  const int high = tiles_t - bt0 < 8 ? tiles_t - bt0 : 8;
  const int in = static_cast<int>(id - band * 8LL * tiles_n);
  ti = bt0 + in % high;
  ni = in / high;
}

// The tile's sums to the output: a wave's lane holds columns 4 (l / 16) .. + 3 of
// token l % 16 in each of its MT x MN tiles, the gate's in the first half of
// the MN and the other weight's in the second.  sh: LDS that nobody reads any more.
template <int WT, int WN, int MT, int MN, bool GATED, int OUT>
__device__ __forceinline__ void tile_epilogue(const LinearArgs& a, f32x4 (&acc)[MN][MT], int64_t t0, int ncol,
                                              int wt, int wn, int lane, uint8_t* sh) {
  constexpr int BT = WT * MT * 16;
  constexpr int MC = GATED ? MN / 2 : MN;
  const int N = a.N;
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

}  // namespace hyena
