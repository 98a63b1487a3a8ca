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

// Exchanges the odd 16-lane rows of a with the even ones of b, and the upper half of
// a with the lower half of b.
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// The other groups' sums to group 0, in their order: acc of group 0 is the tile's afterwards.  The
// groups are done with the LDS at sh.
template <int KG, int NW, int MT, int MN>
__device__ __forceinline__ void join_groups(f32x4 (&acc)[MN][MT], uint8_t* sh, int kg, int wave, int lane) {
  f32x4* const join = reinterpret_cast<f32x4*>(sh) + wave * (MN * MT * 64) + lane;
  if (kg > 0) {
#pragma unroll
    for (int i = 0; i < MN; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) join[((kg - 1) * NW * MN * MT + i * MT + j) * 64] = acc[i][j];
  }
  tile_sync();
  if (kg > 0) return;
#pragma unroll
  for (int g = 0; g < KG - 1; ++g)
#pragma unroll
    for (int i = 0; i < MN; ++i)
#pragma unroll
      for (int j = 0; j < MT; ++j) acc[i][j] += join[(g * NW * MN * MT + i * MT + j) * 64];
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
  // One decision for all elements where there is one to make: the code of a tile's end is read once
  // by each CU, and from memory, as the products go through the L2s (4096 x 128 to 4096,
  // bf16: 27 us with branches at every element, 14 so).
  if constexpr (GATED)
    with_act(a.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = gate<decltype(act)::value>(acc[i][j][e], acc[i + MC][j][e]);
    });
  if constexpr (OUT == OUT_FP8) {
    static_assert(GATED && MC % 4 == 0, "codes come from the gated product");
    float* top = reinterpret_cast<float*>(sh);          // [WN][BT]
    constexpr int GW = RUN / (MC * 16);                 // waves that share a run of columns
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = ncol + i * 16 + cg + e;
          acc[i][j][e] = n < N ? acc[i][j][e] : 0.0f;
          const uint32_t b = mag_bits(acc[i][j][e]);
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
      if (wn % GW == 0 && lane < 16 && ncol < N && t < a.T) a.q_scale[t * runs + ncol / RUN] = scale;
      uint8_t* row = static_cast<uint8_t*>(a.y) + t * a.y_stride;
      {
#pragma unroll
        for (int i = 0; i < MC; i += 4) {
          // lane group g holds words g of four tiles; afterwards the four words of tile g
          uint32_t w[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t c[1];
            const float h[4] = {acc[i + q][j][0], acc[i + q][j][1], acc[i + q][j][2], acc[i + q][j][3]};
            to_codes<4>(h, scale, c);
            w[q] = c[0];
          }
          swap16(w[0], w[1]);
          swap16(w[2], w[3]);
          swap32(w[0], w[2]);
          swap32(w[1], w[3]);
          const int n = ncol + (i + (lane >> 4)) * 16;
          if (t >= a.T || n >= N) continue;
          if (n + 16 <= N) __builtin_memcpy(row + n, w, 16);
          else
            for (int e = 0; n + e < N; ++e) row[n + e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
        }
      }
    }
  } else {
    using O = typename std::conditional<OUT == OUT_BF16, bf16_t, float>::type;
    static_assert(MC % 2 == 0 || OUT == OUT_F32, "tiles in pairs");
    if (!GATED && a.bias) {
#pragma unroll
      for (int i = 0; i < MC; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int n = ncol + i * 16 + cg + e;
          const float b = a.bias[n < N ? n : N - 1];
#pragma unroll
          for (int j = 0; j < MT; ++j) acc[i][j][e] += b;
        }
    }
    const int64_t t = t0 + wt * MT * 16 + (lane & 15);
    O* const row = static_cast<O*>(a.y) + t * a.y_stride;
    const int64_t step = 16 * a.y_stride;
    auto store = [&](auto inside) __attribute__((always_inline)) {
      constexpr bool ALL = decltype(inside)::value;     // the wave's rows and columns all exist
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        const bool row_there = ALL || t + j * 16 < a.T;
        if constexpr (OUT == OUT_BF16) {
          // 16-byte stores: even lane groups g take columns 4g .. 4g + 7 of the first
          // tile, odd ones 4(g - 1) .. of the second
          const int g = lane >> 4, n0 = ncol + (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
          for (int i = 0; i < MC; i += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                w[q][e] = static_cast<uint32_t>(f32_to_bf16(acc[i + q][j][2 * e])) |
                          (static_cast<uint32_t>(f32_to_bf16(acc[i + q][j][2 * e + 1])) << 16);
            swap16(w[0][0], w[1][0]);
            swap16(w[0][1], w[1][1]);
            const uint32_t v[4] = {w[0][0], w[0][1], w[1][0], w[1][1]};
            const int n = n0 + i * 16;
            bf16_t* const to = row + j * step + n;
            if (!row_there) continue;
            if (ALL || n + 8 <= N) __builtin_memcpy(to, v, 16);
            else
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (n + e < N) to[e] = static_cast<bf16_t>(v[e >> 1] >> (16 * (e & 1)));
          }
        } else {
#pragma unroll
          for (int i = 0; i < MC; ++i) {
            const int n = ncol + i * 16 + cg;
            float* const to = row + j * step + n;
            if (!row_there) continue;
            if (ALL || n + 4 <= N) __builtin_memcpy(to, &acc[i][j], 16);
            else
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < N) to[e] = acc[i][j][e];
          }
        }
      }
    };
    if (t0 + (wt + 1) * MT * 16 <= a.T && ncol + MC * 16 <= N) store(std::true_type{});
    else store(std::false_type{});
  }
}

}  // namespace hyena
