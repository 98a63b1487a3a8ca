// attn_paged.hpp -- attention over the paged 8-bit K/V cache (kv_append.hip):
// what the two kernels share (attn_narrow.hip, attn_wide.hip).
//
// The striped attention blocks (evo2_flash README, layer_names table and
// options table: attention beside the Hyena mixers, K/V cache in 8 bits).
// Request r owns query tokens cu[r] .. cu[r+1] and lens[r] cached tokens, its
// queries being the last of them; query head h reads K/V head h / G.  With c =
// scale * k_scale * log2 e per block and query i at position
// pos = lens - (cu[r+1] - cu[r]) + i,
//     s_j = c q.k_j (j <= pos),  m = max (s_j + log2 v_scale),  l = sum 2^(s_j - m),
//     o = sum 2^(s_j - m) v_scale v_j / l,   0 where no token is seen.
//
// The columns of the matrix products are (query, query head of the group)
// pairs of one K/V head, so the heads that share a K/V head read it once.
// S^T = K Q^T puts tokens on the rows: a lane then holds 16 consecutive
// tokens of one column, the softmax of a column is its registers and one or
// two lane exchanges, and the result is already the operand of O^T = V^T P^T.
// V is stored transposed for that product.  e4m3 values are exact in bf16 and
// fp16, so codes are widened in registers and the block scales are applied to S and P.
#pragma once

#include "fp8.hpp"
#include "mfma_common.hpp"
#include "serving.hpp"

namespace hyena {

constexpr float AT_LOG2E = 1.44269504088896340736f;
constexpr float AT_NEG = -__builtin_inff();
constexpr int AT_T = 256;                 // threads
constexpr int AT_TILE = 64;               // cached tokens per tile
constexpr int AT_NARROW = 16;             // columns up to which a request is narrow
constexpr int AT_NARROW2 = 32;            // and in bf16 calls that hold no wider one

// A request: first query token, queries, cached tokens, position of the first
// query.  Queries past T or max_q and tokens past the table are not there; the
// positions of the others do not depend on that, so they come from the offsets
// and the length as given.  Tokens behind the last query's position are dropped
// too: none sees them, and where queries are missing theirs may not have been
// written.  A request without a query in the table counts as cut to it.
struct Request {
  int tok0, queries, len, ahead;
};
__device__ __forceinline__ Request request_of(const AttnArgs& a, int c0, int c1, int lens) {
  Request q;
  q.tok0 = max(c0, 0);
  const int brings = max(max(c1, 0) - q.tok0, 0);          // (the end at 0 first: no difference wraps)
  q.queries = min(max(min(max(c1, 0), a.T) - q.tok0, 0), a.max_q);
  const int cap = a.max_pages << a.page_lg;                // below 2^31
  const int first = max(lens, 0) - brings;
  q.ahead = first < cap ? first : cap - brings;
  q.len = max(min(min(max(lens, 0), cap), q.ahead + q.queries), 0);
  return q;
}
__device__ __forceinline__ Request request_of(const AttnArgs& a, int r) {
  return request_of(a, a.cu[r], a.cu[r + 1], a.lens[r]);
}

// ---------------------------------------------------------------- operands
// Eight codes to bf16 (exact).
__device__ __forceinline__ bf16x8 widen(uint32_t lo, uint32_t hi) {
  bf16x8 r;
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

// Eight floats as NS bf16 parts: one (bf16 queries, exact), or three that carry
// fp32 (fp32 queries and the weights of fp32 calls).
template <int NS>
__device__ __forceinline__ void parts(const float (&x)[8], bf16x8 (&p)[NS]) {
  if constexpr (NS == 1) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = cvt2(x[2 * e], x[2 * e + 1]);
    p[0] = __builtin_bit_cast(bf16x8, w);
  } else {
    u32x4 w0, w1, w2;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t a, b, c;
      split3_pair(x[2 * e], x[2 * e + 1], a, b, c);
      w0[e] = a;
      w1[e] = b;
      w2[e] = c;
    }
    p[0] = __builtin_bit_cast(bf16x8, w0);
    p[1] = __builtin_bit_cast(bf16x8, w1);
    p[2] = __builtin_bit_cast(bf16x8, w2);
  }
}

// Operands of the second product O^T = V^T P^T: V's codes widened, and the weights
// P = 2^(s + log2 v_scale - reference + an offset) in
// * bf16 calls: fp16 of both, one MFMA at bf16's rate.  The codes are exact in it
//   and a weight keeps 11 bits, so its rounding (2^-11 at most) is an eighth of
//   the output's own.  In bf16, with 8 bits, it was as large: a 4096-token chunk
//   at the end of 32768 was 0.0023 off where 32-bit weights and these are 0.0017
//   off, and a row that one weight carries by up to 2^-8, for 1.91 ms instead
//   of 1.98.  Calls bound by the cache take the same time with either.  The offset
//   puts the largest weight near 2^AT_TOP; one below 2^-14 keeps 2^-25 absolutely,
//   2^-32 and less of the largest (v_scale included), far below e4m3's own step;
// * fp32 calls: three bf16 parts of P, without an offset.
// The divisor sums the weights in fp32, unrounded, with v_scale taken out again.
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
constexpr int AT_TOP = 15;                // log2 of the largest fp16 weight
template <int NS> struct Second;
template <> struct Second<1> {
  typedef f16x8 Vec;
  static constexpr int TOP = AT_TOP;
  static __device__ __forceinline__ Vec widen(uint32_t lo, uint32_t hi) {
    Vec r;
    const f16x2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
    const f16x2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
    const f16x2 c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
    const f16x2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
    r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
    r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
    return r;
  }
  static __device__ __forceinline__ void weights(const float (&x)[8], Vec (&p)[1]) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const f32x2 v = {x[2 * e], x[2 * e + 1]};
      w[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2));
    }
    p[0] = __builtin_bit_cast(Vec, w);
  }
  static __device__ __forceinline__ f32x16 mul(Vec a, Vec b, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mul(Vec a, Vec b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <> struct Second<3> {
  typedef bf16x8 Vec;
  static constexpr int TOP = 0;
  static __device__ __forceinline__ Vec widen(uint32_t lo, uint32_t hi) { return hyena::widen(lo, hi); }
  static __device__ __forceinline__ void weights(const float (&x)[8], Vec (&p)[3]) { parts<3>(x, p); }
  static __device__ __forceinline__ f32x16 mul(Vec a, Vec b, f32x16 c) { return mfma(a, b, c); }
  static __device__ __forceinline__ f32x4 mul(Vec a, Vec b, f32x4 c) { return mfma16(a, b, c); }
};

// log2 of a block's V scale and its reciprocal times 2^-top; -inf and 0 where
// there is no page.  A scale of 0 (a cache that was cleared and not written)
// counts as the smallest one.
__device__ __forceinline__ void v_scale_of(float v, int page, int top, float& lv, float& iv) {
  v = fmaxf(v, FP8_MIN_SCALE);
  lv = page >= 0 ? __builtin_amdgcn_logf(v) : AT_NEG;
  iv = page >= 0 ? ldexpf(__builtin_amdgcn_rcpf(v), -top) : 0.0f;
}

// Codes of places >= n of the four in word `at` (places 4 at .. 4 at + 3) to 0.
__device__ __forceinline__ uint32_t keep_places(uint32_t w, int at, int n) {
  const int k = n - 4 * at;
  return k >= 4 ? w : k <= 0 ? 0u : w & ((1u << (8 * k)) - 1);
}

// A load whose address is the same in every lane, through the scalar cache:
// its wait does not queue behind the cache's tiles, which vector loads return
// in order.
template <typename T>
__device__ __forceinline__ T scalar(const T* p) {
  return *(const __attribute__((address_space(4))) T*)(reinterpret_cast<uintptr_t>(p));
}

__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// One value per 16-token run of a tile, the same in every lane; BIG (pages of
// at least a tile): one value for all runs.
template <typename T, bool BIG>
struct PerRun {
  T x[BIG ? 1 : 4];
  // of run k, k per lane
  __device__ __forceinline__ T at(int k) const {
    if constexpr (BIG) {
      return x[0];
    } else {
      // selects of values: an index per lane would move the array to memory
      const T x0 = x[0], x1 = x[1], x2 = x[2], x3 = x[3];
      const T lo = (k & 1) ? x1 : x0, hi = (k & 1) ? x3 : x2;
      return (k & 2) ? hi : lo;
    }
  }
};

// Pages of a tile's runs: -1 past the request's end, or where the table holds
// no page.
template <bool BIG>
__device__ __forceinline__ PerRun<int, BIG> tile_pages(const AttnArgs& a, const int32_t* table, int tile, int len) {
  PerRun<int, BIG> r;
#pragma unroll
  for (int k = 0; k < (BIG ? 1 : 4); ++k) {
    const int tok = tile * AT_TILE + 16 * k, j = tok >> a.page_lg;
    r.x[k] = -1;
    if (tok < len && j < a.max_pages) {
      const int p = scalar(table + j);
      if (p >= 0 && p < a.num_pages) r.x[k] = p;
    }
  }
  return r;
}

template <bool BIG>
__device__ __forceinline__ PerRun<float, BIG> run_scales(const AttnArgs& a, const float* scales,
                                                         const PerRun<int, BIG>& pages, int head) {
  PerRun<float, BIG> r;
#pragma unroll
  for (int k = 0; k < (BIG ? 1 : 4); ++k)
    r.x[k] = scalar(scales + static_cast<int64_t>(max(pages.x[k], 0)) * a.Hkv + head);
  return r;
}

// ---------------------------------------------------------------- partial results
// Where a unit (columns of one request on one K/V head) is worked on by several
// waves or workgroups, each leaves m, l and O of its tokens in the workspace;
// attn_join.hip adds them up.  nt columns per slot: m and l (nt each), O (nt x DH).

// Tables of at most AT_SHORT tiles are not split.
constexpr int AT_SHORT = 4;
inline bool short_table(int64_t max_pages, int page_lg) {
  return (max_pages << page_lg) <= AT_SHORT * AT_TILE;
}

// Narrow: wave w's first unit, begun by an earlier wave, in slot 2 w, its last
// one, continued by the next, in 2 w + 1.
constexpr int AN_GROUPS = 512;            // workgroups: two per CU, all resident
constexpr int AN_WAVES = AN_GROUPS * (AT_T / 64);
struct NarrowSpace {
  int4* head;                // per slot: the unit's first wave, its pieces (0: none), its first query
                             // token, K/V head and columns (from bit 16)
  float* ml;
  float* o;
};
__device__ __forceinline__ NarrowSpace narrow_space(void* p, int nt) {
  NarrowSpace s;
  s.head = static_cast<int4*>(p);
  s.ml = reinterpret_cast<float*>(s.head + 2 * AN_WAVES);
  s.o = s.ml + static_cast<size_t>(2 * AN_WAVES) * 2 * nt;
  return s;
}
// Columns per slot where requests of up to `limit` columns are narrow and the
// call's widest has `cols`.
inline int narrow_columns(int limit, int64_t cols) {
  return static_cast<int>(cols < limit ? cols : limit);
}
inline size_t narrow_bytes(int64_t nt, int DH) {
  return static_cast<size_t>(2 * AN_WAVES) * (sizeof(int4) + 4 * (2 * nt + nt * DH));
}

// Wide: a slot per piece and head.  Eight waves per CU hold wide_target pieces
// at once (two workgroups of four, or one of eight); a unit worth x > 1 of
// them is cut into fewer than 2 x.
constexpr int wide_target(int waves) { return 2048 / waves; }
constexpr int wide_slots(int waves) { return 2 * wide_target(waves); }
struct AttnUnit {
  int pieces, slot;          // and its first slot; piece p lies p * heads slots on
  int tok0, col0, cols;      // the request's first query token; the unit's first column, its columns
  int pad[3];
};
struct WideSpace {
  int* used;                 // units of several pieces
  AttnUnit* head;
  float* ml;
  float* o;
};
__device__ __forceinline__ WideSpace wide_space(void* p, int nt, int waves) {
  WideSpace s;
  s.used = static_cast<int*>(p);
  s.head = reinterpret_cast<AttnUnit*>(static_cast<char*>(p) + 16);
  s.ml = reinterpret_cast<float*>(s.head + wide_slots(waves) / 2);      // a split unit has at least two slots
  s.o = s.ml + static_cast<size_t>(wide_slots(waves)) * 2 * nt;
  return s;
}
inline size_t wide_bytes(int nt, int waves, int DH) {
  return 16 + static_cast<size_t>(wide_slots(waves)) * (sizeof(AttnUnit) / 2 + 4 * (2 * nt + nt * DH));
}

// Columns and waves of a wide unit.  128 columns if no request has more; else
// 256, so that a tile is widened for twice as many.  Heads of 128: eight waves
// of 32 columns (2.26 -> 2.13 ms for a 4096-token chunk at 32768); 64 columns
// per wave need more registers than two waves per SIMD have (2.57 ms).  Heads
// of 64: four waves of 64 columns (1.31 -> 1.20 ms).  fp32's operands fill the
// registers: 32 columns per wave, and heads of 128 spill 9 of them (13 with pages
// under 64 tokens).
struct WideForm {
  int nt, waves;
};
inline WideForm wide_form(int64_t cols, int DH, bool bf16) {
  if (!bf16) return DH == 64 ? WideForm{128, 4} : WideForm{256, 8};
  if (cols <= 128) return WideForm{128, 4};
  return DH == 64 ? WideForm{256, 4} : WideForm{256, 8};
}

// ---------------------------------------------------------------- launches
// Requests of up to `limit` columns (attn_narrow.hip) and of more
// (attn_wide.hip); space NULL: short tables, nothing is split.
hipError_t launch_attn_narrow(const AttnArgs& a, int limit, void* space);
hipError_t launch_attn_wide(const AttnArgs& a, int limit, void* space);
int64_t attn_wide_grid(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv, const WideForm& f);
// Adds up what either left (NULL: was not launched).
hipError_t launch_attn_join(const AttnArgs& a, int limit, void* narrow, void* wide);

}  // namespace hyena
