// attn_paged.hip -- attention over the paged 8-bit K/V cache (kv_append.hip).
//
// The striped attention blocks (evo2_flash README, layer_names table and
// options table: attention beside the Hyena mixers, K/V cache in 8 bits).
// Request r owns query tokens cu[r] .. cu[r+1] and lens[r] cached tokens, its
// queries being the last of them; query head h reads K/V head h / G.  With c =
// scale * k_scale * log2 e per block and query i at position
// pos = lens - (queries) + i,
//     s_j = c q.k_j (j <= pos),  m = max s,  l = sum 2^(s_j - m),
//     o = sum 2^(s_j - m) v_scale v_j / l,   0 where no token is seen.
//
// The columns of the matrix products are (query, query head of the group)
// pairs of one K/V head, so the heads that share a K/V head read it once.
// S^T = K Q^T puts tokens on the rows: a lane then holds 16 consecutive
// tokens of one column, the softmax of a column is 16 registers and two lane
// exchanges, and the result is already the operand of O^T = V^T P^T.  With V
// stored transposed neither product passes through LDS.  e4m3 values are exact
// in bf16, so codes are widened in registers and the block scales are applied
// to S and P.
#include "fp8.hpp"
#include "mfma_common.hpp"
#include "serving.hpp"

namespace hyena {

constexpr float AT_LOG2E = 1.44269504088896340736f;
constexpr float AT_NEG = -__builtin_inff();

// Two kernels share the calls' requests by their columns (queries times group):
//   attn_paged_kernel: up to 16 columns, one MFMA tile wide, bound by reading the
//     cache: four waves on different tiles of the same unit;
//   attn_wide_kernel: more columns, bound by the matrix cores: four waves on 32
//     columns each, tiles widened to bf16 once per workgroup in LDS.

// ---------------------------------------------------------------- work split
// A unit is NT columns of one request on one K/V head; its tokens are cut into
// pieces of `tiles` 64-token tiles, the same for all requests and chosen so
// that about `target` pieces exist: every workgroup then has about the same
// work however the lengths differ, and a single long sequence fills the chip.
// A unit of several pieces leaves partial results in the workspace, one slot
// per piece and head, which attn_join_kernel adds up; a unit of one piece
// writes its rows directly.
constexpr int AT_T = 256;                 // threads
constexpr int AT_TILE = 64;               // cached tokens per tile
constexpr int AT_MIN_PIECE = 4;           // tiles
constexpr int AT_NARROW = 16;             // columns up to which a request is narrow
constexpr int AT_NT = 16;                 // columns per unit, narrow
constexpr int AT_WNT = 128;               // and wide
constexpr int AT_TARGET = 2048;           // pieces aimed at
constexpr int AT_WTARGET = 512;
// a unit worth x > 1 pieces is cut into fewer than 2 x
constexpr int AT_SLOTS = 2 * AT_TARGET;
constexpr int AT_WSLOTS = 2 * AT_WTARGET;
constexpr int AT_JOIN = 512;              // workgroups of the joining launch

struct AttnWork {
  int tok0, queries, len;    // the request: first query token, queries (up to max_q), cached tokens
  int ahead;                 // position of the first query
  int r, unit;               // request, column tile
  int piece, pieces;         // this workgroup's piece of the unit's
  int tiles;                 // tiles per piece
  int slot;                  // workspace slot of piece 0 of the unit (per head)
  int split;                 // number of the unit among those of several pieces (per head)
};

struct AttnShared {
  unsigned long long part[AT_T / 64];
  int items[AT_T / 64], slots[AT_T / 64], splits[AT_T / 64];
  int found[5];              // request, item within it, first slot, first split unit, set
};

__device__ __forceinline__ void request_of(const AttnArgs& a, int r, int& tok0, int& queries, int& len) {
  const int c0 = a.cu[r], c1 = min(a.cu[r + 1], a.T);
  tok0 = max(c0, 0);
  queries = min(max(c1 - tok0, 0), a.max_q);
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_lg;
  len = static_cast<int>(min<int64_t>(max(a.lens[r], 0), cap));
}

// Inclusive sums over the wave.
__device__ __forceinline__ void wave_scan3(int& x, int& y, int& z) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(x, o), b = __shfl_up(y, o), c = __shfl_up(z, o);
    if (lane >= o) {
      x += a;
      y += b;
      z += c;
    }
  }
}

// Finds the work of item `item` among the requests of more than `lo` and at
// most `hi` columns; false if there is none.  Every thread of the workgroup
// takes part.  splits: units of several pieces per head.  Each workgroup walks
// all requests itself (two sums and a scan over them): a launch of its own for
// that costs more at every R up to the limit.  Up to 64 requests each wave
// does it alone, without a barrier; one request needs no scan.
template <int NT, int TARGET>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int lo, int hi, int item, AttnShared& sh,
                                          AttnWork& w, int& splits) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = a.Hq / a.Hkv;
  auto units_of = [&](int queries) {
    const int64_t cols = static_cast<int64_t>(queries) * group;
    return cols > lo && cols <= hi ? static_cast<int>((cols + NT - 1) / NT) : 0;
  };
  auto tiles_of = [](int len) { return (len + AT_TILE - 1) / AT_TILE; };
  auto piece_tiles = [&](unsigned long long work) {
    const unsigned long long even = (work * a.Hkv + TARGET - 1) / TARGET;
    return static_cast<int>(even > AT_MIN_PIECE ? (even < 0x7FFFFFFF ? even : 0x7FFFFFFF) : AT_MIN_PIECE);
  };
  int tiles = 0, at = 0;
  auto pieces_of = [&](int len) {
    const int n = tiles_of(len);
    return n > tiles ? (n - 1) / tiles + 1 : 1;
  };

  if (a.R == 1) {
    int t, q, n;
    request_of(a, 0, t, q, n);
    const int u = units_of(q);
    tiles = piece_tiles(static_cast<unsigned long long>(u) * tiles_of(n));
    const int p = pieces_of(n);
    splits = p > 1 ? u : 0;
    if (item >= u * p) return false;
    w.r = w.slot = w.split = 0;
    at = item;
  } else if (a.R <= 64) {
    int t, q = 0, n = 0;
    if (lane < a.R) request_of(a, lane, t, q, n);
    const int u = units_of(q);
    unsigned long long work = static_cast<unsigned long long>(u) * tiles_of(n);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o);
    tiles = piece_tiles(work);
    const int p = pieces_of(n), items = u * p, slots = p > 1 ? items : 0, split = p > 1 ? u : 0;
    int items_in = items, slots_in = slots, split_in = split;
    wave_scan3(items_in, slots_in, split_in);
    splits = __shfl(split_in, 63);
    const unsigned long long here = __ballot(item < items_in);
    if (!here) return false;
    w.r = __ffsll(static_cast<long long>(here)) - 1;
    at = item - __shfl(items_in - items, w.r);
    w.slot = __shfl(slots_in - slots, w.r);
    w.split = __shfl(split_in - split, w.r);
  } else {
    const int run = (a.R + AT_T - 1) / AT_T;
    const int r0 = min(tid * run, a.R), r1 = min(r0 + run, a.R);
    unsigned long long work = 0;
    for (int r = r0; r < r1; ++r) {
      int t, q, n;
      request_of(a, r, t, q, n);
      work += static_cast<unsigned long long>(units_of(q)) * tiles_of(n);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o);
    if (lane == 0) sh.part[wave] = work;
    if (tid == 0) sh.found[4] = 0;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int i = 0; i < AT_T / 64; ++i) work += sh.part[i];
    tiles = piece_tiles(work);
    int items = 0, slots = 0, split = 0;
    for (int r = r0; r < r1; ++r) {
      int t, q, n;
      request_of(a, r, t, q, n);
      const int u = units_of(q), p = pieces_of(n);
      items += u * p;
      if (p > 1) {
        slots += u * p;
        split += u;
      }
    }
    int before = items, sbefore = slots, ubefore = split;
    wave_scan3(before, sbefore, ubefore);
    if (lane == 63) {
      sh.items[wave] = before;
      sh.slots[wave] = sbefore;
      sh.splits[wave] = ubefore;
    }
    before -= items;
    sbefore -= slots;
    ubefore -= split;
    __syncthreads();
    splits = 0;
#pragma unroll
    for (int i = 0; i < AT_T / 64; ++i) {
      if (i < wave) {
        before += sh.items[i];
        sbefore += sh.slots[i];
        ubefore += sh.splits[i];
      }
      splits += sh.splits[i];
    }
    if (item >= before && item < before + items) {
      for (int r = r0; r < r1; ++r) {
        int t, q, n;
        request_of(a, r, t, q, n);
        const int u = units_of(q), p = pieces_of(n);
        if (item < before + u * p) {
          sh.found[0] = r;
          sh.found[1] = item - before;
          sh.found[2] = sbefore;
          sh.found[3] = ubefore;
          sh.found[4] = 1;
          break;
        }
        before += u * p;
        if (p > 1) {
          sbefore += u * p;
          ubefore += u;
        }
      }
    }
    __syncthreads();
    if (!sh.found[4]) return false;
    w.r = sh.found[0];
    at = sh.found[1];
    w.slot = sh.found[2];
    w.split = sh.found[3];
  }
  // the same in every lane from here on
  w.r = __builtin_amdgcn_readfirstlane(w.r);
  at = __builtin_amdgcn_readfirstlane(at);
  request_of(a, w.r, w.tok0, w.queries, w.len);
  w.ahead = w.len - (min(a.cu[w.r + 1], a.T) - w.tok0);
  w.tiles = __builtin_amdgcn_readfirstlane(tiles);
  w.pieces = pieces_of(w.len);
  w.unit = at / w.pieces;
  w.piece = at % w.pieces;
  w.slot = __builtin_amdgcn_readfirstlane(w.slot) + w.unit * w.pieces;
  w.split = __builtin_amdgcn_readfirstlane(w.split) + w.unit;
  return true;
}

// ---------------------------------------------------------------- workspace
// per kernel: the count of units of several pieces, a header for each, then m,
// l (NT each) and O (NT x DH) per slot
struct AttnUnit {
  int pieces, slot;          // and its first slot; piece p lies p * heads slots on
  int tok0, col0, cols;      // the request's first query token; the unit's first column, its columns
  int pad[3];
};
struct AttnSpace {
  int* used;                 // units of several pieces
  AttnUnit* head;
  float* ml;
  float* o;
};
__host__ __device__ __forceinline__ AttnSpace attn_space(void* p, int nt, int slots) {
  AttnSpace s;
  s.used = static_cast<int*>(p);
  s.head = reinterpret_cast<AttnUnit*>(static_cast<char*>(p) + 16);
  s.ml = reinterpret_cast<float*>(s.head + slots / 2);      // a split unit has at least two slots
  s.o = s.ml + static_cast<size_t>(slots) * 2 * nt;
  return s;
}
constexpr size_t attn_space_bytes(int nt, int slots, int DH) {
  return 16 + static_cast<size_t>(slots) * (16 + 4 * (2 * nt + nt * DH));
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

// Eight floats as NS bf16 parts: one rounding (NS = 1: bf16 queries are exact,
// and P's 2^-9 per weight is below the output's own rounding), or three that
// carry fp32 (NS = 3, fp32 activations).
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

// Codes of places >= n of the four in word `at` (places 4 at .. 4 at + 3) to 0.
__device__ __forceinline__ uint32_t keep_places(uint32_t w, int at, int n) {
  const int k = n - 4 * at;
  return k >= 4 ? w : k <= 0 ? 0u : w & ((1u << (8 * k)) - 1);
}

// ---------------------------------------------------------------- the kernel
// Four waves, each on every fourth tile of the piece with its own m, l and O;
// they are joined through LDS at the end.  Lane l: i = l % 16 is its row of A
// (token of K, dimension of V^T) and its column of B and C, g = l / 16 its
// 16-token run of the tile.  Row i of K's sub-tile t is token 16 (i / 4) + 4 t
// + i % 4, so that C's rows 4 g + r of the four sub-tiles are the run's tokens
// 4 t + r, in order.
template <typename IO, int DH>
__global__ __launch_bounds__(AT_T) void attn_paged_kernel(AttnArgs a, int hi) {
  constexpr int NS = sizeof(IO) == 2 ? 1 : 3;
  constexpr int KH = DH / 64;            // 16-byte loads per K row and lane
  constexpr int KS = DH / 32;            // MFMA steps over the head dimension
  constexpr int DT = DH / 16;            // 16-row tiles of O^T
  constexpr int OROW = DH + 4;
  __shared__ AttnShared sh;
  __shared__ __align__(16) float s_o[AT_T / 64][AT_NT][OROW];
  __shared__ float s_m[AT_T / 64][AT_NT], s_l[AT_T / 64][AT_NT];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i = lane & 15, g = lane >> 4;
  const int head = static_cast<int>(blockIdx.x % a.Hkv);
  const int item = static_cast<int>(blockIdx.x / a.Hkv);
  const int group = a.Hq / a.Hkv;
  const AttnSpace ws = attn_space(a.workspace, AT_NT, AT_SLOTS);
  AttnWork w;
  int splits;
  const bool have = find_work<AT_NT, AT_TARGET>(a, 0, hi, item, sh, w, splits);
  if (blockIdx.x == 0 && tid == 0 && a.workspace) *ws.used = splits * a.Hkv;
  if (!have) return;

  const int cols = w.queries * group, c0 = w.unit * AT_NT;
  const int col = c0 + i;
  const bool live = col < cols;
  const int qi = live ? col / group : 0, qh = live ? col % group : 0;
  const int pos = live ? w.ahead + qi : -1;                  // last token this column sees
  const int first_pos = w.ahead + c0 / group;                // of the unit's first column
  const int last_col = min(c0 + AT_NT, cols) - 1;
  const int seen = max(w.ahead + last_col / group + 1, 0);
  const int t_end = min((seen + AT_TILE - 1) / AT_TILE, (w.piece + 1) * w.tiles);

  bf16x8 qf[KS][NS];
  {
    const IO* qp = static_cast<const IO*>(a.q) + (w.tok0 + qi) * a.q_tok +
                   (static_cast<int64_t>(head) * group + qh) * a.q_head;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8] = {};
      if (live) load8(qp + 64 * (s >> 1) + 16 * g + 8 * (s & 1), 8, x);
      parts<NS>(x, qf[s]);
    }
  }

  const int lg = a.page_lg, pmask = (1 << lg) - 1;
  const int64_t page_bytes = (static_cast<int64_t>(a.Hkv) << lg) * DH;
  const int64_t head_off = (static_cast<int64_t>(head) << lg) * DH;
  const int32_t* table = a.block_table + w.r * a.table_stride;
  // the page of a token, -1 past the end or where the table holds no page
  auto page_of = [&](int tok) {
    const int j = tok >> lg;
    const int p = tok < w.len && j < a.max_pages ? table[j] : -1;
    return p >= 0 && p < a.num_pages ? p : -1;
  };

  f32x4 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d) o[d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  float m = AT_NEG, l = 0.0f;

  u32x4 kr[4][KH], vr[DT];
  float ks, vs;
  int pk, pv, pv_next;
  auto load_k = [&](int tile) {
    const uint8_t* p = a.k_cache + max(pk, 0) * page_bytes + head_off + 16 * g;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const int tok = tile * AT_TILE + 16 * (i >> 2) + 4 * t + (i & 3);
#pragma unroll
      for (int h = 0; h < KH; ++h)
        kr[t][h] = *reinterpret_cast<const u32x4*>(p + (tok & pmask) * DH + 64 * h);
    }
  };
  auto load_v = [&](int tile) {
    const uint8_t* p = a.v_cache + max(pv, 0) * page_bytes + head_off + ((tile * AT_TILE + 16 * g) & pmask);
#pragma unroll
    for (int d = 0; d < DT; ++d)
      vr[d] = *reinterpret_cast<const u32x4*>(p + (static_cast<int64_t>(16 * d + i) << lg));
  };

  // K of the wave's next tile is requested once S no longer needs the current
  // one's registers, V after O; page numbers one tile earlier still
  auto pages = [&](int tile) {
    pk = page_of(tile * AT_TILE + 16 * (i >> 2));
    pv_next = page_of(tile * AT_TILE + 16 * g);
  };
  auto scales = [&]() {
    const int64_t si = static_cast<int64_t>(max(pv_next, 0)) * a.Hkv + head;
    ks = a.k_scale[si];
    vs = pv_next >= 0 ? a.v_scale[si] : 0.0f;
  };
  constexpr int STEP = AT_T / 64;
  int tile = w.piece * w.tiles + wave;
  if (tile < t_end) {
    pages(tile);
    load_k(tile);
    scales();
    pv = pv_next;
    load_v(tile);
    pages(tile + STEP);
  }
  for (; tile < t_end; tile += STEP) {
    const float c = ks * a.scale * AT_LOG2E;
    const float v_scale = vs;
    f32x4 s[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const u32x4 raw = kr[t][k >> 1];
        const bf16x8 kf = (k & 1) ? widen(raw[2], raw[3]) : widen(raw[0], raw[1]);
#pragma unroll
        for (int n = NS - 1; n >= 0; --n) s[t] = mfma16(kf, qf[k][n], s[t]);
      }
    }
    if (tile + STEP < t_end) {
      load_k(tile + STEP);
      scales();
    }
    float x[4][4];
    float top = AT_NEG;
    // places of this lane's run that hold tokens; the tile needs masks where a
    // run is not whole or some column does not see all of it
    const int run0 = tile * AT_TILE + 16 * g;
    const int places = pv >= 0 ? min(max(w.len - run0, 0), 16) : 0;
    const bool masked = __any(places < 16) || tile * AT_TILE + AT_TILE - 1 > first_pos;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) x[t][r] = s[t][r] * c;
    if (masked) {
      const int lim = min(places, pos - run0 + 1);
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (4 * t + r >= lim) x[t][r] = AT_NEG;
      // 0 * NaN: whatever lies past the end must not reach the product
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) vr[d][e] = keep_places(vr[d][e], e, places);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) top = fmaxf(top, x[t][r]);
    top = fmaxf(top, xor16(top, lane));
    top = fmaxf(top, xor32(top, lane >> 5));
    const float m_new = fmaxf(m, top);
    const float base = m_new == AT_NEG ? 0.0f : m_new;      // nothing seen yet: 2^-inf = 0
    if (__any(m_new > m)) {
      const float f = __builtin_amdgcn_exp2f(m - base);
      l *= f;
#pragma unroll
      for (int d = 0; d < DT; ++d) o[d] *= f;
    }
    m = m_new;
    bf16x8 pf[2][NS];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        p[e] = __builtin_amdgcn_exp2f(x[2 * h + (e >> 2)][e & 3] - base);
        l += p[e];
        p[e] *= v_scale;
      }
      parts<NS>(p, pf[h]);
    }
#pragma unroll
    for (int d = 0; d < DT; ++d) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const bf16x8 vf = widen(vr[d][2 * h], vr[d][2 * h + 1]);
#pragma unroll
        for (int n = NS - 1; n >= 0; --n) o[d] = mfma16(vf, pf[h][n], o[d]);
      }
    }
    if (tile + STEP < t_end) {
      pv = pv_next;
      load_v(tile + STEP);
      pages(tile + 2 * STEP);
    }
  }

  // ---- join the four waves
  l += xor16(l, lane);
  l += xor32(l, lane >> 5);
  if (g == 0) {
    s_m[wave][i] = m;
    s_l[wave][i] = l;
  }
#pragma unroll
  for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(&s_o[wave][i][16 * d + 4 * g]) = o[d];
  __syncthreads();
  constexpr int PER = DH / 16;           // dimensions per thread
  const int oc = tid >> 4, od = (tid & 15) * PER;
  float big = AT_NEG;
#pragma unroll
  for (int k = 0; k < AT_T / 64; ++k) big = fmaxf(big, s_m[k][oc]);
  float sum = 0.0f, acc[PER] = {};
#pragma unroll
  for (int k = 0; k < AT_T / 64; ++k) {
    const float mk = s_m[k][oc];
    const float f = mk == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(mk - big);
    sum = fmaf(f, s_l[k][oc], sum);
#pragma unroll
    for (int e = 0; e < PER; ++e) acc[e] = fmaf(f, s_o[k][oc][od + e], acc[e]);
  }
  if (w.pieces == 1) {
    const int cc = c0 + oc;
    if (cc >= cols) return;
    IO* op = static_cast<IO*>(a.out) +
             ((static_cast<int64_t>(w.tok0) + cc / group) * a.Hq + static_cast<int64_t>(head) * group + cc % group) * DH + od;
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < PER; ++e) Io<IO>::st(op, e, acc[e] * inv);
  } else {
    const int64_t slot = static_cast<int64_t>(w.slot + w.piece) * a.Hkv + head;
    if (tid == 0 && w.piece == 0)
      ws.head[static_cast<int64_t>(w.split) * a.Hkv + head] =
          AttnUnit{w.pieces, static_cast<int>(slot), w.tok0, c0, min(AT_NT, cols - c0), {0, 0, 0}};
    if ((tid & 15) == 0) {
      ws.ml[slot * 2 * AT_NT + oc] = big;
      ws.ml[slot * 2 * AT_NT + AT_NT + oc] = sum;
    }
    float* op = ws.o + (slot * AT_NT + oc) * DH + od;
#pragma unroll
    for (int e = 0; e < PER; ++e) op[e] = acc[e];
  }
}

// ---------------------------------------------------------------- wide units
// S^T and O^T of 32 columns per wave on 32x32x16 MFMAs.  Lane l: i = l % 32 its
// row of A and column of B and C, hf = l / 32 its half.  Row i of a 32-token
// half tile is token 16 ((i / 4) % 2) + 4 (i / 8) + i % 4, so that C's rows of
// half hf are the 16 consecutive tokens 16 hf .. + 15, in order: the operand of
// the second product, whose k index runs over tokens of one half the same way.
//
// A tile is read once per workgroup (16 bytes per thread and step), widened to
// bf16 and kept in LDS for the four waves, in two buffers: tile t + 1 is in
// flight from HBM while tile t is multiplied, and written to the other buffer
// after it.  16-byte pieces of a row are permuted by the row's number so that
// lanes on consecutive rows read different banks.
constexpr float AT_SLACK = 8.0f;      // how far (log2) scores may pass the reference before O is rescaled

template <typename IO, int DH>
__global__ __launch_bounds__(AT_T, 2) void attn_wide_kernel(AttnArgs a, int lo) {
  constexpr int NS = sizeof(IO) == 2 ? 1 : 3;
  constexpr int KS = DH / 16;            // MFMA steps over the head dimension
  constexpr int DT = DH / 32;            // 32-row tiles of O^T
  constexpr int KC = DH / 8;             // 16-byte pieces of a K row in LDS
  constexpr int STEPS = DH / 64;         // 16-byte loads per thread of K, and of V
  __shared__ AttnShared sh;
  __shared__ __align__(16) u32x4 s_k[2][AT_TILE * KC];
  __shared__ __align__(16) u32x4 s_v[2][DH * 8];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int i = lane & 31, hf = lane >> 5;
  const int head = static_cast<int>(blockIdx.x % a.Hkv);
  const int item = static_cast<int>(blockIdx.x / a.Hkv);
  const int group = a.Hq / a.Hkv;
  void* space = a.workspace ? static_cast<char*>(a.workspace) + attn_space_bytes(AT_NT, AT_SLOTS, DH) : nullptr;
  const AttnSpace ws = attn_space(space, AT_WNT, AT_WSLOTS);
  AttnWork w;
  int splits;
  const bool have = find_work<AT_WNT, AT_WTARGET>(a, lo, 0x7FFFFFFF, item, sh, w, splits);
  if (blockIdx.x == 0 && tid == 0 && a.workspace) *ws.used = splits * a.Hkv;
  if (!have) return;

  const int cols = w.queries * group;
  // the units that see most tokens first
  const int units = (cols + AT_WNT - 1) / AT_WNT;
  const int unit = units - 1 - w.unit;
  const int c0 = unit * AT_WNT;
  const int wc = c0 + wave * 32;                             // the wave's first column
  const int col = wc + i;
  const bool live = col < cols;
  const int qi = live ? col / group : 0, qh = live ? col % group : 0;
  const int pos = live ? w.ahead + qi : -1;
  const int first_pos = w.ahead + wc / group;                // of the wave's first column
  const int wave_seen = wc < cols ? max(w.ahead + (min(wc + 32, cols) - 1) / group + 1, 0) : 0;
  const int seen = max(w.ahead + (min(c0 + AT_WNT, cols) - 1) / group + 1, 0);
  const int t_begin = w.piece * w.tiles;
  const int t_end = min((seen + AT_TILE - 1) / AT_TILE, t_begin + w.tiles);
  const int t_wave = min((wave_seen + AT_TILE - 1) / AT_TILE, t_end);

  // queries, with the sign of the scale so that scores only grow with them
  bf16x8 qf[KS][NS];
  {
    const IO* qp = static_cast<const IO*>(a.q) + (w.tok0 + qi) * a.q_tok +
                   (static_cast<int64_t>(head) * group + qh) * a.q_head;
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8] = {};
      if (live) load8(qp + 16 * s + 8 * hf, 8, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= sign;
      parts<NS>(x, qf[s]);
    }
  }
  const float scale2 = fabsf(a.scale) * AT_LOG2E;

  const int lg = a.page_lg, pmask = (1 << lg) - 1;
  const int64_t page_bytes = (static_cast<int64_t>(a.Hkv) << lg) * DH;
  const int64_t head_off = (static_cast<int64_t>(head) << lg) * DH;
  const int32_t* table = a.block_table + w.r * a.table_stride;
  auto page_of = [&](int tok) {
    const int j = tok >> lg;
    const int p = tok < w.len && j < a.max_pages ? table[j] : -1;
    return p >= 0 && p < a.num_pages ? p : -1;
  };

  // ---- staging: step u of a thread is row kr + u KROWS of K (16 dimensions from
  // 16 kc) and row vd + 64 u of V^T (16 tokens from 16 vc)
  constexpr int KP = DH / 16;            // 16-code pieces of a K row
  constexpr int KROWS = AT_T / KP;
  const int kr = tid / KP, kc = tid % KP;
  const int vd = tid >> 2, vc = tid & 3;
  u32x4 rk[STEPS], rv[STEPS];
  int pk[STEPS], pv;
  auto pages_of = [&](int tile) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) pk[u] = page_of(tile * AT_TILE + ((kr + u * KROWS) & ~15));
    pv = page_of(tile * AT_TILE + 16 * vc);
  };
  auto fetch = [&](int tile) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int tok = tile * AT_TILE + kr + u * KROWS;
      rk[u] = *reinterpret_cast<const u32x4*>(a.k_cache + max(pk[u], 0) * page_bytes + head_off +
                                              (tok & pmask) * DH + 16 * kc);
      rv[u] = *reinterpret_cast<const u32x4*>(a.v_cache + max(pv, 0) * page_bytes + head_off +
                                              (static_cast<int64_t>(vd + 64 * u) << lg) +
                                              ((tile * AT_TILE + 16 * vc) & pmask));
    }
    // places of this thread's V run that hold tokens: the rest must not reach
    // the product (0 * NaN)
    const int n = pv >= 0 ? w.len - (tile * AT_TILE + 16 * vc) : 0;
    if (n < 16) {
#pragma unroll
      for (int u = 0; u < STEPS; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) rv[u][e] = keep_places(rv[u][e], e, n);
    }
  };
  auto stage = [&](int buf) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int row = kr + u * KROWS;                        // token of the tile
      const int at = (row & 32) | (8 * ((row >> 2) & 3)) | (4 * ((row >> 4) & 1)) | (row & 3);
      u32x4* kd = s_k[buf] + at * KC;
      kd[(2 * kc) ^ (at & (KC - 1))] = __builtin_bit_cast(u32x4, widen(rk[u][0], rk[u][1]));
      kd[(2 * kc + 1) ^ (at & (KC - 1))] = __builtin_bit_cast(u32x4, widen(rk[u][2], rk[u][3]));
      const int d = vd + 64 * u;
      u32x4* vdst = s_v[buf] + d * 8;
      vdst[(2 * vc) ^ (d & 7)] = __builtin_bit_cast(u32x4, widen(rv[u][0], rv[u][1]));
      vdst[(2 * vc + 1) ^ (d & 7)] = __builtin_bit_cast(u32x4, widen(rv[u][2], rv[u][3]));
    }
  };

  f32x16 o[DT];
#pragma unroll
  for (int d = 0; d < DT; ++d)
#pragma unroll
    for (int r = 0; r < 16; ++r) o[d][r] = 0.0f;
  float m = AT_NEG, l = 0.0f;

  if (t_begin < t_end) {
    pages_of(t_begin);
    fetch(t_begin);
    stage(0);
    if (t_begin + 1 < t_end) pages_of(t_begin + 1);
  }
  __syncthreads();
  for (int tile = t_begin; tile < t_end; ++tile) {
    const int buf = (tile - t_begin) & 1;
    const bool more = tile + 1 < t_end;
    if (more) {
      fetch(tile + 1);
      if (tile + 2 < t_end) pages_of(tile + 2);
    }
    if (tile < t_wave) {
      // scales and places of this lane's two runs
      float c[2], vl[2], iv[2];
      int places[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int run = tile * AT_TILE + 32 * h + 16 * hf;
        const int p = page_of(run);
        const int64_t si = static_cast<int64_t>(max(p, 0)) * a.Hkv + head;
        places[h] = p >= 0 ? min(w.len - run, 16) : 0;
        c[h] = a.k_scale[si] * scale2;
        const float vs = a.v_scale[si];
        vl[h] = p >= 0 ? __builtin_amdgcn_logf(vs) : AT_NEG;
        iv[h] = p >= 0 ? 1.0f / vs : 0.0f;
      }
      f32x16 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int r = 0; r < 16; ++r) s[h][r] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const int row = 32 * h + i;
          const bf16x8 kf = __builtin_bit_cast(bf16x8, s_k[buf][row * KC + ((2 * k + hf) ^ (row & (KC - 1)))]);
#pragma unroll
          for (int n = NS - 1; n >= 0; --n) s[h] = mfma(kf, qf[k][n], s[h]);
        }
      }
      const bool masked = __any(places[0] < 16 || places[1] < 16) ||
                          tile * AT_TILE + AT_TILE - 1 > first_pos;
      float top = AT_NEG;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (masked) {
          const int lim = min(places[h], pos - (tile * AT_TILE + 32 * h + 16 * hf) + 1);
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r >= lim) s[h][r] = AT_NEG;
        }
        float t = s[h][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) t = fmaxf(t, s[h][r]);
        // a masked score times a scale of 0, or times what stands for no page, would be NaN
        top = fmaxf(top, t == AT_NEG ? AT_NEG : t * c[h]);
      }
      top = fmaxf(top, xor32(top, hf));
      if (__any(top > m + AT_SLACK || (m == AT_NEG && top > m))) {
        const float m_new = fmaxf(m, top);
        const float f = m_new == AT_NEG ? 1.0f : __builtin_amdgcn_exp2f(m - m_new);
        l *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[d][r] *= f;
        m = m_new;
      }
      const float base = m == AT_NEG ? 0.0f : m;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float off = vl[h] - base;
        float sum = 0.0f;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float x = s[h][8 * q + e];
            p[e] = __builtin_amdgcn_exp2f(masked && x == AT_NEG ? AT_NEG : fmaf(x, c[h], off));
            sum += p[e];
          }
          bf16x8 pf[NS];
          parts<NS>(p, pf);
#pragma unroll
          for (int d = 0; d < DT; ++d) {
            const int row = 32 * d + i;
            const bf16x8 vf = __builtin_bit_cast(bf16x8, s_v[buf][row * 8 + ((4 * h + 2 * hf + q) ^ (row & 7))]);
#pragma unroll
            for (int n = NS - 1; n >= 0; --n) o[d] = mfma(vf, pf[n], o[d]);
          }
        }
        l = fmaf(sum, iv[h], l);
      }
    }
    if (more) stage(buf ^ 1);
    __syncthreads();
  }

  l += xor32(l, hf);
  if (!live) return;
  if (w.pieces == 1) {
    IO* op = static_cast<IO*>(a.out) +
             ((static_cast<int64_t>(w.tok0) + qi) * a.Hq + static_cast<int64_t>(head) * group + qh) * DH;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // rows 8 b + 4 hf .. + 3 of the 32
#pragma unroll
        for (int r = 0; r < 4; ++r) Io<IO>::st(op, 32 * d + 8 * b + 4 * hf + r, o[d][4 * b + r] * inv);
      }
  } else {
    const int64_t slot = static_cast<int64_t>(w.slot + w.piece) * a.Hkv + head;
    if (tid == 0 && w.piece == 0)
      ws.head[static_cast<int64_t>(w.split) * a.Hkv + head] =
          AttnUnit{w.pieces, static_cast<int>(slot), w.tok0, c0, min(AT_WNT, cols - c0), {0, 0, 0}};
    const int oc = wave * 32 + i;
    if (hf == 0) {
      ws.ml[slot * 2 * AT_WNT + oc] = m;
      ws.ml[slot * 2 * AT_WNT + AT_WNT + oc] = l;
    }
    float* op = ws.o + (slot * AT_WNT + oc) * DH;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<f32x4*>(op + 32 * d + 8 * b + 4 * hf) =
            f32x4{o[d][4 * b], o[d][4 * b + 1], o[d][4 * b + 2], o[d][4 * b + 3]};
  }
}

// ---------------------------------------------------------------- joining pieces
// out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p over a unit's pieces.  A
// workgroup takes 16 columns of a unit: DH / 4 lanes per column, four values
// each; with fewer columns than it has lanes for, the lanes left over take
// every other (fourth, eighth) piece and are added through LDS.  The grid is
// fixed and walks the units, whose number only the device knows.
template <typename IO, int DH, int NT>
__global__ __launch_bounds__(AT_T) void attn_join_kernel(AttnArgs a, size_t skip, int slots) {
  constexpr int LPC = DH / 4;              // lanes per column
  constexpr int SETS = AT_T / LPC;         // columns the workgroup holds at once
  __shared__ float s_m[SETS], s_l[SETS];
  __shared__ __align__(16) f32x4 s_o[SETS][LPC];
  const AttnSpace ws = attn_space(static_cast<char*>(a.workspace) + skip, NT, slots);
  const int64_t tasks = static_cast<int64_t>(*ws.used) * (NT / 16);
  const int group = a.Hq / a.Hkv;
  const int set = threadIdx.x / LPC, d = (threadIdx.x % LPC) * 4;
  for (int64_t task = blockIdx.x; task < tasks; task += gridDim.x) {
    const int64_t unit = task / (NT / 16);
    const int first = static_cast<int>(task % (NT / 16)) * 16;
    const AttnUnit u = ws.head[unit];
    const int head = static_cast<int>(unit % a.Hkv);
    const int cols = min(u.cols - first, 16);
    if (cols <= 0) continue;
    int lg = 0;                            // log2 of the columns side by side
    while ((1 << lg) < cols && (1 << lg) < SETS) ++lg;
    const int side = 1 << lg, ways = SETS >> lg;
    const int way = set >> lg;
    for (int c0 = 0; c0 < cols; c0 += side) {
      const int c = c0 + (set & (side - 1));
      float m = AT_NEG, l = 0.0f;
      f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
      if (c < cols) {
#pragma unroll 4
        for (int p = way; p < u.pieces; p += ways) {
          const int64_t s = u.slot + static_cast<int64_t>(p) * a.Hkv;
          const float pm = ws.ml[s * 2 * NT + first + c], pl = ws.ml[s * 2 * NT + NT + first + c];
          const f32x4 po = *reinterpret_cast<const f32x4*>(ws.o + (s * NT + first + c) * DH + d);
          const float big = fmaxf(m, pm);
          const float fo = m == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(m - big);
          const float fp = pm == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(pm - big);
          l = l * fo + pl * fp;
          o = o * fo + po * fp;
          m = big;
        }
      }
      if (ways > 1) {
        if (d == 0) {
          s_m[set] = m;
          s_l[set] = l;
        }
        s_o[set][d >> 2] = o;
        __syncthreads();
        float big = AT_NEG;
        for (int k = 0; k < ways; ++k) big = fmaxf(big, s_m[(k << lg) + (set & (side - 1))]);
        l = 0.0f;
        o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < ways; ++k) {
          const int from = (k << lg) + (set & (side - 1));
          const float f = s_m[from] == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(s_m[from] - big);
          l += f * s_l[from];
          o += f * s_o[from][d >> 2];
        }
        __syncthreads();
      }
      if (way == 0 && c < cols) {
        const int cc = u.col0 + first + c;
        IO* op = static_cast<IO*>(a.out) + ((static_cast<int64_t>(u.tok0) + cc / group) * a.Hq +
                                            static_cast<int64_t>(head) * group + cc % group) * DH + d;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int e = 0; e < 4; ++e) Io<IO>::st(op, e, o[e] * inv);
      }
    }
  }
}

// ---------------------------------------------------------------- host
static int64_t most_units(int64_t R, int64_t T, int64_t max_cols, int64_t group, int64_t nt) {
  // ceil per request: at most one unit more than its columns' share, and at
  // most the units of max_cols columns
  const int64_t share = T * group / nt + R;
  const int64_t each = R * ((max_cols + nt - 1) / nt);
  return share < each ? share : each;
}

static bool may_split(int64_t max_pages, int page_lg) {
  return (max_pages << page_lg) > AT_MIN_PIECE * AT_TILE;
}

struct AttnGrids {
  bool split;
  int64_t narrow, wide;      // workgroups; 0: not launched
  int limit;                 // a request of up to so many columns is narrow
};

static AttnGrids grids_of(int64_t R, int64_t T, int64_t max_q, int64_t max_pages, int page_lg,
                          int64_t Hq, int64_t Hkv) {
  const int64_t group = Hq / Hkv, cols = max_q * group;
  AttnGrids g{};
  g.split = may_split(max_pages, page_lg);
  // a request of its own is wide if it may be: one launch
  const bool wide = cols > AT_NARROW;
  g.limit = wide && R == 1 ? 0 : AT_NARROW;
  if (wide)
    g.wide = (most_units(R, T, cols, group, AT_WNT) + (g.split ? AT_WTARGET / Hkv + 1 : 0)) * Hkv;
  if (g.limit)
    g.narrow = (most_units(R, T, cols < AT_NARROW ? cols : AT_NARROW, group, AT_NT) +
                (g.split ? AT_TARGET / Hkv + 1 : 0)) * Hkv;
  return g;
}

bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t max_pages, int page_lg,
                     int64_t Hq, int64_t Hkv) {
  const AttnGrids g = grids_of(R, T, max_q, max_pages, page_lg, Hq, Hkv);
  constexpr int64_t most = (int64_t(1) << 32) / AT_T;
  return g.narrow < most && g.wide < most;
}

size_t attn_paged_workspace(int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq, int64_t Hkv,
                            int DH) {
  if (!may_split(max_pages, page_lg)) return 0;
  return attn_space_bytes(AT_NT, AT_SLOTS, DH) +
         (max_q * (Hq / Hkv) > AT_NARROW ? attn_space_bytes(AT_WNT, AT_WSLOTS, DH) : 0);
}

hipError_t launch_attn_paged(const AttnArgs& a) {
  const AttnGrids g = grids_of(a.R, a.T, a.max_q, a.max_pages, a.page_lg, a.Hq, a.Hkv);
  const size_t skip = attn_space_bytes(AT_NT, AT_SLOTS, a.DH);
  auto go = [&](auto narrow, auto wide, auto join, auto wide_join) {
    if (g.wide) wide<<<static_cast<unsigned>(g.wide), AT_T, 0, a.stream>>>(a, g.limit);
    if (g.narrow) narrow<<<static_cast<unsigned>(g.narrow), AT_T, 0, a.stream>>>(a, g.limit);
    if (g.split && g.narrow) join<<<AT_JOIN, AT_T, 0, a.stream>>>(a, 0, AT_SLOTS);
    if (g.split && g.wide) wide_join<<<AT_JOIN, AT_T, 0, a.stream>>>(a, skip, AT_WSLOTS);
  };
  if (a.bf16) {
    if (a.DH == 64) go(attn_paged_kernel<bf16_t, 64>, attn_wide_kernel<bf16_t, 64>,
       attn_join_kernel<bf16_t, 64, AT_NT>, attn_join_kernel<bf16_t, 64, AT_WNT>);
    else go(attn_paged_kernel<bf16_t, 128>, attn_wide_kernel<bf16_t, 128>,
       attn_join_kernel<bf16_t, 128, AT_NT>, attn_join_kernel<bf16_t, 128, AT_WNT>);
  } else {
    if (a.DH == 64) go(attn_paged_kernel<float, 64>, attn_wide_kernel<float, 64>,
       attn_join_kernel<float, 64, AT_NT>, attn_join_kernel<float, 64, AT_WNT>);
    else go(attn_paged_kernel<float, 128>, attn_wide_kernel<float, 128>,
       attn_join_kernel<float, 128, AT_NT>, attn_join_kernel<float, 128, AT_WNT>);
  }
  return hipGetLastError();
}

}  // namespace hyena
