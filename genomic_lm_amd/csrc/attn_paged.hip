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

// ---------------------------------------------------------------- work split
// A unit is NT columns of one request on one K/V head; its tokens are cut into
// pieces of `piece` 64-token tiles, the same for all requests and chosen so
// that about AT_TARGET pieces exist: every workgroup then has about the same
// work however the lengths differ, and a single long sequence fills the chip.
// A unit of several pieces leaves partial results in the workspace, one slot
// per piece and head, which attn_join_kernel adds up; a unit of one piece
// writes its rows directly.
constexpr int AT_T = 256;                 // threads
constexpr int AT_TILE = 64;               // cached tokens per tile
constexpr int AT_NT = 16;                 // columns per unit
constexpr int AT_TARGET = 2048;           // pieces aimed at
constexpr int AT_MIN_PIECE = 4;           // tiles: one per wave
constexpr int AT_SLOTS = 2 * AT_TARGET;   // a unit of x > 1 pieces worth of work is cut into < 2 x

struct AttnWork {
  int tok0, queries, len;    // the request: first query token, queries (up to max_q), cached tokens
  int ahead;                 // position of the first query
  int r, unit;               // request, column tile
  int piece, pieces;         // this workgroup's piece of the unit's
  int tiles;                 // tiles per piece
  int slot;                  // workspace slot of piece 0 of the unit (per head)
};

struct AttnShared {
  unsigned long long part[AT_T / 64];
  int items[AT_T / 64], slots[AT_T / 64];
  int found[4];              // request, item within it, first slot, set
};

__device__ __forceinline__ void request_of(const AttnArgs& a, int r, int& tok0, int& queries, int& len) {
  const int c0 = a.cu[r], c1 = min(a.cu[r + 1], a.T);
  tok0 = max(c0, 0);
  queries = min(max(c1 - tok0, 0), a.max_q);
  const int64_t cap = static_cast<int64_t>(a.max_pages) << a.page_lg;
  len = static_cast<int>(min<int64_t>(max(a.lens[r], 0), cap));
}

__device__ __forceinline__ int wave_sum_i(int x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) x += __shfl_xor(x, o);
  return x;
}

// Finds the work of item `item`; false if there is none.  Every thread of the
// workgroup takes part.  total_slots: slots in use per head.
__device__ __forceinline__ bool find_work(const AttnArgs& a, int item, AttnShared& sh, AttnWork& w,
                                          int& total_slots) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = a.Hq / a.Hkv;
  const int run = (a.R + AT_T - 1) / AT_T;
  const int r0 = min(tid * run, a.R), r1 = min(r0 + run, a.R);
  auto units_of = [&](int queries) {
    return static_cast<int>((static_cast<int64_t>(queries) * group + AT_NT - 1) / AT_NT);
  };
  auto tiles_of = [](int len) { return (len + AT_TILE - 1) / AT_TILE; };

  // all tiles of all units
  unsigned long long work = 0;
  for (int r = r0; r < r1; ++r) {
    int t, q, n;
    request_of(a, r, t, q, n);
    work += static_cast<unsigned long long>(units_of(q)) * tiles_of(n);
  }
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o);
  if (lane == 0) sh.part[wave] = work;
  if (tid == 0) sh.found[3] = 0;
  __syncthreads();
  work = 0;
#pragma unroll
  for (int i = 0; i < AT_T / 64; ++i) work += sh.part[i];
  const unsigned long long even = (work * a.Hkv + AT_TARGET - 1) / AT_TARGET;
  const int tiles = static_cast<int>(even > AT_MIN_PIECE ? (even < 0x7FFFFFFF ? even : 0x7FFFFFFF) : AT_MIN_PIECE);
  auto pieces_of = [&](int len) {
    const int n = tiles_of(len);
    return n > tiles ? (n - 1) / tiles + 1 : 1;
  };

  // items and slots before this thread's requests
  int items = 0, slots = 0;
  for (int r = r0; r < r1; ++r) {
    int t, q, n;
    request_of(a, r, t, q, n);
    const int u = units_of(q), p = pieces_of(n);
    items += u * p;
    if (p > 1) slots += u * p;
  }
  int before = items, sbefore = slots;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int x = __shfl_up(before, o), y = __shfl_up(sbefore, o);
    if (lane >= o) {
      before += x;
      sbefore += y;
    }
  }
  if (lane == 63) {
    sh.items[wave] = before;
    sh.slots[wave] = sbefore;
  }
  before -= items;
  sbefore -= slots;
  __syncthreads();
  total_slots = 0;
#pragma unroll
  for (int i = 0; i < AT_T / 64; ++i) {
    if (i < wave) {
      before += sh.items[i];
      sbefore += sh.slots[i];
    }
    total_slots += sh.slots[i];
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
        sh.found[3] = 1;
        break;
      }
      before += u * p;
      if (p > 1) sbefore += u * p;
    }
  }
  __syncthreads();
  if (!sh.found[3]) return false;
  w.r = sh.found[0];
  request_of(a, w.r, w.tok0, w.queries, w.len);
  w.ahead = w.len - (min(a.cu[w.r + 1], a.T) - w.tok0);
  w.pieces = pieces_of(w.len);
  w.unit = sh.found[1] / w.pieces;
  w.piece = sh.found[1] % w.pieces;
  w.tiles = tiles;
  w.slot = sh.found[2] + w.unit * w.pieces;
  return true;
}

// ---------------------------------------------------------------- workspace
// int4 header, int4 per slot, then m, l (AT_NT each) and O (AT_NT x DH) per slot
struct AttnSpace {
  int* used;                 // slots in use
  int4* head;                // pieces (0: not a unit's first), first query token, first column, columns
  float* ml;
  float* o;
};
__host__ __device__ __forceinline__ AttnSpace attn_space(void* p) {
  AttnSpace s;
  s.used = static_cast<int*>(p);
  s.head = reinterpret_cast<int4*>(p) + 1;
  s.ml = reinterpret_cast<float*>(s.head + AT_SLOTS);
  s.o = s.ml + AT_SLOTS * 2 * AT_NT;
  return s;
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
__global__ __launch_bounds__(AT_T) void attn_paged_kernel(AttnArgs a) {
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
  const AttnSpace ws = attn_space(a.workspace);
  AttnWork w;
  int total_slots;
  const bool have = find_work(a, item, sh, w, total_slots);
  if (blockIdx.x == 0 && tid == 0 && a.workspace) *ws.used = total_slots * a.Hkv;
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
  int pk, pv;
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

  for (int tile = w.piece * w.tiles + wave; tile < t_end; tile += AT_T / 64) {
    pk = page_of(tile * AT_TILE + 16 * (i >> 2));
    pv = page_of(tile * AT_TILE + 16 * g);
    load_k(tile);
    load_v(tile);
    const int64_t si = static_cast<int64_t>(max(pv, 0)) * a.Hkv + head;
    ks = a.k_scale[si];
    vs = pv >= 0 ? a.v_scale[si] : 0.0f;
    const float c = ks * a.scale * AT_LOG2E;

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
        p[e] *= vs;
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
    if (tid == 0)
      ws.head[slot] = make_int4(w.piece == 0 ? w.pieces : 0, w.tok0, c0, min(AT_NT, cols - c0));
    if ((tid & 15) == 0) {
      ws.ml[slot * 2 * AT_NT + oc] = big;
      ws.ml[slot * 2 * AT_NT + AT_NT + oc] = sum;
    }
    float* op = ws.o + (slot * AT_NT + oc) * DH + od;
#pragma unroll
    for (int e = 0; e < PER; ++e) op[e] = acc[e];
  }
}

// Joins the pieces of each unit that has several: one workgroup per slot, at
// work where the slot is its unit's first.
template <typename IO, int DH>
__global__ __launch_bounds__(AT_T) void attn_join_kernel(AttnArgs a) {
  const AttnSpace ws = attn_space(a.workspace);
  const int64_t slot = blockIdx.x;
  if (slot >= *ws.used) return;
  const int4 h = ws.head[slot];
  if (h.x == 0) return;
  const int head = static_cast<int>(slot % a.Hkv), group = a.Hq / a.Hkv;
  for (int i = threadIdx.x; i < h.w * DH; i += AT_T) {
    const int c = i / DH, d = i % DH;
    float big = AT_NEG;
    for (int p = 0; p < h.x; ++p) big = fmaxf(big, ws.ml[(slot + static_cast<int64_t>(p) * a.Hkv) * 2 * AT_NT + c]);
    float sum = 0.0f, acc = 0.0f;
    for (int p = 0; p < h.x; ++p) {
      const int64_t s = slot + static_cast<int64_t>(p) * a.Hkv;
      const float mk = ws.ml[s * 2 * AT_NT + c];
      const float f = mk == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(mk - big);
      sum = fmaf(f, ws.ml[s * 2 * AT_NT + AT_NT + c], sum);
      acc = fmaf(f, ws.o[(s * AT_NT + c) * DH + d], acc);
    }
    const int cc = h.z + c;
    IO* op = static_cast<IO*>(a.out) +
             ((static_cast<int64_t>(h.y) + cc / group) * a.Hq + static_cast<int64_t>(head) * group + cc % group) * DH;
    Io<IO>::st(op, d, sum == 0.0f ? 0.0f : acc / sum);
  }
}

// ---------------------------------------------------------------- host
static int64_t most_units(int64_t R, int64_t T, int64_t max_q, int64_t group) {
  // ceil per request: at most one unit more than its columns' share, and at
  // most the units of max_q queries
  const int64_t share = T * group / AT_NT + R;
  const int64_t each = R * ((max_q * group + AT_NT - 1) / AT_NT);
  return share < each ? share : each;
}

static bool may_split(int64_t max_pages, int page_lg) {
  return (max_pages << page_lg) > AT_MIN_PIECE * AT_TILE;
}

static int64_t grid_of(int64_t R, int64_t T, int64_t max_q, int64_t max_pages, int page_lg,
                       int64_t Hq, int64_t Hkv) {
  const int64_t units = most_units(R, T, max_q, Hq / Hkv);
  return (units + (may_split(max_pages, page_lg) ? AT_TARGET / Hkv + 1 : 0)) * Hkv;
}

bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t max_pages, int page_lg,
                     int64_t Hq, int64_t Hkv) {
  return grid_of(R, T, max_q, max_pages, page_lg, Hq, Hkv) < (int64_t(1) << 32) / AT_T;
}

size_t attn_paged_workspace(int64_t max_pages, int page_lg, int DH) {
  if (!may_split(max_pages, page_lg)) return 0;
  return 16 + static_cast<size_t>(AT_SLOTS) * (16 + 4 * (2 * AT_NT + AT_NT * DH));
}

hipError_t launch_attn_paged(const AttnArgs& a) {
  const bool split = may_split(a.max_pages, a.page_lg);
  const unsigned grid = static_cast<unsigned>(
      grid_of(a.R, a.T, a.max_q, a.max_pages, a.page_lg, a.Hq, a.Hkv));
  auto go = [&](auto kernel, auto join) {
    kernel<<<grid, AT_T, 0, a.stream>>>(a);
    if (split) join<<<AT_SLOTS, AT_T, 0, a.stream>>>(a);
  };
  if (a.bf16) {
    if (a.DH == 64) go(attn_paged_kernel<bf16_t, 64>, attn_join_kernel<bf16_t, 64>);
    else go(attn_paged_kernel<bf16_t, 128>, attn_join_kernel<bf16_t, 128>);
  } else {
    if (a.DH == 64) go(attn_paged_kernel<float, 64>, attn_join_kernel<float, 64>);
    else go(attn_paged_kernel<float, 128>, attn_join_kernel<float, 128>);
  }
  return hipGetLastError();
}

}  // namespace hyena
