// attn_wide.hip -- attention over the paged cache for requests of many columns
// (attn_paged.hpp): prefill chunks.  4 DH flops per column and cached token
// against 2 DH bytes per cached token, so from some tens of columns on the
// matrix cores and the softmax's vector work bound it.
#include "attn_paged.hpp"

namespace hyena {

// A unit is AT_WNT columns of one request on one K/V head; its tokens are cut
// into pieces of `tiles` 64-token tiles, the same for all requests and chosen
// so that about AT_WTARGET pieces exist: chunks with few columns over long
// contexts then still fill the chip.  A unit of several pieces leaves partial
// results in the workspace, one slot per piece and head, which
// attn_wide_join_kernel adds up; a unit of one piece writes its rows directly.
constexpr int AT_WNT = 128;               // columns per unit
constexpr int AT_WTARGET = 512;           // pieces aimed at: two workgroups per CU
constexpr int AT_MIN_PIECE = 4;           // tiles
constexpr int AT_WSLOTS = 2 * AT_WTARGET; // a unit worth x > 1 pieces is cut into fewer than 2 x
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

// Finds the work of item `item` among the requests of more than `lo` columns;
// false if there is none.  Every thread of the workgroup
// takes part.  splits: units of several pieces per head.  Each workgroup walks
// all requests itself (two sums and a scan over them): a launch of its own for
// that costs more at every R up to the limit.  Up to 64 requests each wave
// does it alone, without a barrier; one request needs no scan.
__device__ __forceinline__ bool find_work(const AttnArgs& a, int lo, int item, AttnShared& sh,
                                          AttnWork& w, int& splits) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = a.Hq / a.Hkv;
  auto units_of = [&](int queries) {
    const int64_t cols = static_cast<int64_t>(queries) * group;
    return cols > lo ? static_cast<int>((cols + AT_WNT - 1) / AT_WNT) : 0;
  };
  auto tiles_of = [](int len) { return (len + AT_TILE - 1) / AT_TILE; };
  auto piece_tiles = [&](unsigned long long work) {
    const unsigned long long even = (work * a.Hkv + AT_WTARGET - 1) / AT_WTARGET;
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
  w.r = uni(w.r);
  at = uni(at);
  w.tiles = uni(tiles);
  request_of(a, w.r, w.tok0, w.queries, w.len);
  w.tok0 = uni(w.tok0);
  w.queries = uni(w.queries);
  w.len = uni(w.len);
  w.ahead = w.len - (min(scalar(a.cu + w.r + 1), a.T) - w.tok0);
  w.pieces = uni(pieces_of(w.len));
  w.unit = uni(at / w.pieces);
  w.piece = at - w.unit * w.pieces;
  w.slot = uni(w.slot) + w.unit * w.pieces;
  w.split = uni(w.split) + w.unit;
  return true;
}

// ---------------------------------------------------------------- workspace
// the count of units of several pieces, a header for each, then m, l (AT_WNT
// each) and O (AT_WNT x DH) per slot
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
__device__ __forceinline__ AttnSpace attn_space(void* p) {
  AttnSpace s;
  s.used = static_cast<int*>(p);
  s.head = reinterpret_cast<AttnUnit*>(static_cast<char*>(p) + 16);
  s.ml = reinterpret_cast<float*>(s.head + AT_WSLOTS / 2);      // a split unit has at least two slots
  s.o = s.ml + static_cast<size_t>(AT_WSLOTS) * 2 * AT_WNT;
  return s;
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

template <typename IO, int DH, bool BIG>
__global__ __launch_bounds__(AT_T, 2) void attn_wide_kernel(AttnArgs a, int lo, void* space) {
  constexpr int NS = sizeof(IO) == 2 ? 1 : 3;
  constexpr int KS = DH / 16;            // MFMA steps over the head dimension
  constexpr int DT = DH / 32;            // 32-row tiles of O^T
  constexpr int KC = DH / 8;             // 16-byte pieces of a K row in LDS
  constexpr int STEPS = DH / 64;         // 16-byte loads per thread of K, and of V
  __shared__ AttnShared sh;
  __shared__ __align__(16) u32x4 s_k[2][AT_TILE * KC];
  __shared__ __align__(16) u32x4 s_v[2][DH * 8];

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int i = lane & 31, hf = lane >> 5;
  const int head = static_cast<int>(blockIdx.x % a.Hkv);
  const int item = static_cast<int>(blockIdx.x / a.Hkv);
  const int group = a.Hq / a.Hkv;
  const AttnSpace ws = attn_space(space);
  AttnWork w;
  int splits;
  const bool have = find_work(a, lo, item, sh, w, splits);
  if (blockIdx.x == 0 && tid == 0 && space) *ws.used = splits * a.Hkv;
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
  const int first_pos = uni(w.ahead + wc / group);                // of the wave's first column
  const int wave_seen = wc < cols ? max(w.ahead + (min(wc + 32, cols) - 1) / group + 1, 0) : 0;
  const int seen = max(w.ahead + (min(c0 + AT_WNT, cols) - 1) / group + 1, 0);
  const int t_begin = w.piece * w.tiles;
  const int t_end = uni(min((seen + AT_TILE - 1) / AT_TILE, t_begin + w.tiles));
  const int t_wave = uni(min((wave_seen + AT_TILE - 1) / AT_TILE, t_end));

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

  // ---- staging: step u of a thread is row kr + u KROWS of K (16 dimensions from
  // 16 kc) and row vd + 64 u of V^T (16 tokens from 16 vc)
  constexpr int KP = DH / 16;            // 16-code pieces of a K row
  constexpr int KROWS = AT_T / KP;
  const int kr = tid / KP, kc = tid % KP;
  const int vd = tid >> 2, vc = tid & 3;
  u32x4 rk[STEPS], rv[STEPS];
  auto block = [&](const uint8_t* cache, int page) { return cache + max(page, 0) * page_bytes + head_off; };
  auto fetch = [&](int tile, const PerRun<int, BIG>& pages) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int row = kr + u * KROWS;
      const uint8_t* kb = block(a.k_cache, pages.at(row >> 4));
      const uint8_t* vb = block(a.v_cache, pages.at(vc));
      if constexpr (BIG) {
        kb += ((tile * AT_TILE) & pmask) * DH;
        vb += (tile * AT_TILE) & pmask;
        rk[u] = *reinterpret_cast<const u32x4*>(kb + (row * DH + 16 * kc));
        rv[u] = *reinterpret_cast<const u32x4*>(vb + (((vd + 64 * u) << lg) + 16 * vc));
      } else {
        rk[u] = *reinterpret_cast<const u32x4*>(kb + (((tile * AT_TILE + row) & pmask) * DH + 16 * kc));
        rv[u] = *reinterpret_cast<const u32x4*>(vb + (((vd + 64 * u) << lg) + ((tile * AT_TILE + 16 * vc) & pmask)));
      }
    }
  };
  // places of this thread's V run that hold tokens: the rest must not reach
  // the product (0 * NaN)
  auto cut = [&](int tile, const PerRun<int, BIG>& pages) {
    const int n = pages.at(vc) >= 0 ? w.len - (tile * AT_TILE + 16 * vc) : 0;
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

  PerRun<int, BIG> pg{}, pg_next{}, pg_later{};
  PerRun<float, BIG> ks{}, vs{};
  if (t_begin < t_end) {
    pg = tile_pages<BIG>(a, table, t_begin, w.len);
    fetch(t_begin, pg);
    cut(t_begin, pg);
    stage(0);
    ks = run_scales(a, a.k_scale, pg, head);
    vs = run_scales(a, a.v_scale, pg, head);
    if (t_begin + 1 < t_end) pg_next = tile_pages<BIG>(a, table, t_begin + 1, w.len);
  }
  __syncthreads();
  for (int tile = t_begin; tile < t_end; ++tile) {
    const int buf = (tile - t_begin) & 1;
    const bool more = tile + 1 < t_end;
    // scales and places of this lane's two runs
    float c[2], vl[2], iv[2];
    int places[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int run = tile * AT_TILE + 32 * h + 16 * hf;
      const int p = pg.at(2 * h + hf);
      const float v = vs.at(2 * h + hf);
      places[h] = p >= 0 ? min(w.len - run, 16) : 0;
      // above 0 (and no NaN where there is no page): a masked score stays -inf
      c[h] = fmaxf(ks.at(2 * h + hf) * scale2, 0x1p-126f);
      vl[h] = p >= 0 ? __builtin_amdgcn_logf(v) : AT_NEG;
      iv[h] = p >= 0 ? __builtin_amdgcn_rcpf(v) : 0.0f;
    }
    if (more) {
      fetch(tile + 1, pg_next);
      ks = run_scales(a, a.k_scale, pg_next, head);
      vs = run_scales(a, a.v_scale, pg_next, head);
      if (tile + 2 < t_end) pg_later = tile_pages<BIG>(a, table, tile + 2, w.len);
    }
    if (tile < t_wave) {
      f32x16 s[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[h][r] = 0.0f;
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = 32 * h + i;
          const bf16x8 kf = __builtin_bit_cast(bf16x8, s_k[buf][row * KC + ((2 * k + hf) ^ (row & (KC - 1)))]);
#pragma unroll
          for (int n = NS - 1; n >= 0; --n) s[h] = mfma(kf, qf[k][n], s[h]);
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
        top = fmaxf(top, t * c[h]);
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
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[h][8 * q + e], c[h], off));
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
    if (more) {
      cut(tile + 1, pg_next);
      stage(buf ^ 1);
    }
    pg = pg_next;
    pg_next = pg_later;
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
template <typename IO, int DH>
__global__ __launch_bounds__(AT_T) void attn_wide_join_kernel(AttnArgs a, void* space) {
  constexpr int NT = AT_WNT;
  constexpr int LPC = DH / 4;              // lanes per column
  constexpr int SETS = AT_T / LPC;         // columns the workgroup holds at once
  __shared__ float s_m[SETS], s_l[SETS];
  __shared__ __align__(16) f32x4 s_o[SETS][LPC];
  const AttnSpace ws = attn_space(space);
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
static bool may_split(int64_t max_pages, int page_lg) {
  return (max_pages << page_lg) > AT_MIN_PIECE * AT_TILE;
}

size_t attn_wide_workspace(int64_t max_pages, int page_lg, int DH) {
  if (!may_split(max_pages, page_lg)) return 0;
  return 16 + static_cast<size_t>(AT_WSLOTS) * (sizeof(AttnUnit) / 2 + 4 * (2 * AT_WNT + AT_WNT * DH));
}

int64_t attn_wide_grid(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv) {
  // ceil per request: at most one unit more than its columns' share, and at
  // most the units of max_q queries
  const int64_t group = Hq / Hkv;
  const int64_t share = T * group / AT_WNT + R;
  const int64_t each = R * ((max_q * group + AT_WNT - 1) / AT_WNT);
  return ((share < each ? share : each) + AT_WTARGET / Hkv + 1) * Hkv;
}

hipError_t launch_attn_wide(const AttnArgs& a, int limit, void* workspace) {
  const unsigned grid = static_cast<unsigned>(attn_wide_grid(a.R, a.T, a.max_q, a.Hq, a.Hkv));
  const bool split = may_split(a.max_pages, a.page_lg);
  void* space = split ? workspace : nullptr;
  const bool big = (1 << a.page_lg) >= AT_TILE;
  auto go = [&](auto big_pages, auto small_pages, auto join) {
    if (big) big_pages<<<grid, AT_T, 0, a.stream>>>(a, limit, space);
    else small_pages<<<grid, AT_T, 0, a.stream>>>(a, limit, space);
    if (split) join<<<AT_JOIN, AT_T, 0, a.stream>>>(a, workspace);
  };
  if (a.bf16) {
    if (a.DH == 64)
      go(attn_wide_kernel<bf16_t, 64, true>, attn_wide_kernel<bf16_t, 64, false>, attn_wide_join_kernel<bf16_t, 64>);
    else
      go(attn_wide_kernel<bf16_t, 128, true>, attn_wide_kernel<bf16_t, 128, false>, attn_wide_join_kernel<bf16_t, 128>);
  } else {
    if (a.DH == 64)
      go(attn_wide_kernel<float, 64, true>, attn_wide_kernel<float, 64, false>, attn_wide_join_kernel<float, 64>);
    else
      go(attn_wide_kernel<float, 128, true>, attn_wide_kernel<float, 128, false>, attn_wide_join_kernel<float, 128>);
  }
  return hipGetLastError();
}

}  // namespace hyena
