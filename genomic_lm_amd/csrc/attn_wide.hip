// attn_wide.hip -- attention over the paged cache for requests of many columns
// (attn_paged.hpp): prefill chunks.  4 DH flops per column and cached token
// against 2 DH bytes per cached token, so from some tens of columns on the
// matrix cores and the softmax's vector work bound it.
//
// 4096 tokens at the end of 32768 of 32 heads of 128, bf16: 1.97 to 2.07
// ms by card, up to 1.04 PFLOP/s of the 2.06 TFLOP under the mask; the library's square product of 16384
// reaches 1.34 and one of 8192 1.20.  Power bounds both: with cache and queries
// all zero, the same instructions take 1.83 ms where random ones took 2.25 (128
// columns per unit then), and the product of 8192 runs at 1.72 PFLOP/s.  So what
// counts is work per column: 256 columns to a unit widen and stage a tile for
// twice as many (2.26 -> 2.13 ms), and O is rescaled only where a maximum rises by
// more than AT_SLACK.  Scores of the next tile ahead of this one's softmax (2.29
// ms), fixed orders of matrix and vector instructions (2.32 to 2.50) and
// accumulators in the other register file (2.29) were slower than the plain order.
// Heads of 64 take 1.20 ms for half the products: the softmax costs the same per
// score, 12.3 vector instructions to an MFMA there against 7.7.
#include "attn_paged.hpp"

namespace hyena {

// A unit is NT columns of one request on one K/V head; its tokens are cut into
// pieces of `tiles` 64-token tiles, the same for all requests and chosen so
// that about wide_target(W) pieces exist, what the chip holds at once: chunks
// with few columns over long contexts then still fill it.  A unit of several
// pieces leaves partial results in the workspace, one slot per piece and head,
// which attn_join.hip adds up; a unit of one piece writes its rows
// directly.
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
  unsigned long long part[8];        // per wave
  int items[8], slots[8], splits[8];
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
// all requests itself (two sums and a scan over them, of lengths that L2 holds)
// instead of waiting for a launch that does it once.  Up to 64 requests each wave
// does it alone, without a barrier; one request needs no scan.
template <int NT, int W>
__device__ __forceinline__ bool find_work(const AttnArgs& a, int lo, int item, AttnShared& sh,
                                          AttnWork& w, int& splits) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = a.Hq / a.Hkv;
  auto units_of = [&](int queries) {
    const int64_t cols = static_cast<int64_t>(queries) * group;
    return cols > lo ? static_cast<int>((cols + NT - 1) / NT) : 0;
  };
  auto tiles_of = [](int len) { return (len + AT_TILE - 1) / AT_TILE; };
  auto piece_tiles = [&](unsigned long long work) {
    const unsigned long long even = (work * a.Hkv + wide_target(W) - 1) / wide_target(W);
    return static_cast<int>(even > AT_SHORT ? (even < 0x7FFFFFFF ? even : 0x7FFFFFFF) : AT_SHORT);
  };
  int tiles = 0, at = 0;
  auto pieces_of = [&](int len) {
    const int n = tiles_of(len);
    return n > tiles ? (n - 1) / tiles + 1 : 1;
  };

  if (a.R == 1) {
    const Request q = request_of(a, 0);
    const int u = units_of(q.queries);
    tiles = piece_tiles(static_cast<unsigned long long>(u) * tiles_of(q.len));
    const int p = pieces_of(q.len);
    splits = p > 1 ? u : 0;
    if (item >= u * p) return false;
    w.r = w.slot = w.split = 0;
    at = item;
  } else if (a.R <= 64) {
    Request q{};
    if (lane < a.R) q = request_of(a, lane);
    const int u = units_of(q.queries);
    unsigned long long work = static_cast<unsigned long long>(u) * tiles_of(q.len);
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o);
    tiles = piece_tiles(work);
    const int p = pieces_of(q.len), items = u * p, slots = p > 1 ? items : 0, split = p > 1 ? u : 0;
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
    const int run = (a.R + 64 * W - 1) / (64 * W);
    const int r0 = min(tid * run, a.R), r1 = min(r0 + run, a.R);
    unsigned long long work = 0;
    for (int r = r0; r < r1; ++r) {
      const Request q = request_of(a, r);
      work += static_cast<unsigned long long>(units_of(q.queries)) * tiles_of(q.len);
    }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) work += __shfl_xor(work, o);
    if (lane == 0) sh.part[wave] = work;
    if (tid == 0) sh.found[4] = 0;
    __syncthreads();
    work = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) work += sh.part[i];
    tiles = piece_tiles(work);
    int items = 0, slots = 0, split = 0;
    for (int r = r0; r < r1; ++r) {
      const Request q = request_of(a, r);
      const int u = units_of(q.queries), p = pieces_of(q.len);
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
    for (int i = 0; i < W; ++i) {
      if (i < wave) {
        before += sh.items[i];
        sbefore += sh.slots[i];
        ubefore += sh.splits[i];
      }
      splits += sh.splits[i];
    }
    if (item >= before && item < before + items) {
      for (int r = r0; r < r1; ++r) {
        const Request q = request_of(a, r);
        const int u = units_of(q.queries), p = pieces_of(q.len);
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
  const Request q = request_of(a, scalar(a.cu + w.r), scalar(a.cu + w.r + 1), scalar(a.lens + w.r));
  w.tok0 = q.tok0;
  w.queries = q.queries;
  w.len = q.len;
  w.ahead = q.ahead;
  w.pieces = uni(pieces_of(w.len));
  w.unit = uni(at / w.pieces);
  w.piece = at - w.unit * w.pieces;
  w.slot = uni(w.slot) + w.unit * w.pieces;
  w.split = uni(w.split) + w.unit;
  return true;
}

// ---------------------------------------------------------------- wide units
// S^T and O^T of 32 columns per wave on 32x32x16 MFMAs.  Lane l: i = l % 32 its
// row of A and column of B and C, hf = l / 32 its half.  Row i of a 32-token
// half tile is token 16 ((i / 4) % 2) + 4 (i / 8) + i % 4, so that C's rows of
// half hf are the 16 consecutive tokens 16 hf .. + 15, in order: the operand of
// the second product, whose k index runs over tokens of one half the same way.
//
// A tile is read once per workgroup (16 bytes per thread and step), widened to
// bf16 and kept in LDS for the W waves of 32 CW columns each, in two buffers:
// tile t + 1, in flight from HBM since tile t - 1, is written to the other buffer
// beside tile t's scores.  16-byte pieces of a row are permuted by the row's
// number so that lanes on consecutive rows read different banks; V's rows, two of
// which span all banks, by half their number.  Bank conflicts are a sixth of the
// cycles in which LDS works (chunk of 4096 at 32768, heads of 128).
constexpr float AT_SLACK = 8.0f;      // how far (log2) scores may pass the reference before O is rescaled

template <typename IO, int DH, bool BIG, int CW, int W>
__global__ __launch_bounds__(64 * W, 2) void attn_wide_kernel(AttnArgs a, int lo, void* space) {
  constexpr int THREADS = 64 * W;
  constexpr int WNT = 32 * CW * W;       // columns per unit
  constexpr int NS = sizeof(IO) == 2 ? 1 : 3;
  using PV = Second<NS>;
  constexpr int TOP = PV::TOP ? PV::TOP - static_cast<int>(AT_SLACK) : 0;   // of a weight at the reference
  constexpr int KS = DH / 16;            // MFMA steps over the head dimension
  constexpr int DT = DH / 32;            // 32-row tiles of O^T
  constexpr int KC = DH / 8;             // 16-byte pieces of a K row in LDS
  constexpr int STEPS = 4 * DH / THREADS; // 16-byte loads per thread of K, and of V
  __shared__ AttnShared sh;
  __shared__ __align__(16) u32x4 s_k[2][AT_TILE * KC];
  __shared__ __align__(16) u32x4 s_v[2][DH * 8];

  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int i = lane & 31, hf = lane >> 5;
  const int head = static_cast<int>(blockIdx.x % a.Hkv);
  const int item = static_cast<int>(blockIdx.x / a.Hkv);
  const int group = a.Hq / a.Hkv;
  const WideSpace ws = wide_space(space, WNT, W);
  AttnWork w;
  int splits;
  const bool have = find_work<WNT, W>(a, lo, item, sh, w, splits);
  if (blockIdx.x == 0 && tid == 0 && space) *ws.used = splits * a.Hkv;
  if (!have) return;

  const int cols = w.queries * group;
  // the units that see most tokens first
  const int units = (cols + WNT - 1) / WNT;
  const int unit = units - 1 - w.unit;
  const int c0 = unit * WNT;
  const int wc = c0 + wave * 32 * CW;                        // the wave's first column
  bool live[CW];
  int qi[CW], qh[CW], pos[CW];                               // query, head, last token seen
#pragma unroll
  for (int b = 0; b < CW; ++b) {
    const int col = wc + 32 * b + i;
    live[b] = col < cols;
    qi[b] = live[b] ? col / group : 0;
    qh[b] = live[b] ? col % group : 0;
    pos[b] = live[b] ? w.ahead + qi[b] : -1;
  }
  const int first_pos = uni(w.ahead + wc / group);           // of the wave's first column
  auto seen_by = [&](int end) { return min(max(w.ahead + (min(end, cols) - 1) / group + 1, 0), w.len); };
  const int wave_seen = wc < cols ? seen_by(wc + 32 * CW) : 0;
  const int seen = seen_by(c0 + WNT);
  const int t_begin = w.piece * w.tiles;
  const int t_end = uni(min((seen + AT_TILE - 1) / AT_TILE, t_begin + w.tiles));
  const int t_wave = uni(min((wave_seen + AT_TILE - 1) / AT_TILE, t_end));

  // queries, with the sign of the scale so that scores only grow with them
  bf16x8 qf[CW][KS][NS];
#pragma unroll
  for (int b = 0; b < CW; ++b) {
    const IO* qp = static_cast<const IO*>(a.q) + (w.tok0 + qi[b]) * a.q_tok +
                   (static_cast<int64_t>(head) * group + qh[b]) * a.q_head;
    const float sign = a.scale < 0.0f ? -1.0f : 1.0f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      float x[8] = {};
      if (live[b]) load8(qp + 16 * s + 8 * hf, 8, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= sign;
      parts<NS>(x, qf[b][s]);
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
  constexpr int KROWS = THREADS / KP;
  const int kr = tid / KP, kc = tid % KP;
  constexpr int VROWS = THREADS / 4;
  const int vd = tid >> 2, vc = tid & 3;
  u32x4 rk[STEPS], rv[STEPS];
  // Pages and scales of AHEAD tiles at a time, a run (BIG: a tile) per lane; a
  // tile's are then read from its lanes, without a load to wait for.
  constexpr int RUNS = BIG ? 1 : 4;
  constexpr int AHEAD = 64 / RUNS;
  struct TileInfo {
    PerRun<int, BIG> page;
    PerRun<float, BIG> ks, vs;
  };
  int ahead_from = 0, ahead_page = -1;
  float ahead_ks = 0.0f, ahead_vs = 0.0f;
  auto look_ahead = [&](int from) {
    ahead_from = from;
    // tiles past the request's last count as the one behind it: a table may hold
    // all but 1024 of 2^31 tokens, and 64 tiles further would wrap
    const int tile = min(from + lane / RUNS, (w.len + AT_TILE - 1) / AT_TILE);
    const int tok = tile * AT_TILE + (lane % RUNS) * 16, j = tok >> lg;
    const int p = tok < w.len && j < a.max_pages ? table[j] : -1;
    ahead_page = p >= 0 && p < a.num_pages ? p : -1;
    const int64_t si = static_cast<int64_t>(max(ahead_page, 0)) * a.Hkv + head;
    ahead_ks = a.k_scale[si];
    ahead_vs = a.v_scale[si];
  };
  auto info_of = [&](int tile) {
    if (tile >= ahead_from + AHEAD) look_ahead(tile);
    TileInfo t;
#pragma unroll
    for (int k = 0; k < RUNS; ++k) {
      const int from = (tile - ahead_from) * RUNS + k;
      t.page.x[k] = __builtin_amdgcn_readlane(ahead_page, from);
      t.ks.x[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ahead_ks), from));
      t.vs.x[k] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(ahead_vs), from));
    }
    return t;
  };
  auto block = [&](const uint8_t* cache, int page) { return cache + max(page, 0) * page_bytes + head_off; };
  auto fetch_k = [&](int tile, const PerRun<int, BIG>& pages) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int row = kr + u * KROWS;
      const uint8_t* b = block(a.k_cache, pages.at(row >> 4));
      if constexpr (BIG)
        rk[u] = *reinterpret_cast<const u32x4*>(b + ((tile * AT_TILE) & pmask) * DH + (row * DH + 16 * kc));
      else
        rk[u] = *reinterpret_cast<const u32x4*>(b + (((tile * AT_TILE + row) & pmask) * DH + 16 * kc));
    }
  };
  auto fetch_v = [&](int tile, const PerRun<int, BIG>& pages) {
    const uint8_t* b = block(a.v_cache, pages.at(vc));
    if constexpr (BIG) b += (tile * AT_TILE) & pmask;
#pragma unroll
    for (int u = 0; u < STEPS; ++u)
      rv[u] = *reinterpret_cast<const u32x4*>(
          b + (((vd + VROWS * u) << lg) + (BIG ? 16 * vc : (tile * AT_TILE + 16 * vc) & pmask)));
  };
  auto stage_k = [&](int buf) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int row = kr + u * KROWS;                        // token of the tile
      const int at = (row & 32) | (8 * ((row >> 2) & 3)) | (4 * ((row >> 4) & 1)) | (row & 3);
      u32x4* kd = s_k[buf] + at * KC;
      kd[(2 * kc) ^ (at & (KC - 1))] = __builtin_bit_cast(u32x4, widen(rk[u][0], rk[u][1]));
      kd[(2 * kc + 1) ^ (at & (KC - 1))] = __builtin_bit_cast(u32x4, widen(rk[u][2], rk[u][3]));
    }
  };
  // places of this thread's V run that hold tokens: the rest must not reach the
  // product (0 * NaN)
  auto cut = [&](int tile, const PerRun<int, BIG>& pages) {
    const int n = pages.at(vc) >= 0 ? w.len - (tile * AT_TILE + 16 * vc) : 0;
    if (__any(n < 16)) {
#pragma unroll
      for (int u = 0; u < STEPS; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) rv[u][e] = keep_places(rv[u][e], e, n);
    }
  };
  auto stage_v = [&](int buf) {
#pragma unroll
    for (int u = 0; u < STEPS; ++u) {
      const int d = vd + VROWS * u;
      u32x4* vdst = s_v[buf] + d * 8;
      vdst[(2 * vc) ^ ((d >> 1) & 7)] = __builtin_bit_cast(u32x4, PV::widen(rv[u][0], rv[u][1]));
      vdst[(2 * vc + 1) ^ ((d >> 1) & 7)] = __builtin_bit_cast(u32x4, PV::widen(rv[u][2], rv[u][3]));
    }
  };

  f32x16 o[CW][DT];
  float m[CW], l[CW];
#pragma unroll
  for (int b = 0; b < CW; ++b) {
    m[b] = AT_NEG;
    l[b] = 0.0f;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[b][d][r] = 0.0f;
  }

  // S^T of a tile from K's buffer
  auto scores = [&](int buf, f32x16 (&s)[CW][2]) {
#pragma unroll
    for (int b = 0; b < CW; ++b)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][h][r] = 0.0f;
#pragma unroll
    for (int k = 0; k < KS; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = 32 * h + i;
        const bf16x8 kf = __builtin_bit_cast(bf16x8, s_k[buf][row * KC + ((2 * k + hf) ^ (row & (KC - 1)))]);
#pragma unroll
        for (int b = 0; b < CW; ++b)
#pragma unroll
          for (int n = NS - 1; n >= 0; --n) s[b][h] = mfma(kf, qf[b][k][n], s[b][h]);
      }
  };

  // scales of this lane's two runs of the tile in work: of the scores, log2 and
  // reciprocal of V's (times 2^-TOP)
  float c[2], vl[2], iv[2];
  // masks of a tile's scores, the columns' maxima (of s + log2 v_scale, what the
  // weights hold), and O moved to a new reference where one has risen by more
  // than AT_SLACK
  auto judge = [&](int tile, f32x16 (&s)[CW][2], const TileInfo& t) {
    int places[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int p = t.page.at(2 * h + hf);
      places[h] = p >= 0 ? min(w.len - (tile * AT_TILE + 32 * h + 16 * hf), 16) : 0;
      // above 0 (and no NaN where there is no page): a masked score stays -inf
      c[h] = fmaxf(t.ks.at(2 * h + hf) * scale2, 0x1p-126f);
      v_scale_of(t.vs.at(2 * h + hf), p, TOP, vl[h], iv[h]);
    }
    if (__any(places[0] < 16 || places[1] < 16) || tile * AT_TILE + AT_TILE - 1 > first_pos) {
#pragma unroll
      for (int b = 0; b < CW; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int lim = min(places[h], pos[b] - (tile * AT_TILE + 32 * h + 16 * hf) + 1);
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (r >= lim) s[b][h][r] = AT_NEG;
        }
    }
    float top[CW];
    bool risen = false;
#pragma unroll
    for (int b = 0; b < CW; ++b) {
      top[b] = AT_NEG;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = s[b][h][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) x = fmaxf(x, s[b][h][r]);
        top[b] = fmaxf(top[b], fmaf(x, c[h], vl[h]));
      }
      top[b] = fmaxf(top[b], xor32(top[b], hf));
      risen |= top[b] > m[b] + AT_SLACK;
    }
    if (__any(risen)) {
#pragma unroll
      for (int b = 0; b < CW; ++b) {
        const float m_new = fmaxf(m[b], top[b]);
        const float f = m_new == AT_NEG ? 1.0f : __builtin_amdgcn_exp2f(m[b] - m_new);
        l[b] *= f;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[b][d][r] *= f;
        m[b] = m_new;
      }
    }
  };

  // P = 2^(c s + log2 v_scale - m + TOP), its sums, and O^T += V^T P^T
  auto weigh = [&](int buf, const f32x16 (&s)[CW][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float off[CW], sum[CW];
#pragma unroll
      for (int b = 0; b < CW; ++b) {
        off[b] = vl[h] - (m[b] == AT_NEG ? 0.0f : m[b] - TOP);
        sum[b] = 0.0f;
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        typename PV::Vec pf[CW][NS];
#pragma unroll
        for (int b = 0; b < CW; ++b) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(fmaf(s[b][h][8 * q + e], c[h], off[b]));
            sum[b] += p[e];
          }
          PV::weights(p, pf[b]);
        }
#pragma unroll
        for (int d = 0; d < DT; ++d) {
          const int row = 32 * d + i;
          const auto vf =
              __builtin_bit_cast(typename PV::Vec, s_v[buf][row * 8 + ((4 * h + 2 * hf + q) ^ ((row >> 1) & 7))]);
#pragma unroll
          for (int b = 0; b < CW; ++b)
#pragma unroll
            for (int n = NS - 1; n >= 0; --n) o[b][d] = PV::mul(vf, pf[b][n], o[b][d]);
        }
      }
#pragma unroll
      for (int b = 0; b < CW; ++b) l[b] = fmaf(sum[b], iv[h], l[b]);
    }
  };

  // Tile t + 1 is written to the other buffers beside tile t's first product, so
  // one barrier per tile is enough, and tile t + 2 is then requested.  Past the
  // end the last tile is requested and written again.
  if (t_begin < t_end) {
    const int last = t_end - 1;
    look_ahead(t_begin);
    TileInfo t0 = info_of(t_begin), t1 = info_of(min(t_begin + 1, last));
    fetch_k(t_begin, t0.page);
    fetch_v(t_begin, t0.page);
    cut(t_begin, t0.page);
    stage_k(0);
    stage_v(0);
    fetch_k(min(t_begin + 1, last), t1.page);
    fetch_v(min(t_begin + 1, last), t1.page);
    __syncthreads();
    for (int tile = t_begin; tile < t_end; ++tile) {
      const int buf = (tile - t_begin) & 1, after = min(tile + 2, last);
      const TileInfo t2 = info_of(after);
      cut(min(tile + 1, last), t1.page);
      if (tile < t_wave) {
        f32x16 s[CW][2];
        scores(buf, s);
        stage_k(buf ^ 1);
        stage_v(buf ^ 1);
        fetch_k(after, t2.page);
        fetch_v(after, t2.page);
        judge(tile, s, t0);
        weigh(buf, s);
      } else {
        stage_k(buf ^ 1);
        stage_v(buf ^ 1);
        fetch_k(after, t2.page);
        fetch_v(after, t2.page);
      }
      t0 = t1;
      t1 = t2;
      __syncthreads();
    }
  }

#pragma unroll
  for (int b = 0; b < CW; ++b) {
    l[b] += xor32(l[b], hf);
    if (!live[b]) continue;
    if (w.pieces == 1) {
      IO* op = static_cast<IO*>(a.out) + ((static_cast<int64_t>(w.tok0) + qi[b]) * a.Hq +
                                          static_cast<int64_t>(head) * group + qh[b]) * DH;
      const float inv = l[b] == 0.0f ? 0.0f : ldexpf(1.0f, -TOP) / l[b];
      // rows 8 e + 4 hf .. + 3 of each 32
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) Io<IO>::st(op, 32 * d + 8 * e + 4 * hf + r, o[b][d][4 * e + r] * inv);
    } else {
      const int64_t slot = static_cast<int64_t>(w.slot + w.piece) * a.Hkv + head;
      const int oc = wave * 32 * CW + 32 * b + i;
      if (hf == 0) {
        ws.ml[slot * 2 * WNT + oc] = m[b];
        ws.ml[slot * 2 * WNT + WNT + oc] = l[b];
      }
      float* op = ws.o + (slot * WNT + oc) * DH;
#pragma unroll
      for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          *reinterpret_cast<f32x4*>(op + 32 * d + 8 * e + 4 * hf) =
              f32x4{o[b][d][4 * e], o[b][d][4 * e + 1], o[b][d][4 * e + 2], o[b][d][4 * e + 3]} * ldexpf(1.0f, -TOP);
    }
  }
  if (w.pieces > 1 && tid == 0 && w.piece == 0)
    ws.head[static_cast<int64_t>(w.split) * a.Hkv + head] =
        AttnUnit{w.pieces, static_cast<int>(w.slot * a.Hkv + head), w.tok0, c0, min(WNT, cols - c0), {0, 0, 0}};
}

// ---------------------------------------------------------------- host
int64_t attn_wide_grid(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv, const WideForm& f) {
  // ceil per request: at most one unit more than its columns' share, and at
  // most the units of max_q queries
  const int64_t group = Hq / Hkv;
  const int64_t share = T * group / f.nt + R;
  const int64_t each = R * ((max_q * group + f.nt - 1) / f.nt);
  return ((share < each ? share : each) + wide_target(f.waves) / Hkv + 1) * Hkv;
}

hipError_t launch_attn_wide(const AttnArgs& a, int limit, void* space) {
  const WideForm f = wide_form(static_cast<int64_t>(a.max_q) * (a.Hq / a.Hkv), a.DH, a.bf16);
  const unsigned grid = static_cast<unsigned>(attn_wide_grid(a.R, a.T, a.max_q, a.Hq, a.Hkv, f));
  auto go = [&](auto big_pages, auto small_pages) {
    if ((1 << a.page_lg) >= AT_TILE) big_pages<<<grid, 64 * f.waves, 0, a.stream>>>(a, limit, space);
    else small_pages<<<grid, 64 * f.waves, 0, a.stream>>>(a, limit, space);
  };
  // columns per wave in sets of 32: nt = 32 CW W
  if (!a.bf16) {
    if (a.DH == 64) go(attn_wide_kernel<float, 64, true, 1, 4>, attn_wide_kernel<float, 64, false, 1, 4>);
    else go(attn_wide_kernel<float, 128, true, 1, 8>, attn_wide_kernel<float, 128, false, 1, 8>);
  } else if (f.nt == 256) {
    if (a.DH == 64) go(attn_wide_kernel<bf16_t, 64, true, 2, 4>, attn_wide_kernel<bf16_t, 64, false, 2, 4>);
    else go(attn_wide_kernel<bf16_t, 128, true, 1, 8>, attn_wide_kernel<bf16_t, 128, false, 1, 8>);
  } else {
    if (a.DH == 64) go(attn_wide_kernel<bf16_t, 64, true, 1, 4>, attn_wide_kernel<bf16_t, 64, false, 1, 4>);
    else go(attn_wide_kernel<bf16_t, 128, true, 1, 4>, attn_wide_kernel<bf16_t, 128, false, 1, 4>);
  }
  return hipGetLastError();
}

}  // namespace hyena
