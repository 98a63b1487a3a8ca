// attn_narrow.hip -- attention over the paged cache for requests of up to 16
// columns, or 32 (attn_paged.hpp): single tokens, or a few with shared heads.
// Bound by reading the cache, 2 DH bytes per cached token and K/V head.
//
// All tiles of all units (a unit: one request on one K/V head) form one list,
// and every wave takes the same number of consecutive ones: however the lengths
// differ, all waves of one resident grid read equally much, from the first
// cycle to the last.  A wave goes through its units one after another, the next
// tile always in flight, across the border of two units as within one.  A unit
// that lies within one wave's share is written by it; the others leave partial
// results (m, l, O) in the workspace, at most two per wave, which
// attn_join.hip adds up.
//
// Heads of 128, bf16: one token over 262144 cached ones of 32 heads 367 us,
// 5.9 TB/s with the join; 64 tokens over up to 8192 of 8 shared heads 101 us and
// the join's 6, 5.0 TB/s; one over 1024 of 32 heads 6 us, the chain of loads of a
// wave that has one tile.  Cutting every request into pieces of one length
// instead took 145 us for the 64, whose lengths differ.
#include "attn_paged.hpp"

namespace hyena {

// A tile in the list, and its request; the same in every lane.
struct Place {
  int r, head, tile, tiles;
  int tok0, queries, len;
  int ahead;                 // position of the request's first query
};

// Tiles of a request per K/V head: 0 if it is not narrow or has no query, and
// one (of masked tokens) if it has queries and nothing cached: their rows are
// written too.
__device__ __forceinline__ int unit_tiles(int queries, int len, int group, int limit) {
  const int64_t cols = static_cast<int64_t>(queries) * group;
  return cols > 0 && cols <= limit ? max((len + AT_TILE - 1) / AT_TILE, 1) : 0;
}

__device__ __forceinline__ void set_request(const AttnArgs& a, int limit, int r, Place& p) {
  const Request q = request_of(a, scalar(a.cu + r), scalar(a.cu + r + 1), scalar(a.lens + r));
  p.r = r;
  p.tok0 = q.tok0;
  p.queries = q.queries;
  p.len = q.len;
  p.ahead = q.ahead;
  p.tiles = unit_tiles(p.queries, p.len, a.Hq / a.Hkv, limit);
}

// The tile after p; there is one.
__device__ __forceinline__ void advance(const AttnArgs& a, int limit, Place& p) {
  if (++p.tile < p.tiles) return;
  p.tile = 0;
  if (++p.head < a.Hkv) return;
  p.head = 0;
  do set_request(a, limit, p.r + 1, p); while (p.tiles == 0 && p.r + 1 < a.R);
}

constexpr int AN_PAIR = 4;

struct NarrowShared {
  unsigned long long before[AT_T], part[AT_T / 64];
};

// The share of wave `w`: its first tile `p`, its number in the list `at`, and
// the tiles per wave; returns the wave's number of tiles.  Every thread of the
// workgroup takes part.
__device__ __forceinline__ long long find_share(const AttnArgs& a, int limit, int w, NarrowShared& sh,
                                                Place& p, long long& at, long long& per) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int group = a.Hq / a.Hkv;
  auto weight = [&](int r) {
    const Request q = request_of(a, r);
    return static_cast<long long>(unit_tiles(q.queries, q.len, group, limit)) * a.Hkv;
  };
  // With more than AN_PAIR columns two tiles at least: a piece of one tile would
  // write and read again as many bytes as the tile (1 x 65536 tokens of one head,
  // 16 columns 26 -> 19 us, 32 columns 28 -> 22 us; four tiles at 32 columns are
  // as fast there and slower in short calls, 17.4 against 15.7 us at 1 x 16384).
  // Beside wide requests the narrow ones are taken to be single tokens.
  const int64_t most = static_cast<int64_t>(a.max_q) * group, cols = most <= limit ? most : group;
  const int least = cols > AN_PAIR ? 2 : 1;
  auto share = [&](long long total) {
    per = max((total + AN_WAVES - 1) / AN_WAVES, static_cast<long long>(least));
    at = per * w;
    return min(per, total - at);
  };
  auto into = [&](int r, long long rest) {
    set_request(a, limit, r, p);
    p.head = uni(static_cast<int>(rest / p.tiles));
    p.tile = uni(static_cast<int>(rest % p.tiles));
  };
  auto shfl = [](long long x, int from) { return __shfl(x, from); };

  if (a.R == 1) {
    const long long n = share(weight(0));
    if (n > 0) into(0, at);
    return n;
  }
  if (a.R <= 64) {
    const long long mine = lane < a.R ? weight(lane) : 0;
    long long end = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const long long x = __shfl_up(end, o);
      if (lane >= o) end += x;
    }
    const long long n = share(shfl(end, 63));
    if (n <= 0) return n;
    const int r = __ffsll(static_cast<long long>(__ballot(at < end))) - 1;
    into(uni(r), at - shfl(end - mine, r));
    return n;
  }
  const int run = (a.R + AT_T - 1) / AT_T;
  const int r0 = min(tid * run, a.R), r1 = min(r0 + run, a.R);
  long long mine = 0;
  for (int r = r0; r < r1; ++r) mine += weight(r);
  long long end = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long x = __shfl_up(end, o);
    if (lane >= o) end += x;
  }
  if (lane == 63) sh.part[wave] = end;
  __syncthreads();
  long long total = 0, base = 0;
#pragma unroll
  for (int i = 0; i < AT_T / 64; ++i) {
    if (i < wave) base += sh.part[i];
    total += sh.part[i];
  }
  sh.before[tid] = base + end - mine;
  __syncthreads();
  const long long n = share(total);
  if (n <= 0) return n;
  // the last thread whose requests begin at or before `at`
  int t = 0;
#pragma unroll
  for (int i = 0; i < AT_T / 64; ++i) {
    const unsigned long long le = __ballot(static_cast<long long>(sh.before[64 * i + lane]) <= at);
    if (le) t = 64 * i + 63 - __clzll(static_cast<long long>(le));
  }
  t = uni(t);
  long long rest = at - static_cast<long long>(sh.before[t]);
  int r = t * run;
  for (;;) {
    const long long x = weight(r);
    if (rest < x) break;
    rest -= x;
    ++r;                                  // ends: the thread's requests hold the tile
  }
  into(uni(r), rest);
  return n;
}

// Lane l: i = l % 16 is its row of A (token of K, dimension of V^T) and its
// column of B and C, g = l / 16 its 16-token run of the tile.  Row i of K's
// sub-tile t is token 16 (i / 4) + 4 t + i % 4, so that C's rows 4 g + r of the
// four sub-tiles are the run's tokens 4 t + r, in order: the operand of the
// second product.
//
// Two waves per SIMD with 16 KiB of the next tile in flight each, 128 KiB per
// CU: more than a CU's share of HBM, ~10 bytes a cycle, delivers in the ~2000
// cycles of a loaded memory's latency.  Three waves leave fewer registers than a
// tile, the next one and O need: 119 to 124 us against 111 at 64 x 8192.
template <typename IO, int DH, bool BIG, int CT>
__global__ __launch_bounds__(AT_T, 2) void attn_narrow_kernel(AttnArgs a, int limit, void* space, int nt) {
  constexpr int NS = sizeof(IO) == 2 ? 1 : 3;
  using PV = Second<NS>;
  constexpr int TOP = PV::TOP;           // log2 of the largest weight
  constexpr int KH = DH / 64;            // 16-byte loads per K row and lane
  constexpr int KS = DH / 32;            // MFMA steps over the head dimension
  constexpr int DT = DH / 16;            // 16-row tiles of O^T
  constexpr bool AHEAD = CT == 1;        // the next unit's queries are loaded early: registers allow it
  __shared__ NarrowShared sh;

  const int tid = threadIdx.x, lane = tid & 63;
  const int i = lane & 15, g = lane >> 4;
  const int wave = uni(static_cast<int>(blockIdx.x) * (AT_T / 64) + (tid >> 6));
  const int group = a.Hq / a.Hkv;
  const NarrowSpace ws = narrow_space(space, nt);
  Place cur;
  long long at = 0, per = 1;
  int left;
  if (!space) {                          // short tables: a unit per wave
    if (wave >= static_cast<int64_t>(a.R) * a.Hkv) return;
    set_request(a, limit, wave / a.Hkv, cur);
    cur.head = wave % a.Hkv;
    cur.tile = 0;
    left = cur.tiles;
  } else {
    left = uni(static_cast<int>(find_share(a, limit, wave, sh, cur, at, per)));
  }
  if (space && lane < 2) ws.head[2 * wave + lane] = int4{0, 0, 0, 0};   // no partial results yet
  if (left > 0) {
    const int lg = a.page_lg, pmask = (1 << lg) - 1;
    const int64_t page_bytes = (static_cast<int64_t>(a.Hkv) << lg) * DH;
    const float scale2 = a.scale * AT_LOG2E;
    const int krow = 16 * (i >> 2) + (i & 3);            // this lane's token of K's sub-tile 0

    u32x4 kr[4][KH], vr[DT];
    bf16x8 qf[CT][KS][NS];
    auto pages_of = [&](const Place& p) {
      return tile_pages<BIG>(a, a.block_table + p.r * a.table_stride, p.tile, p.len);
    };
    // the block of a page; per lane unless BIG
    auto block = [&](const uint8_t* cache, int page, int head) {
      return cache + max(page, 0) * page_bytes + ((static_cast<int64_t>(head) << lg) * DH);
    };
    auto load_k = [&](const Place& p, const PerRun<int, BIG>& pages) {
      const uint8_t* b = block(a.k_cache, pages.at(i >> 2), p.head);
      int off;
      if constexpr (BIG) {
        b += ((p.tile * AT_TILE) & pmask) * DH;
        off = krow * DH + 16 * g;
      } else {
        off = ((p.tile * AT_TILE + krow) & pmask) * DH + 16 * g;   // 4 t + krow stays in the run's page
      }
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int h = 0; h < KH; ++h)
          kr[t][h] = *reinterpret_cast<const u32x4*>(b + off + 4 * t * DH + 64 * h);
    };
    auto load_v = [&](const Place& p, const PerRun<int, BIG>& pages) {
      const uint8_t* b = block(a.v_cache, pages.at(g), p.head);
      int off;
      if constexpr (BIG) {
        b += (p.tile * AT_TILE) & pmask;
        off = (i << lg) + 16 * g;
      } else {
        off = (i << lg) + ((p.tile * AT_TILE + 16 * g) & pmask);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d)
        vr[d] = *reinterpret_cast<const u32x4*>(b + off + (d << (lg + 4)));
    };
    // the queries of a unit, on their way while another's last tiles are computed,
    // and their operands once they are needed
    Vec8<IO> qr[CT][KS];
    auto load_q = [&](const Place& p) {
#pragma unroll
      for (int n = 0; n < CT; ++n) {
        const int col = 16 * n + i;
        const IO* qp = static_cast<const IO*>(a.q) + (p.tok0 + col / group) * a.q_tok +
                       (static_cast<int64_t>(p.head) * group + col % group) * a.q_head + 16 * g;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          qr[n][s] = Vec8<IO>{};
          if (col < p.queries * group) qr[n][s].load(qp + 64 * (s >> 1) + 8 * (s & 1));
        }
      }
    };
    auto set_q = [&]() {
#pragma unroll
      for (int n = 0; n < CT; ++n)
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = qr[n][s].get(e);
          parts<NS>(x, qf[n][s]);
        }
    };

    f32x4 o[CT][DT];
    float m[CT], l[CT];
    auto clear = [&]() {
#pragma unroll
      for (int n = 0; n < CT; ++n) {
#pragma unroll
        for (int d = 0; d < DT; ++d) o[n][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        m[n] = AT_NEG;
        l[n] = 0.0f;
      }
    };

    Place next = cur, later = cur;
    int from = cur.tile;                   // the unit's first tile in this share
    PerRun<int, BIG> pg = pages_of(cur), pg_next = pg, pg_later = pg;
    load_q(cur);
    load_k(cur, pg);
    load_v(cur, pg);
    PerRun<float, BIG> ks = run_scales(a, a.k_scale, pg, cur.head), vs = run_scales(a, a.v_scale, pg, cur.head);
    set_q();
    if (left > 1) {
      advance(a, limit, next);
      pg_next = pages_of(next);
      if (AHEAD && next.tile == 0) load_q(next);
    }
    clear();
    for (;;) {
      // cur is in flight or loaded, next's pages are known
      const bool more = left > 1;
      const float c = ks.at(g) * scale2;
      const int page = pg.at(g);
      float lv, iv;                        // log2 of V's scale, its reciprocal (times 2^-TOP)
      v_scale_of(vs.at(g), page, TOP, lv, iv);
      const bool ends = cur.tile + 1 == cur.tiles;
      if (left > 2) {
        later = next;
        advance(a, limit, later);
        pg_later = pages_of(later);
      }
      f32x4 s[CT][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) {
#pragma unroll
        for (int n = 0; n < CT; ++n) s[n][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          const u32x4 raw = kr[t][k >> 1];
          const bf16x8 kf = (k & 1) ? widen(raw[2], raw[3]) : widen(raw[0], raw[1]);
#pragma unroll
          for (int n = 0; n < CT; ++n)
#pragma unroll
            for (int e = NS - 1; e >= 0; --e) s[n][t] = mfma16(kf, qf[n][k][e], s[n][t]);
        }
      }
      const int run0 = cur.tile * AT_TILE + 16 * g;
      const int places = page >= 0 ? min(max(cur.len - run0, 0), 16) : 0;
      if (more) {
        if (ends) {
          if (!AHEAD) load_q(next);
          set_q();
        }
        if (AHEAD && left > 2 && later.tile == 0) load_q(later);
        load_k(next, pg_next);
        ks = run_scales(a, a.k_scale, pg_next, next.head);
        vs = run_scales(a, a.v_scale, pg_next, next.head);
      }

      // masks where a run is not whole or some column does not see all of it
      const bool mask = __any(places < 16) || cur.tile * AT_TILE + AT_TILE - 1 > cur.ahead;
      if (mask) {
        // 0 * NaN: whatever lies past the end must not reach the product
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) vr[d][e] = keep_places(vr[d][e], e, places);
      }
      typename PV::Vec pf[CT][2][NS];
#pragma unroll
      for (int n = 0; n < CT; ++n) {
        const int pos = cur.ahead + (16 * n + i) / group;  // last token this column sees
        float x[4][4];
        float top = AT_NEG;
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) x[t][r] = fmaf(s[n][t][r], c, lv);
        if (mask) {
          const int lim = min(places, pos - run0 + 1);
#pragma unroll
          for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (4 * t + r >= lim) x[t][r] = AT_NEG;
        }
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) top = fmaxf(top, x[t][r]);
        top = fmaxf(top, xor16(top, lane));
        top = fmaxf(top, xor32(top, lane >> 5));
        const float m_new = fmaxf(m[n], top);
        const float base = m_new == AT_NEG ? 0.0f : m_new;  // nothing seen yet: 2^-inf = 0
        if (__any(m_new > m[n])) {
          const float f = __builtin_amdgcn_exp2f(m[n] - base);
          l[n] *= f;
#pragma unroll
          for (int d = 0; d < DT; ++d) o[n][d] *= f;
        }
        m[n] = m_new;
        const float from_base = base - TOP;
        float sum = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float p[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(x[2 * h + (e >> 2)][e & 3] - from_base);
            sum += p[e];
          }
          PV::weights(p, pf[n][h]);
        }
        l[n] = fmaf(sum, iv, l[n]);
      }
#pragma unroll
      for (int d = 0; d < DT; ++d) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const auto vf = PV::widen(vr[d][2 * h], vr[d][2 * h + 1]);
#pragma unroll
          for (int n = 0; n < CT; ++n)
#pragma unroll
            for (int e = NS - 1; e >= 0; --e) o[n][d] = PV::mul(vf, pf[n][h][e], o[n][d]);
        }
      }
      if (more) load_v(next, pg_next);

      if (ends || !more) {
        // leave the unit: its columns are on lanes i of every g
        const int cols = cur.queries * group;
#pragma unroll
        for (int n = 0; n < CT; ++n) {
          const int col = 16 * n + i;
          l[n] += xor16(l[n], lane);
          l[n] += xor32(l[n], lane >> 5);
          if (col >= cols) continue;
          if (from == 0 && ends) {
            const float inv = l[n] == 0.0f ? 0.0f : ldexpf(1.0f, -TOP) / l[n];
            IO* op = static_cast<IO*>(a.out) + ((static_cast<int64_t>(cur.tok0) + col / group) * a.Hq +
                                                static_cast<int64_t>(cur.head) * group + col % group) * DH;
#pragma unroll
            for (int d = 0; d < DT; ++d)
#pragma unroll
              for (int r = 0; r < 4; ++r) Io<IO>::st(op, 16 * d + 4 * g + r, o[n][d][r] * inv);
          } else {
            const int64_t slot = 2 * static_cast<int64_t>(wave) + (from == 0 ? 1 : 0);
            if (g == 0) {
              ws.ml[(slot * 2) * nt + col] = m[n];
              ws.ml[(slot * 2 + 1) * nt + col] = l[n];
            }
            float* op = ws.o + (slot * nt + col) * DH;
#pragma unroll
            for (int d = 0; d < DT; ++d) *reinterpret_cast<f32x4*>(op + 16 * d + 4 * g) = o[n][d] * ldexpf(1.0f, -TOP);
          }
        }
        if (!(from == 0 && ends)) {
          // the waves that share the unit: the list's places of its tiles by `per`
          const long long begin = at - cur.tile, last = begin + cur.tiles - 1;
          const int w0 = from == 0 ? wave : static_cast<int>(begin / per);
          if (lane == (from == 0 ? 1 : 0))   // the lane that cleared it
            ws.head[2 * wave + lane] =
                make_int4(w0, static_cast<int>(last / per) - w0 + 1, cur.tok0, cur.head | cols << 16);
        }
        if (!more) break;
        clear();
        from = 0;
      }
      ++at;
      cur = next;
      next = later;
      pg = pg_next;
      pg_next = pg_later;
      --left;
    }
  }
}

// ---------------------------------------------------------------- host
hipError_t launch_attn_narrow(const AttnArgs& a, int limit, void* space) {
  const int nt = narrow_columns(limit, static_cast<int64_t>(a.max_q) * (a.Hq / a.Hkv));
  const int64_t units = static_cast<int64_t>(a.R) * a.Hkv;
  const unsigned grid = space ? AN_GROUPS : static_cast<unsigned>((units + AT_T / 64 - 1) / (AT_T / 64));
  auto go = [&](auto big_pages, auto small_pages) {
    if ((1 << a.page_lg) >= AT_TILE) big_pages<<<grid, AT_T, 0, a.stream>>>(a, limit, space, nt);
    else small_pages<<<grid, AT_T, 0, a.stream>>>(a, limit, space, nt);
  };
  auto sets = [&](auto ct) {
    constexpr int CT = decltype(ct)::value;
    if (a.DH == 64) go(attn_narrow_kernel<bf16_t, 64, true, CT>, attn_narrow_kernel<bf16_t, 64, false, CT>);
    else go(attn_narrow_kernel<bf16_t, 128, true, CT>, attn_narrow_kernel<bf16_t, 128, false, CT>);
  };
  if (a.bf16) {
    if (nt <= 16) sets(std::integral_constant<int, 1>{}); else sets(std::integral_constant<int, 2>{});
  } else {
    if (a.DH == 64) go(attn_narrow_kernel<float, 64, true, 1>, attn_narrow_kernel<float, 64, false, 1>);
    else go(attn_narrow_kernel<float, 128, true, 1>, attn_narrow_kernel<float, 128, false, 1>);
  }
  return hipGetLastError();
}

}  // namespace hyena
