// kv_append.hip -- new keys and values quantised into the paged 8-bit cache.
//
// The striped attention blocks keep their K/V cache in 8 bits (evo2_flash
// README, options table: the fp8 KV cache).  A block of the cache is one page
// of P tokens of one head, with a scale of its own:
//     K  (pages, heads, P, DH),  V  (pages, heads, DH, P),  scales (pages, heads)
// V is stored transposed so that the attention's second product reads tokens,
// its summation axis, contiguously.
//
// For the tokens that a call writes into a block, a = their largest magnitude:
//     s1 = 2^ceil(log2(a / 448)),   s = s1 in a fresh block, else max(s0, s1)
// old codes (those of the places before the lowest that the call writes) times
// s0 / s, new codes e4m3(x / s).  A block is fresh when its first place is
// written by the call.  Scales are powers of two: a block whose
// scale grows is moved without a second rounding (only codes that fall below
// e4m3's normal range lose bits), and a power of two costs a floating format
// no precision.
//
// A token whose key or value holds an infinity or a NaN is stored with a NaN
// key and without its non-finite values: queries that see the token get NaN,
// others do not, as a value of NaN would reach every query through 0 * NaN.
// Scales are taken over finite values.
//
// Reads 2 DH (2 or 4) bytes per token and head and writes 2 DH: HBM bound for
// chunks (13624 tokens of 32 heads of 128, bf16: 78 us, 4.3 TB/s).  For single
// tokens the writes to V are DH single bytes, each in a 64-byte row of its own,
// and a row is what memory reads and writes for it: 128 tokens of 32 heads take
// 10.8 us and move 33 MB out and 28 MB in for 3.1 MB of data.  The attention, for
// which V lies so, reads every row thousands of times for that one write.
#include "fp8.hpp"
#include "serving.hpp"

namespace hyena {

constexpr int KA_T = 256;
constexpr int KA_SHORT = 4;      // runs of up to this many tokens go to one wave
constexpr int KA_GAP = 64;       // (one per lane: a wave looks so far back and ahead)

struct KvPtr {
  const void* src;               // (T, heads, DH) rows, strides in elements
  int64_t tok, head;
  uint8_t* cache;
  float* scale;
};

// Largest finite magnitude, and whether a non-finite one was seen.
__device__ __forceinline__ void see(float x, uint32_t& top, bool& bad) {
  const uint32_t m = mag_bits(x);
  if (m >= 0x7F800000u) bad = true;
  else top = m > top ? m : top;
}

// The codes of the first n0 tokens of a block times f, by `team` lanes.
template <int DH, bool VT>
__device__ __forceinline__ void move_old(uint8_t* blk, int n0, int P, float f, int id, int team) {
  if constexpr (!VT) {
    uint32_t* w = reinterpret_cast<uint32_t*>(blk);
    for (int i = id; i < n0 * (DH / 4); i += team) w[i] = fp8x4_scale(w[i], f);
  } else {
    // words of each row; places past n0 in the last word keep their bytes
    const int words = (n0 + 3) >> 2;
    for (int i = id; i < DH * words; i += team) {
      const int j = i % words, held = n0 - 4 * j;
      uint32_t* w = reinterpret_cast<uint32_t*>(blk + static_cast<int64_t>(i / words) * P) + j;
      const uint32_t old = *w, keep = held >= 4 ? 0u : 0xFFFFFFFFu << (8 * held);
      *w = (fp8x4_scale(old, f) & ~keep) | (old & keep);
    }
  }
}

// One workgroup takes `per` consecutive tokens of one head: the runs that open
// there.  A run is the tokens of one page, which stand together in the call,
// fewer than KA_GAP tokens without a slot between two of them.  Short runs go
// to a wave each, longer ones to the workgroup.
template <typename IO, int DH>
struct Append {
  static constexpr int LPT = DH / 8;               // lanes per token, eight dimensions each
  static constexpr int TPW = 64 / LPT;             // tokens a wave holds at once
  static constexpr int TPG = KA_T / LPT;           // tokens the workgroup holds at once
  static constexpr int STEPS = 64 / TPG;           // steps of a 64-token piece
  static constexpr int VROW = 64 + 4;              // padded row of the transposed tile
  static constexpr unsigned long long LANES = (1ull << LPT) - 1;

  struct Run {
    int64_t t;                                     // first token
    int64_t blk;                                   // block of the cache
    int n0, n;                                     // lowest place, tokens from the first to the last
    bool straight;                                 // place n0 + j for token j
    const int64_t* slots;                          // of the run's tokens
    int64_t page0, pages;                          // first slot of the page, slots of the cache
    uint8_t *kb, *vb;                              // the block's codes

    // the place of token j, -1 if it has none
    __device__ __forceinline__ int place(int j) const {
      if (straight) return n0 + j;
      const int64_t s = slots[j];
      return s >= 0 && s < pages ? static_cast<int>(s - page0) : -1;
    }
  };

  // the wave's run of at most KA_SHORT tokens: one token per LPT lanes
  static __device__ __forceinline__ void by_wave(const KvPtr& kp, const KvPtr& vp, const IO* ks,
                                                 const IO* vs, const Run& u, int P) {
    const int lane = threadIdx.x & 63, j = lane / LPT, c = (lane % LPT) * 8;
    float ok = 0.0f, ov = 0.0f;
    if (u.n0) {
      ok = kp.scale[u.blk];
      ov = vp.scale[u.blk];
    }
    float k[8] = {}, v[8] = {};
    const int at = j < u.n ? u.place(j) : -1;
    if (at >= 0) {
      load8(ks + (u.t + j) * kp.tok + c, 8, k);
      load8(vs + (u.t + j) * vp.tok + c, 8, v);
    }
    uint32_t tk = 0, tv = 0;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      see(k[e], tk, bad);
      see(v[e], tv, bad);
    }
    const bool poison = ((__ballot(bad) >> (j * LPT)) & LANES) != 0;
    float sk = block_scale(max64(tk)), sv = block_scale(max64(tv));
    if (u.n0) {
      if (sk > ok) move_old<DH, false>(u.kb, u.n0, P, ok / sk, lane, 64); else sk = ok;
      if (sv > ov) move_old<DH, true>(u.vb, u.n0, P, ov / sv, lane, 64); else sv = ov;
      // the moved words before the new bytes that share them
      __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
    }
    if (lane == 0) {
      kp.scale[u.blk] = sk;
      vp.scale[u.blk] = sv;
    }
    if (at < 0) return;
    const float ik = 1.0f / sk, iv = 1.0f / sv;          // powers of two: exact
    uint32_t w[2];
    w[0] = fp8x4(k[0] * ik, k[1] * ik, k[2] * ik, k[3] * ik);
    w[1] = fp8x4(k[4] * ik, k[5] * ik, k[6] * ik, k[7] * ik);
    if (poison) w[0] = w[1] = FP8_NAN * 0x01010101u;
    __builtin_memcpy(u.kb + at * DH + c, w, 8);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = mag_bits(v[e]) >= 0x7F800000u ? 0.0f : v[e] * iv;
    w[0] = fp8x4(v[0], v[1], v[2], v[3]);
    w[1] = fp8x4(v[4], v[5], v[6], v[7]);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      u.vb[static_cast<int64_t>(c + e) * P + at] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }

  // The workgroup's run: largest magnitudes first, then codes, in pieces of 64
  // tokens (one piece unless P > 64, kept in registers between the two).
  // Thread: tokens STEPS j0 .. + STEPS - 1 of the piece, so that its codes of
  // one dimension of V are neighbours in the transposed row.
  static __device__ __forceinline__ void by_group(const KvPtr& kp, const KvPtr& vp, const IO* ks,
                                                  const IO* vs, const Run& u, int P, uint8_t* vt,
                                                  uint32_t (*sh_top)[KA_T / 64]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int j0 = (tid / LPT) * STEPS, c = (tid % LPT) * 8;
    float ok = 0.0f, ov = 0.0f;
    if (u.n0) {
      ok = kp.scale[u.blk];
      ov = vp.scale[u.blk];
    }
    Vec8<IO> k[STEPS], v[STEPS];
    uint32_t tk = 0, tv = 0;
    uint32_t poison = 0;                   // bit q: token q holds a non-finite value
    auto piece = [&](int p0) {
      // past the run's end: its last token again, which has a slot
      int j = min(p0 + j0, u.n - 1);
      const IO* kr = ks + (u.t + j) * kp.tok + c;
      const IO* vr = vs + (u.t + j) * vp.tok + c;
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        k[q].load(kr);
        v[q].load(vr);
        if (j + 1 < u.n) {
          ++j;
          kr += kp.tok;
          vr += vp.tok;
        }
      }
      poison = 0;
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        if (u.place(min(p0 + j0 + q, u.n - 1)) < 0) continue;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          see(k[q].get(e), tk, bad);
          see(v[q].get(e), tv, bad);
        }
        if (bad) poison |= 1u << q;
      }
      if (__any(poison)) {
        // of the token: every lane that holds a part of it
#pragma unroll
        for (int o = 1; o < LPT; o <<= 1) poison |= static_cast<uint32_t>(__shfl_xor(static_cast<int>(poison), o));
      }
    };
    const int pieces = (u.n + 63) >> 6;
    for (int p = 0; p < pieces; ++p) piece(p * 64);
    tk = max64(tk);
    tv = max64(tv);
    if (lane == 0) {
      sh_top[0][wave] = tk;
      sh_top[1][wave] = tv;
    }
    __syncthreads();                       // (also: the old scales are read)
#pragma unroll
    for (int w = 0; w < KA_T / 64; ++w) {
      tk = max(tk, sh_top[0][w]);
      tv = max(tv, sh_top[1][w]);
    }
    float sk = block_scale(tk), sv = block_scale(tv);
    if (u.n0) {
      const bool mk = sk > ok, mv = sv > ov;
      if (mk) move_old<DH, false>(u.kb, u.n0, P, ok / sk, tid, KA_T); else sk = ok;
      if (mv) move_old<DH, true>(u.vb, u.n0, P, ov / sv, tid, KA_T); else sv = ov;
      if (mk || mv) __syncthreads();       // the moved words before the new bytes that share them
    }
    if (tid == 0) {
      kp.scale[u.blk] = sk;
      vp.scale[u.blk] = sv;
    }
    const float ik = 1.0f / sk, iv = 1.0f / sv;
    for (int p = 0; p < pieces; ++p) {
      const int p0 = p * 64;
      if (pieces > 1) piece(p0);
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        const int j = p0 + j0 + q;
        uint32_t w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = fp8x4(k[q].get(4 * h) * ik, k[q].get(4 * h + 1) * ik, k[q].get(4 * h + 2) * ik,
                       k[q].get(4 * h + 3) * ik);
        if ((poison >> q) & 1) w[0] = w[1] = FP8_NAN * 0x01010101u;
        const int at = j < u.n ? u.place(j) : -1;
        if (at >= 0) __builtin_memcpy(u.kb + at * DH + c, w, 8);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int q = 0; q < STEPS; ++q) f[q] = v[q].get(e) * iv;
        if (poison) {
#pragma unroll
          for (int q = 0; q < STEPS; ++q)
            if (mag_bits(v[q].get(e)) >= 0x7F800000u) f[q] = 0.0f;
        }
        uint8_t* to = vt + (c + e) * VROW + j0;
        const uint32_t w = fp8x4(f[0], f[1], f[2], f[3]);
        if constexpr (STEPS == 4) *reinterpret_cast<uint32_t*>(to) = w;
        else *reinterpret_cast<uint16_t*>(to) = static_cast<uint16_t>(w);
      }
      __syncthreads();
      // rows of V: 64 places of one dimension, from place n0 + p0
      const int m = u.n - p0 < 64 ? u.n - p0 : 64;
      if (u.straight && m == 64 && ((u.n0 + p0) & 15) == 0) {
        uint8_t* out = u.vb + u.n0 + p0;
#pragma unroll
        for (int i = tid; i < DH * 4; i += KA_T) {
          const int d = i >> 2, o = (i & 3) * 16;
          const uint32_t* from = reinterpret_cast<const uint32_t*>(vt + d * VROW + o);
          *reinterpret_cast<uint4*>(out + static_cast<int64_t>(d) * P + o) =
              make_uint4(from[0], from[1], from[2], from[3]);
        }
      } else {
        for (int i = tid; i < DH * m; i += KA_T) {
          const int d = i / m, o = i % m, at = u.place(p0 + o);
          if (at >= 0) u.vb[static_cast<int64_t>(d) * P + at] = vt[d * VROW + o];
        }
      }
      __syncthreads();
    }
  }
};

// Four waves per SIMD for bf16 (128 VGPRs; heads of 128 spill one): 81 us against
// 86 us at three and 104 us at five (more spills) for 13624 tokens of 32 heads of
// 128; fp32 would spill.
template <typename IO, int DH>
__global__ __launch_bounds__(KA_T, sizeof(IO) == 2 ? 4 : 2) void kv_append_kernel(KvPtr kp, KvPtr vp,
                                                         const int64_t* __restrict__ slots,
                                                         int64_t num_pages, int lg, int T, int H,
                                                         int per) {
  using A = Append<IO, DH>;
  __shared__ __align__(16) uint8_t vt[DH * A::VROW];
  __shared__ uint32_t sh_top[2][KA_T / 64];
  const int P = 1 << lg, pmask = P - 1;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int head = static_cast<int>(blockIdx.x % H);
  const int64_t first = static_cast<int64_t>(blockIdx.x / H) * per;
  const int64_t limit = num_pages << lg;
  const IO* ks = static_cast<const IO*>(kp.src) + head * kp.head;
  const IO* vs = static_cast<const IO*>(vp.src) + head * vp.head;

  auto slot_of = [&](int64_t t) -> int64_t {
    const int64_t s = t >= 0 && t < T ? slots[t] : -1;
    return s >= 0 && s < limit ? s : -1;
  };
  // the slots of 64 tokens from the workgroup's first on and of the 64 before
  // it, the same in every wave: a token opens a run unless the nearest token
  // with a slot before it is in its page and less than KA_GAP tokens away
  const int64_t mine = slot_of(first + lane), old = slot_of(first - 1 - lane);
  const unsigned long long valid = __ballot(mine >= 0), prior = __ballot(old >= 0);
  const int64_t up = __shfl_up(mine, 1);
  const unsigned long long below = valid & ((1ull << lane) - 1);
  const int near = below ? 63 - __clzll(static_cast<long long>(below)) : 0;
  const int back = prior ? __ffsll(static_cast<long long>(prior)) - 1 : 0;
  const int64_t in_window = __shfl(mine, near), in_prior = __shfl(old, back);
  const int64_t last = below ? in_window : prior ? in_prior : -1;
  const int away = below ? lane - near : lane + 1 + back;
  const bool joins = mine >= 0 && last >= 0 && (last >> lg) == (mine >> lg) && away < KA_GAP;
  const unsigned long long opens = valid & ~__ballot(joins);
  const unsigned long long next = __ballot(lane > 0 && mine >= 0 && mine == up + 1 && up >= 0);
  unsigned long long todo = opens & (per < 64 ? (1ull << per) - 1 : ~0ull);
  int turn = 0;
  while (todo) {
    const int i = __ffsll(static_cast<long long>(todo)) - 1;
    todo &= todo - 1;
    typename A::Run u;
    u.t = first + i;
    const int64_t s = __shfl(mine, i);
    const int64_t page = s >> lg;
    u.n0 = static_cast<int>(s & pmask);
    // to the last token with a slot before the next run
    const unsigned long long above = i == 63 ? 0 : ~0ull << (i + 1);
    const unsigned long long stop = opens & above;
    const unsigned long long mem = valid & above & (stop ? (stop & -stop) - 1 : ~0ull);
    u.n = mem ? 64 - __clzll(static_cast<long long>(mem)) - i : 1;
    u.straight = ((above & ((u.n == 64 - i) ? ~0ull : (1ull << (i + u.n)) - 1)) & ~next) == 0;
    if (!stop) {
      // no other run in the window: look on, KA_GAP - 1 tokens past the last one
      for (;;) {
        const int64_t v = lane < KA_GAP - 1 ? slot_of(u.t + u.n + lane) : -1;
        const unsigned long long has = __ballot(v >= 0), other = __ballot(v >= 0 && (v >> lg) != page);
        const unsigned long long in = other ? has & ((other & -other) - 1) : has;
        if (!in) break;
        const int m = 64 - __clzll(static_cast<long long>(in));
        const unsigned long long run = __ballot(v == s + u.n + lane);
        u.straight &= (~run & (m == 64 ? ~0ull : (1ull << m) - 1)) == 0;
        u.n += m;
        if (other) break;
      }
    }
    u.slots = slots + u.t;
    u.page0 = page << lg;
    u.pages = limit;
    u.blk = page * H + head;
    u.kb = kp.cache + u.blk * static_cast<int64_t>(P) * DH;
    u.vb = vp.cache + u.blk * static_cast<int64_t>(P) * DH;
    if (!u.straight) {
      // places in any order: the older codes are those before the lowest
      int over = 0;                      // P - place
      for (int j = lane; j < u.n; j += 64) {
        const int at = u.place(j);
        if (at >= 0) over = max(over, P - at);
      }
      u.n0 = P - static_cast<int>(max64(static_cast<uint32_t>(over)));
    }
    if (u.n <= KA_SHORT) {
      if ((turn++ & (KA_T / 64 - 1)) == wave) A::by_wave(kp, vp, ks, vs, u, P);
    } else {
      A::by_group(kp, vp, ks, vs, u, P, vt, sh_top);
    }
  }
}

// Tokens per workgroup: few, so that single tokens spread over the chip; 64 in
// long calls, where most tokens continue a run and open none.  With 4 and with 64,
// 32 heads of 128 in bf16 (fp32): 256 single tokens 26 and 52 us (28 and 44), 64
// runs of 16 29 and 33 (32 and 33); but one chunk of 512 13.3 and 12.7 (12.8 and
// 13.1), of 1024 17 and 14 (20 and 14), of 4096 50 and 29 (62 and 40).  The number of
// tokens, all that the host knows, is the rule: it favours single tokens, at the
// cost of chunks of 1024 to 4096.
static int tokens_per_group(int64_t T) { return T <= 4096 ? 4 : 64; }
static int64_t append_grid(int64_t T, int64_t H) {
  const int per = tokens_per_group(T);
  return (T + per - 1) / per * H;
}

bool kv_append_fits(int64_t T, int64_t H) { return append_grid(T, H) < (int64_t(1) << 32) / KA_T; }

hipError_t launch_kv_append(const KvAppendArgs& a) {
  const int per = tokens_per_group(a.T);
  const unsigned grid = static_cast<unsigned>(append_grid(a.T, a.H));
  const KvPtr k{a.k, a.k_tok, a.k_head, a.k_cache, a.k_scale};
  const KvPtr v{a.v, a.v_tok, a.v_head, a.v_cache, a.v_scale};
  auto go = [&](auto kernel) {
    kernel<<<grid, KA_T, 0, a.stream>>>(k, v, a.slots, a.num_pages, a.page_lg, a.T, a.H, per);
  };
  if (a.bf16) {
    if (a.DH == 64) go(kv_append_kernel<bf16_t, 64>); else go(kv_append_kernel<bf16_t, 128>);
  } else {
    if (a.DH == 64) go(kv_append_kernel<float, 64>); else go(kv_append_kernel<float, 128>);
  }
  return hipGetLastError();
}

}  // namespace hyena
