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
// old codes times s0 / s, new codes e4m3(x / s).  A block is fresh when its
// first place is written by the call.  Scales are powers of two: a block whose
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
// chunks; for single tokens the writes to V are DH single bytes, each in a
// line of its own, and the call is bound by their latency.
#include "fp8.hpp"
#include "serving.hpp"

namespace hyena {

constexpr int KA_T = 256;
constexpr int KA_SHORT = 4;      // runs of up to this many tokens go to one wave

struct KvPtr {
  const void* src;               // (T, heads, DH) rows, strides in elements
  int64_t tok, head;
  uint8_t* cache;
  float* scale;
};

// Largest finite magnitude and the presence of a non-finite one, per element.
__device__ __forceinline__ void see(const float (&x)[8], uint32_t& top, bool& bad) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t m = mag_bits(x[e]);
    if (m >= 0x7F800000u) bad = true;
    else top = m > top ? m : top;
  }
}

__device__ __forceinline__ uint32_t wave_max_u(uint32_t x) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = static_cast<uint32_t>(__shfl_xor(static_cast<int>(x), o));
    x = x > y ? x : y;
  }
  return x;
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

// One workgroup takes `per` consecutive tokens of one head: the runs of
// consecutive places of one page that start there.  Short runs go to a wave
// each, longer ones to the workgroup.
template <typename IO, int DH>
__global__ __launch_bounds__(KA_T) void kv_append_kernel(KvPtr kp, KvPtr vp,
                                                         const int64_t* __restrict__ slots,
                                                         int64_t num_pages, int lg, int T, int H,
                                                         int per) {
  constexpr int LPT = DH / 8;               // lanes per token
  constexpr int TPW = 64 / LPT;             // tokens a wave holds at once
  constexpr int TPG = KA_T / LPT;           // tokens the workgroup holds at once
  constexpr int STEPS = 64 / TPG;           // steps of a 64-token piece
  constexpr int VROW = 64 + 8;              // padded row of the transposed tile
  __shared__ __align__(16) uint8_t vt[DH * VROW];
  __shared__ uint32_t sh_top[2][KA_T / 64];
  const int P = 1 << lg, pmask = P - 1;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int head = static_cast<int>(blockIdx.x % H);
  const int64_t first = static_cast<int64_t>(blockIdx.x / H) * per;
  const int64_t limit = num_pages << lg;
  const IO* ks = static_cast<const IO*>(kp.src) + head * kp.head;
  const IO* vs = static_cast<const IO*>(vp.src) + head * vp.head;

  auto slot_of = [&](int64_t t) -> int64_t {
    const int64_t s = t >= 0 && t < T ? slots[t] : -1;
    return s >= 0 && s < limit ? s : -1;
  };
  // does token t open a run: a valid slot that does not continue the one before it
  auto opens = [&](int64_t t) {
    const int64_t s = slot_of(t);
    if (s < 0) return false;
    return (s & pmask) == 0 || slot_of(t - 1) != s - 1;
  };
  // tokens of the run that t opens (every lane of the wave takes part)
  auto run_of = [&](int64_t t, int64_t s) {
    const int room = P - static_cast<int>(s & pmask);
    int n = 0;
    while (n < room) {
      const int i = n + lane;
      const bool in = i < room && slot_of(t + i) == s + i;
      const unsigned long long miss = ~__ballot(in);
      if (miss) return n + __ffsll(static_cast<long long>(miss)) - 1;
      n += 64;
    }
    return room;
  };

  // which of the tokens open a run (per <= 64; the same in every wave)
  unsigned long long todo = __ballot(lane < per && opens(first + lane));
  int turn = 0;
  while (todo) {
    const int i = __ffsll(static_cast<long long>(todo)) - 1;
    todo &= todo - 1;
    const int64_t t = first + i;
    const int64_t s = slot_of(t);
    const int64_t page = s >> lg;
    const int n0 = static_cast<int>(s & pmask);
    const int64_t blk = page * H + head;
    const int64_t base = blk * static_cast<int64_t>(P) * DH;
    const int n = run_of(t, s);
    uint8_t* kb = kp.cache + base;
    uint8_t* vb = vp.cache + base;

    if (n <= KA_SHORT && n <= TPW) {
      if ((turn++ & (KA_T / 64 - 1)) != wave) continue;
      const int j = lane / LPT, c = (lane % LPT) * 8;
      float k[8] = {}, v[8] = {};
      if (j < n) {
        load8(ks + (t + j) * kp.tok + c, 8, k);
        load8(vs + (t + j) * vp.tok + c, 8, v);
      }
      uint32_t tk = 0, tv = 0;
      bool bad = false;
      see(k, tk, bad);
      see(v, tv, bad);
      const unsigned long long bads = __ballot(bad);
      const bool poison = ((bads >> (j * LPT)) & ((1ull << LPT) - 1)) != 0;
      float sk = block_scale(wave_max_u(tk)), sv = block_scale(wave_max_u(tv));
      if (n0) {
        const float ok = kp.scale[blk], ov = vp.scale[blk];
        if (sk > ok) move_old<DH, false>(kb, n0, P, ok / sk, lane, 64); else sk = ok;
        if (sv > ov) move_old<DH, true>(vb, n0, P, ov / sv, lane, 64); else sv = ov;
        // the moved words before the new bytes that share them
        __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "workgroup");
      }
      if (lane == 0) {
        kp.scale[blk] = sk;
        vp.scale[blk] = sv;
      }
      if (j < n) {
        const float ik = 1.0f / sk, iv = 1.0f / sv;      // powers of two: exact
        uint32_t w[2];
        w[0] = fp8x4(k[0] * ik, k[1] * ik, k[2] * ik, k[3] * ik);
        w[1] = fp8x4(k[4] * ik, k[5] * ik, k[6] * ik, k[7] * ik);
        if (poison) w[0] = w[1] = FP8_NAN * 0x01010101u;
        __builtin_memcpy(kb + (n0 + j) * DH + c, w, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (mag_bits(v[e]) >= 0x7F800000u) v[e] = 0.0f;
        w[0] = fp8x4(v[0] * iv, v[1] * iv, v[2] * iv, v[3] * iv);
        w[1] = fp8x4(v[4] * iv, v[5] * iv, v[6] * iv, v[7] * iv);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          vb[static_cast<int64_t>(c + e) * P + n0 + j] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
      }
      continue;
    }

    // ---- the workgroup's run: largest magnitudes first, then codes, in
    // pieces of 64 tokens (one piece unless P > 64)
    const int j0 = tid / LPT, c = (tid % LPT) * 8;
    float k[STEPS][8], v[STEPS][8];
    uint32_t tk = 0, tv = 0;
    bool bad[STEPS];
    auto piece = [&](int p0) {
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        const int j = p0 + q * TPG + j0;
        const int64_t m = j < n ? 8 : 0;
        load8(ks + (t + (j < n ? j : 0)) * kp.tok + c, m, k[q]);
        load8(vs + (t + (j < n ? j : 0)) * vp.tok + c, m, v[q]);
      }
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        bad[q] = false;
        see(k[q], tk, bad[q]);
        see(v[q], tv, bad[q]);
      }
    };
    const int pieces = (n + 63) >> 6;
    for (int p = 0; p < pieces; ++p) piece(p * 64);
    tk = wave_max_u(tk);
    tv = wave_max_u(tv);
    if (lane == 0) {
      sh_top[0][wave] = tk;
      sh_top[1][wave] = tv;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < KA_T / 64; ++w) {
      tk = max(tk, sh_top[0][w]);
      tv = max(tv, sh_top[1][w]);
    }
    float sk = block_scale(tk), sv = block_scale(tv);
    if (n0) {
      const float ok = kp.scale[blk], ov = vp.scale[blk];
      if (sk > ok) move_old<DH, false>(kb, n0, P, ok / sk, tid, KA_T); else sk = ok;
      if (sv > ov) move_old<DH, true>(vb, n0, P, ov / sv, tid, KA_T); else sv = ov;
    }
    __syncthreads();                       // old scales read, old codes moved
    if (tid == 0) {
      kp.scale[blk] = sk;
      vp.scale[blk] = sv;
    }
    const float ik = 1.0f / sk, iv = 1.0f / sv;
    for (int p = 0; p < pieces; ++p) {
      const int p0 = p * 64;
      if (pieces > 1) piece(p0);
#pragma unroll
      for (int q = 0; q < STEPS; ++q) {
        const int j = p0 + q * TPG + j0;
        const unsigned long long bads = __ballot(bad[q]);
        const bool poison = ((bads >> ((lane / LPT) * LPT)) & ((1ull << LPT) - 1)) != 0;
        uint32_t w[2];
        w[0] = fp8x4(k[q][0] * ik, k[q][1] * ik, k[q][2] * ik, k[q][3] * ik);
        w[1] = fp8x4(k[q][4] * ik, k[q][5] * ik, k[q][6] * ik, k[q][7] * ik);
        if (poison) w[0] = w[1] = FP8_NAN * 0x01010101u;
        if (j < n) __builtin_memcpy(kb + static_cast<int64_t>(n0 + j) * DH + c, w, 8);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (mag_bits(v[q][e]) >= 0x7F800000u) v[q][e] = 0.0f;
        w[0] = fp8x4(v[q][0] * iv, v[q][1] * iv, v[q][2] * iv, v[q][3] * iv);
        w[1] = fp8x4(v[q][4] * iv, v[q][5] * iv, v[q][6] * iv, v[q][7] * iv);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          vt[(c + e) * VROW + (j - p0)] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
      }
      __syncthreads();
      // rows of V: 64 places of one dimension, from place n0 + p0
      const int m = n - p0 < 64 ? n - p0 : 64;
      uint8_t* out = vb + n0 + p0;
      if (m == 64 && ((n0 + p0) & 7) == 0) {
        for (int i = tid; i < DH * 8; i += KA_T) {
          const int d = i >> 3, o = (i & 7) * 8;
          *reinterpret_cast<uint64_t*>(out + static_cast<int64_t>(d) * P + o) =
              *reinterpret_cast<const uint64_t*>(vt + d * VROW + o);
        }
      } else {
        for (int i = tid; i < DH * m; i += KA_T) {
          const int d = i / m, o = i % m;
          out[static_cast<int64_t>(d) * P + o] = vt[d * VROW + o];
        }
      }
      __syncthreads();
    }
  }
}

// Tokens per workgroup: few, so that single tokens spread over the chip; 64 in
// long calls, where most tokens continue a run and open none.
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
