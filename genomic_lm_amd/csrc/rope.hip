// rope.hip -- norms of query and key heads with the rotary positions in the
// same pass.
//
// The striped attention blocks turn their queries and keys by position (MHA with
// rotary embedding, base 10000 and 32-fold linear scaling for 262K: Evo2-7B-262K
// model card, Architecture; the frequencies in fp32 and the multiply in fp32:
// Implementation Notes, 'Custom rotary embedding').  Per head of DH columns
//     x' = x / sqrt(mean(x^2) + eps) * w          (where a norm is asked for)
//     a' = a cos f - b sin f,  b' = b cos f + a sin f,   f = position * inv_freq[i],
// for the pairs (a, b) = columns (i, i + R / 2) or (2i, 2i + 1) of the first R.
//
// Bound by memory: 32768 tokens of 32 + 32 heads of 128 201 to 216 us by card, 5.0 to 5.3 TB/s (heads of 80, 40
// turning, whose half is no multiple of 8 and goes element by element, 418, 1.6 TB/s); 16 tokens of
// 32 + 4 heads 6.7 us in a graph, the chain of a position, its angle and its sine.  The angle of
// a position up to 2^31 needs 64 bits, once for all heads of a token.  One copy of the loop
// for queries and keys was slower (251 us).
#include "fp8.hpp"
#include "projection.hpp"

namespace hyena {

template <typename IO, int V>
__device__ __forceinline__ void load_v(const IO* p, int n, float* x) {
  if constexpr (V == 8) {
    float t[8];
    load8(p, n, t);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = t[e];
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) x[e] = e < n ? Io<IO>::ld(p, e) : 0.0f;
  }
}
template <typename IO, int V>
__device__ __forceinline__ void store_v(IO* p, int n, const float* x) {
  if constexpr (V == 8) {
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = x[e];
    store8(p, n, t);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e)
      if (e < n) Io<IO>::st(p, e, x[e]);
  }
}

constexpr int ROPE_MAX_HALF = 128;      // pairs of a head

// Four waves, TB tokens: 4 / TB waves to a token.  A head is taken by LH lanes, each with NI items:
// V pairs, or 2V columns that do not turn; a lane has the same items of every head, so the
// weights and a token's turns stay in its registers.
template <typename IO, int V, int LH, int NI, int TB, bool INTER>
__global__ __launch_bounds__(256, TB == 4 && V == 8 && sizeof(IO) == 2 ? 6 : 1) void qk_norm_rope_kernel(RopeArgs a) {
  __shared__ float2 turn[TB][ROPE_MAX_HALF];
  constexpr int B = TB == 1 ? 2 : 1;                      // heads loaded at once
  constexpr int SLOTS = 256 / TB / LH;                   // heads of a token at a time
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB;
  const int half = a.rotary >> 1, DH = a.DH;
  const int lane = threadIdx.x & (LH - 1);
  const int tok = threadIdx.x / (256 / TB);
  const int slot = threadIdx.x % (256 / TB) / LH;
  const int64_t t = t0 + tok;
  const int pos = t < a.T && a.positions ? a.positions[t] : 0;
  const bool here = t < a.T && pos >= 0;
  const int pairs = half / V;                            // items that turn
  int at[NI][2];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int item = lane + i * LH;
    at[i][0] = item >= pairs ? a.rotary + (item - pairs) * 2 * V : INTER ? item * 2 * V : item * V;
    at[i][1] = item >= pairs || INTER ? at[i][0] + V : at[i][0] + half;
  }
  float v[B][NI][2 * V];
  auto load = [&](int which, int h0) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < B; ++b) {
      const int h = h0 + b * SLOTS;
      if (h >= a.heads[which] || !here) continue;
      const IO* x = static_cast<const IO*>(a.x[which]) + t * a.tok[which] + h * a.head[which];
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        load_v<IO, V>(x + at[i][0], DH - at[i][0], v[b][i]);
        load_v<IO, V>(x + at[i][1], DH - at[i][1], v[b][i] + V);
      }
    }
  };
  load(0, slot);
  float w[NI][2 * V];
  auto load_weight = [&](int which) __attribute__((always_inline)) {
    if (!a.norm) return;
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int e = 0; e < 2 * V; ++e) {
        const int c = at[i][e / V] + e % V;
        w[i][e] = a.weight[which] && c < DH ? a.weight[which][c] : 1.0f;
      }
  };
  load_weight(0);
  for (int i = threadIdx.x; i < TB * half; i += 256) {
    const int k = i / half, p = i - k * half;
    const int at_pos = t0 + k < a.T ? a.positions[t0 + k] : 0;
    // revolutions in 64 bits, their fraction in 32
    const double r = static_cast<double>(at_pos) * static_cast<double>(a.inv_freq[p]) * 0.15915494309189535;
    float s, c;
    sincospif(2.0f * static_cast<float>(r - rint(r)), &s, &c);
    turn[k][p] = make_float2(c, s);
  }
  __syncthreads();
  if (!here) return;                                     // a token's lanes together
  float cs[NI][V], sn[NI][V];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int p = (lane + i * LH) * V + e;
      const float2 f = p < half ? turn[tok][p] : make_float2(1.0f, 0.0f);
      cs[i][e] = f.x;
      sn[i][e] = f.y;
    }

#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (which) load_weight(1);
    for (int h0 = slot; h0 < a.heads[which]; h0 += B * SLOTS) {
      if (which || h0 != slot) load(which, h0);
#pragma unroll
      for (int b = 0; b < B; ++b) {
        const int h = h0 + b * SLOTS;
        if (h >= a.heads[which]) continue;               // LH lanes together
        float(&x)[NI][2 * V] = v[b];
        if (a.norm) {
          float ss = 0.0f;
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) ss = fmaf(x[i][e], x[i][e], ss);
#pragma unroll
          for (int o = 1; o < LH; o <<= 1) ss += __shfl_xor(ss, o);
          // rows whose squares leave fp32 are scaled first, as hyena_add_rmsnorm does
          float unit = 1.0f, eps = a.eps;
          if (!(fmaxf(ss, eps) < 0x1p126f)) unit = 0x1p-96f;
          else if (ss < 0x1p-100f && eps < 0x1p-64f) unit = 0x1p96f;
          if (unit != 1.0f) {
            ss = 0.0f;
#pragma unroll
            for (int i = 0; i < NI; ++i)
#pragma unroll
              for (int e = 0; e < 2 * V; ++e) {
                x[i][e] *= unit;
                ss = fmaf(x[i][e], x[i][e], ss);
              }
#pragma unroll
            for (int o = 1; o < LH; o <<= 1) ss += __shfl_xor(ss, o);
            eps = eps * unit * unit;
          }
          const float inv = rsqrtf(ss / static_cast<float>(DH) + eps);
#pragma unroll
          for (int i = 0; i < NI; ++i)
#pragma unroll
            for (int e = 0; e < 2 * V; ++e) x[i][e] = x[i][e] * inv * w[i][e];
        }
        IO* y = static_cast<IO*>(a.out[which]) + t * a.out_tok[which] + h * a.out_head[which];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (lane + i * LH < pairs) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
              float& p = x[i][INTER ? 2 * e : e];
              float& r = x[i][INTER ? 2 * e + 1 : e + V];
              const float pa = p, ra = r;
              p = fmaf(pa, cs[i][e], -ra * sn[i][e]);
              r = fmaf(ra, cs[i][e], pa * sn[i][e]);
            }
          }
          store_v<IO, V>(y + at[i][0], DH - at[i][0], x[i]);
          store_v<IO, V>(y + at[i][1], DH - at[i][1], x[i] + V);
        }
      }
    }
  }
}

template <typename IO, int V, int LH, int NI>
static void rope_go(const RopeArgs& a) {
  // few tokens: all waves of a workgroup take one
  const bool few = a.T <= 1024;
  auto go = [&](auto kernel) {
    kernel<<<static_cast<unsigned>(few ? a.T : (a.T + 3) / 4), 256, 0, a.stream>>>(a);
  };
  if (a.interleaved) few ? go(qk_norm_rope_kernel<IO, V, LH, NI, 1, true>) : go(qk_norm_rope_kernel<IO, V, LH, NI, 4, true>);
  else few ? go(qk_norm_rope_kernel<IO, V, LH, NI, 1, false>) : go(qk_norm_rope_kernel<IO, V, LH, NI, 4, false>);
}

template <typename IO>
static void rope_heads(const RopeArgs& a) {
  const int half = a.rotary / 2, rest = a.DH - a.rotary;
  auto items = [&](int V) { return half / V + (rest + 2 * V - 1) / (2 * V); };
  if (half % 8 == 0) {
    const int n = items(8);
    if (n <= 4) rope_go<IO, 8, 4, 1>(a);
    else if (n <= 8) rope_go<IO, 8, 8, 1>(a);
    else rope_go<IO, 8, 16, 1>(a);       // ceil(DH / 16) items, at most 16
  } else {
    rope_go<IO, 1, 64, 2>(a);
  }
}

hipError_t launch_qk_norm_rope(const RopeArgs& a) {
  if (a.bf16) rope_heads<bf16_t>(a);
  else rope_heads<float>(a);
  return hipGetLastError();
}

}  // namespace hyena
