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

// TB tokens per workgroup.  A head is taken by LH lanes, each with NI items: V
// pairs, or 2V columns that do not turn.
template <typename IO, int V, int LH, int NI, int TB>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(RopeArgs a) {
  __shared__ float2 turn[TB][ROPE_MAX_HALF];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * TB;
  const int half = a.rotary >> 1;
  for (int i = threadIdx.x; i < TB * half; i += 256) {
    const int tok = i / half, p = i - tok * half;
    const int64_t t = t0 + tok;
    const int pos = t < a.T ? a.positions[t] : 0;
    // revolutions in 64 bits, their fraction in 32
    const double r = static_cast<double>(pos) * static_cast<double>(a.inv_freq[p]) * 0.15915494309189535;
    float s, c;
    sincospif(2.0f * static_cast<float>(r - rint(r)), &s, &c);
    turn[tok][p] = make_float2(c, s);
  }
  __syncthreads();
  const int lane = threadIdx.x & (LH - 1);
  const int heads = a.heads[0] + a.heads[1];
  const int pairs = half / V;                            // items that turn
  const int DH = a.DH;
  for (int u = threadIdx.x / LH; u < TB * heads; u += 256 / LH) {
    const int tok = u / heads, head = u - tok * heads;
    const int64_t t = t0 + tok;
    if (t >= a.T) break;                                 // LH lanes together
    if (a.positions && a.positions[t] < 0) continue;
    const int which = head >= a.heads[0];
    const int h = head - (which ? a.heads[0] : 0);
    const IO* x = static_cast<const IO*>(a.x[which]) + t * a.tok[which] + h * a.head[which];
    float v[NI][2 * V];
    int at[NI][2];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int item = lane + i * LH;
      if (item < pairs) {
        at[i][0] = a.interleaved ? item * 2 * V : item * V;
        at[i][1] = a.interleaved ? item * 2 * V + V : item * V + half;
      } else {
        at[i][0] = a.rotary + (item - pairs) * 2 * V;
        at[i][1] = at[i][0] + V;
      }
      load_v<IO, V>(x + at[i][0], DH - at[i][0], v[i]);
      load_v<IO, V>(x + at[i][1], DH - at[i][1], v[i] + V);
    }
    if (a.norm) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) ss = fmaf(v[i][e], v[i][e], ss);
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
            v[i][e] *= unit;
            ss = fmaf(v[i][e], v[i][e], ss);
          }
#pragma unroll
        for (int o = 1; o < LH; o <<= 1) ss += __shfl_xor(ss, o);
        eps = eps * unit * unit;
      }
      const float inv = rsqrtf(ss / static_cast<float>(DH) + eps);
      const float* w = a.weight[which];
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int e = 0; e < 2 * V; ++e) {
          const int c = at[i][e / V] + e % V;
          v[i][e] = v[i][e] * inv * (w && c < DH ? w[c] : 1.0f);
        }
    }
    IO* y = static_cast<IO*>(a.out[which]) + t * a.out_tok[which] + h * a.out_head[which];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int item = lane + i * LH;
      if (item < pairs) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float2 f = turn[tok][item * V + e];
          float& p = a.interleaved ? v[i][2 * e] : v[i][e];
          float& r = a.interleaved ? v[i][2 * e + 1] : v[i][e + V];
          const float pa = p, ra = r;
          p = fmaf(pa, f.x, -ra * f.y);
          r = fmaf(ra, f.x, pa * f.y);
        }
      }
      store_v<IO, V>(y + at[i][0], DH - at[i][0], v[i]);
      store_v<IO, V>(y + at[i][1], DH - at[i][1], v[i] + V);
    }
  }
}

template <typename IO, int V, int LH, int NI>
static void rope_go(const RopeArgs& a) {
  // few tokens: one per workgroup
  if (a.T <= 1024) {
    qk_norm_rope_kernel<IO, V, LH, NI, 1><<<static_cast<unsigned>(a.T), 256, 0, a.stream>>>(a);
  } else {
    constexpr int TB = 4;
    qk_norm_rope_kernel<IO, V, LH, NI, TB><<<static_cast<unsigned>((a.T + TB - 1) / TB), 256, 0, a.stream>>>(a);
  }
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
