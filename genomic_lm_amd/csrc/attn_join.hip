// attn_join.hip -- the pieces of attention units added up (attn_paged.hpp):
//     out = sum_p 2^(m_p - m) O_p / sum_p 2^(m_p - m) l_p,   m = max m_p.
// One launch for what both kernels left: its time is that of a launch and of
// four dependent loads (4 us on an idle chip); the data is small, 6 us for 64
// tokens over 8192 of 8 heads.
#include "attn_paged.hpp"

namespace hyena {

constexpr int AJ_WIDE = 512;               // workgroups that walk the wide units

template <int DH>
struct JoinShared {
  static constexpr int LPC = DH / 4;       // lanes per column, four values each
  static constexpr int SETS = AT_T / LPC;  // columns the workgroup holds at once
  float m[SETS], l[SETS];
  __align__(16) f32x4 o[SETS][LPC];
};

// Columns first, first + step, ... (`count` of them) of a unit.  The sets of
// lanes that they leave over take every other (fourth, ...) piece and are added
// through LDS.
template <typename IO, int DH, typename Slot>
__device__ __forceinline__ void join_columns(const AttnArgs& a, JoinShared<DH>& sh, const float* ml,
                                             const float* part, int nt, int pieces, Slot slot_of,
                                             int first, int step, int count, int tok0, int col0, int head) {
  using S = JoinShared<DH>;
  const int set = threadIdx.x / S::LPC, d = (threadIdx.x % S::LPC) * 4;
  const int group = a.Hq / a.Hkv;
  int lg = 0;                              // log2 of the columns side by side
  while ((1 << lg) < count && (1 << lg) < S::SETS) ++lg;
  const int side = 1 << lg, ways = S::SETS >> lg, way = set >> lg;
  for (int k0 = 0; k0 < count; k0 += side) {
    const int k = k0 + (set & (side - 1));
    const int c = first + k * step;
    float m = AT_NEG, l = 0.0f;
    f32x4 o{0.0f, 0.0f, 0.0f, 0.0f};
    if (k < count) {
#pragma unroll 8
      for (int p = way; p < pieces; p += ways) {
        const int64_t slot = slot_of(p);
        const float pm = ml[(slot * 2) * nt + c], pl = ml[(slot * 2 + 1) * nt + c];
        const f32x4 po = *reinterpret_cast<const f32x4*>(part + (slot * nt + c) * DH + d);
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
        sh.m[set] = m;
        sh.l[set] = l;
      }
      sh.o[set][d >> 2] = o;
      __syncthreads();
      float big = AT_NEG;
      for (int y = 0; y < ways; ++y) big = fmaxf(big, sh.m[(y << lg) + (set & (side - 1))]);
      l = 0.0f;
      o = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      for (int y = 0; y < ways; ++y) {
        const int z = (y << lg) + (set & (side - 1));
        const float f = sh.m[z] == AT_NEG ? 0.0f : __builtin_amdgcn_exp2f(sh.m[z] - big);
        l += f * sh.l[z];
        o += f * sh.o[z][d >> 2];
      }
      __syncthreads();
    }
    if (way == 0 && k < count) {
      const int cc = col0 + c;
      IO* op = static_cast<IO*>(a.out) + ((static_cast<int64_t>(tok0) + cc / group) * a.Hq +
                                          static_cast<int64_t>(head) * group + cc % group) * DH + d;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
      for (int e = 0; e < 4; ++e) Io<IO>::st(op, e, o[e] * inv);
    }
  }
}

// Workgroups [0, wide_groups) walk the wide units, 16 columns at a time, whose
// number only the device knows.  Of the others each belongs to a wave of the
// narrow kernel and to the two units that it may have left in part; the
// workgroups of one unit share its columns, so that few units of many pieces
// still occupy many.
template <typename IO, int DH>
__global__ __launch_bounds__(AT_T) void attn_join_kernel(AttnArgs a, void* narrow, int nt, void* wide,
                                                         WideForm form, int wide_groups) {
  __shared__ JoinShared<DH> sh;
  const int b = static_cast<int>(blockIdx.x);
  if (b < wide_groups) {
    const WideSpace ws = wide_space(wide, form.nt, form.waves);
    const int64_t tasks = static_cast<int64_t>(*ws.used) * (form.nt / 16);
    for (int64_t task = b; task < tasks; task += wide_groups) {
      const int64_t unit = task / (form.nt / 16);
      const int first = static_cast<int>(task % (form.nt / 16)) * 16;
      const AttnUnit u = ws.head[unit];
      auto slot_of = [&](int p) { return u.slot + static_cast<int64_t>(p) * a.Hkv; };
      join_columns<IO, DH>(a, sh, ws.ml, ws.o, form.nt, u.pieces, slot_of, first, 1, min(u.cols - first, 16),
                           u.tok0, u.col0, static_cast<int>(unit % a.Hkv));
    }
    return;
  }
  const NarrowSpace ws = narrow_space(narrow, nt);
  const int w = b - wide_groups;
  const int4 slots[2] = {ws.head[2 * w], ws.head[2 * w + 1]};
#pragma unroll
  for (int z = 1; z >= 0; --z) {
    const int4 h = slots[z];               // first wave, pieces, first query token, head and columns
    // of the unit's waves as many workgroups as give each lane eight pieces, the
    // loads it has in flight
    constexpr int BATCH = 8 * JoinShared<DH>::SETS;
    const int y = w - h.x, cols = h.w >> 16;
    const int n = min(min(h.y, cols), (h.y * cols + BATCH - 1) / BATCH);
    if (y >= n) continue;
    auto slot_of = [&](int p) { return 2 * static_cast<int64_t>(h.x + p) + (p == 0 ? 1 : 0); };
    join_columns<IO, DH>(a, sh, ws.ml, ws.o, nt, h.y, slot_of, y, n, (cols - y + n - 1) / n, h.z, 0,
                         h.w & 0xFFFF);
  }
}

hipError_t launch_attn_join(const AttnArgs& a, int limit, void* narrow, void* wide) {
  const int64_t cols = static_cast<int64_t>(a.max_q) * (a.Hq / a.Hkv);
  const int nt = narrow_columns(limit, cols);
  const int wide_groups = wide ? AJ_WIDE : 0;
  const unsigned grid = wide_groups + (narrow ? AN_WAVES : 0);
  auto go = [&](auto kernel) {
    kernel<<<grid, AT_T, 0, a.stream>>>(a, narrow, nt, wide, wide_form(cols, a.DH, a.bf16),
                                         wide_groups);
  };
  if (a.bf16) {
    if (a.DH == 64) go(attn_join_kernel<bf16_t, 64>); else go(attn_join_kernel<bf16_t, 128>);
  } else {
    if (a.DH == 64) go(attn_join_kernel<float, 64>); else go(attn_join_kernel<float, 128>);
  }
  return hipGetLastError();
}

}  // namespace hyena
