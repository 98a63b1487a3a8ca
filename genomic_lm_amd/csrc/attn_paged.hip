// attn_paged.hip -- which kernels a call of attention over the paged cache takes
// (attn_paged.hpp): requests of few columns (queries times query heads per K/V
// head) are bound by reading the cache, wider ones by the matrix cores.  The
// lengths are on the device, so each kernel picks its requests there; a call
// that cannot hold wide requests launches only the narrow kernel, and a single
// request goes to the kernel that its largest width asks for.
//
// Up to 16 columns are narrow; in bf16 calls whose widest request has at most
// 32, all are (two sets of 16 per wave): single tokens of 32 query heads on one
// K/V head, or four tokens of 8.  32 columns over 64 x 8192 tokens of 8 K/V
// heads of 128: 142 us there, 214 us as wide units, which are laid out for 128;
// one request of 65536 tokens on one K/V head: 22 against 65 us.  fp32 heads
// of 128 use 253 of 256 registers for one set, so fp32 keeps to 16.  A call that
// holds a wider request keeps to 16 too, so single tokens of 32 heads on one K/V
// head are wide units there.
#include "attn_paged.hpp"

namespace hyena {

struct AttnRoute {
  bool narrow, wide;
  int limit;                 // a request of up to so many columns is narrow
};

static AttnRoute route_of(int64_t R, int64_t max_q, int64_t Hq, int64_t Hkv, bool bf16) {
  AttnRoute r;
  const int64_t cols = max_q * (Hq / Hkv);
  r.limit = bf16 && cols <= AT_NARROW2 ? AT_NARROW2 : AT_NARROW;
  r.wide = cols > r.limit;
  if (r.wide && R == 1) r.limit = 0;
  r.narrow = r.limit > 0;
  return r;
}

static size_t narrow_space_bytes(const AttnRoute& r, int64_t max_q, int64_t Hq, int64_t Hkv, int DH) {
  return r.narrow ? (narrow_bytes(narrow_columns(r.limit, max_q * (Hq / Hkv)), DH) + 15) / 16 * 16 : 0;
}

bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv) {
  // less than 2^32 threads in the largest grid, of either form
  constexpr int64_t most = (int64_t(1) << 32) / 512;
  return attn_wide_grid(R, T, max_q, Hq, Hkv, WideForm{128, 4}) < most && R * Hkv < most;
}

size_t attn_paged_workspace(int64_t R, int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq,
                            int64_t Hkv, int DH) {
  if (short_table(max_pages, page_lg)) return 0;
  size_t most = 0;
  for (bool bf16 : {false, true}) {
    const AttnRoute r = route_of(R, max_q, Hq, Hkv, bf16);
    const WideForm f = wide_form(max_q * (Hq / Hkv), DH, bf16);
    const size_t n = narrow_space_bytes(r, max_q, Hq, Hkv, DH) + (r.wide ? wide_bytes(f.nt, f.waves, DH) : 0);
    most = n > most ? n : most;
  }
  return most;
}

hipError_t launch_attn_paged(const AttnArgs& a) {
  const AttnRoute r = route_of(a.R, a.max_q, a.Hq, a.Hkv, a.bf16);
  const bool split = !short_table(a.max_pages, a.page_lg);
  void* narrow = split && r.narrow ? a.workspace : nullptr;
  void* wide = split && r.wide ? static_cast<char*>(a.workspace) +
                                     narrow_space_bytes(r, a.max_q, a.Hq, a.Hkv, a.DH)
                               : nullptr;
  hipError_t e = hipSuccess;
  if (r.wide) e = launch_attn_wide(a, r.limit, wide);
  if (e == hipSuccess && r.narrow) e = launch_attn_narrow(a, r.limit, narrow);
  if (e == hipSuccess && split) e = launch_attn_join(a, r.limit, narrow, wide);
  return e;
}

}  // namespace hyena
