// attn_paged.hip -- which kernels a call of attention over the paged cache takes
// (attn_paged.hpp): requests of up to AT_NARROW columns (queries times query
// heads per K/V head) are bound by reading the cache, wider ones by the matrix
// cores.  The lengths are on the device, so each kernel picks its requests
// there; a call that cannot hold wide requests launches only the narrow one,
// and a single request goes to the kernel that its largest width asks for.
#include "attn_paged.hpp"

namespace hyena {

struct AttnRoute {
  bool narrow, wide;
  int limit;                 // a request of up to so many columns is narrow
};

static AttnRoute route_of(int64_t R, int64_t max_q, int64_t Hq, int64_t Hkv) {
  AttnRoute r;
  r.wide = max_q * (Hq / Hkv) > AT_NARROW;
  r.limit = r.wide && R == 1 ? 0 : AT_NARROW;
  r.narrow = r.limit > 0;
  return r;
}

static size_t narrow_space_bytes(const AttnRoute& r, int64_t max_q, int64_t Hq, int64_t Hkv, int DH) {
  const int64_t cols = max_q * (Hq / Hkv);
  return r.narrow ? (narrow_bytes(cols < AT_NARROW ? cols : AT_NARROW, DH) + 15) / 16 * 16 : 0;
}

bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv) {
  // less than 2^32 threads in the largest grid, of either form
  constexpr int64_t most = (int64_t(1) << 32) / 512;
  return attn_wide_grid(R, T, max_q, Hq, Hkv, WideForm{128, 4}) < most && R * Hkv < most;
}

size_t attn_paged_workspace(int64_t R, int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq,
                            int64_t Hkv, int DH) {
  if (short_table(max_pages, page_lg)) return 0;
  const AttnRoute r = route_of(R, max_q, Hq, Hkv);
  size_t wide = 0;
  for (bool bf16 : {false, true}) {
    const WideForm f = wide_form(max_q * (Hq / Hkv), DH, bf16);
    const size_t n = wide_bytes(f.nt, f.waves, DH);
    wide = r.wide && n > wide ? n : wide;
  }
  return narrow_space_bytes(r, max_q, Hq, Hkv, DH) + wide;
}

hipError_t launch_attn_paged(const AttnArgs& a) {
  const AttnRoute r = route_of(a.R, a.max_q, a.Hq, a.Hkv);
  const bool split = !short_table(a.max_pages, a.page_lg);
  void* narrow = split && r.narrow ? a.workspace : nullptr;
  void* wide = split && r.wide ? static_cast<char*>(a.workspace) +
                                     narrow_space_bytes(r, a.max_q, a.Hq, a.Hkv, a.DH)
                               : nullptr;
  hipError_t e = hipSuccess;
  if (r.wide) e = launch_attn_wide(a, r.limit, wide);
  if (e == hipSuccess && r.narrow) e = launch_attn_narrow(a, r.limit, narrow);
  if (e == hipSuccess && split) e = launch_attn_join(a, narrow, wide);
  return e;
}

}  // namespace hyena
