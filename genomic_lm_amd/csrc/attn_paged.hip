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

static size_t narrow_bytes(const AttnRoute& r, int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq,
                           int64_t Hkv, int DH) {
  return r.narrow ? (attn_narrow_workspace(max_pages, page_lg, max_q * (Hq / Hkv), DH) + 15) / 16 * 16 : 0;
}

bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv) {
  return attn_wide_grid(R, T, max_q, Hq, Hkv) < (int64_t(1) << 32) / AT_T;
}

size_t attn_paged_workspace(int64_t R, int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq,
                            int64_t Hkv, int DH) {
  const AttnRoute r = route_of(R, max_q, Hq, Hkv);
  return narrow_bytes(r, max_q, max_pages, page_lg, Hq, Hkv, DH) +
         (r.wide ? attn_wide_workspace(max_pages, page_lg, DH) : 0);
}

hipError_t launch_attn_paged(const AttnArgs& a) {
  const AttnRoute r = route_of(a.R, a.max_q, a.Hq, a.Hkv);
  if (r.wide) {
    const size_t skip = narrow_bytes(r, a.max_q, a.max_pages, a.page_lg, a.Hq, a.Hkv, a.DH);
    const hipError_t e = launch_attn_wide(
        a, r.limit, a.workspace ? static_cast<char*>(a.workspace) + skip : nullptr);
    if (e != hipSuccess) return e;
  }
  return r.narrow ? launch_attn_narrow(a, r.limit, a.workspace) : hipSuccess;
}

}  // namespace hyena
