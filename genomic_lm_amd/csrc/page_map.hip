// page_map.hip -- the page tables and slots of one serving step from request
// lengths.
//
// Request r holds old_lens[r] cached tokens and brings new_lens[r] more; its
// token at position p lives in page block_table[r][p / P] at place p mod P.
//     lens  = old + new,  cu = prefix sums of new
//     need  = pages(lens) - pages(old),  pages(n) = min(ceil(n / P), max_pages)
//     table[r][pages(old) + j] = free[head + (need of earlier requests) + j]
//     slot(t) = page * P + p mod P
// All integers, no atomics: the result does not depend on how work is spread.
//
// The data is small (12 bytes a token), so the cost is the latency of a
// launch; one launch does everything.  The prefix sums over the requests are
// repeated by every workgroup (R loads from L2, one scan) instead of being
// handed from a first launch to a second: the kernel takes 5.6 us for 16 decoding
// requests and 7.7 us for 512 requests with 139701 tokens, so the scan costs
// less than the ~4 us that the shortest dependent launch takes.
#include "serving.hpp"

namespace hyena {

constexpr int PM_T = 256;          // threads
constexpr int PM_TOK = 4;          // tokens per thread

// Sums of non-negative ints stop at 2^31 - 1, so lengths that add up to more
// give counts that no token index reaches instead of negative ones.
__device__ __forceinline__ int add_sat(int a, int b) {
  const uint32_t s = static_cast<uint32_t>(a) + static_cast<uint32_t>(b);
  return static_cast<int>(s < 0x7FFFFFFFu ? s : 0x7FFFFFFFu);
}

// Inclusive scan over the wave.
__device__ __forceinline__ int wave_scan(int x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int y = __shfl_up(x, o);
    if (lane >= o) x = add_sat(x, y);
  }
  return x;
}

__global__ __launch_bounds__(PM_T) void page_map_kernel(
    const int32_t* __restrict__ old_lens, const int32_t* __restrict__ new_lens, int R,
    int32_t* block_table, int64_t table_stride, int max_pages,
    const int32_t* __restrict__ free_pages, int num_free, const int32_t* __restrict__ free_head,
    int lg, int32_t* __restrict__ cu, int32_t* __restrict__ lens, int32_t* __restrict__ positions,
    int64_t* __restrict__ slots, int T, int32_t* __restrict__ status) {
  extern __shared__ int sm[];
  int* s_cu = sm;                  // R + 1: first token of each request
  int* s_need = sm + R + 1;        // R: pages taken by earlier requests
  int* s_part = s_need + R;        // 12: wave totals of the two scans and of the unplaced tokens
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int head = free_head ? max(*free_head, 0) : 0;
  const int mask = (1 << lg) - 1;
  auto pages = [&](int n) {        // whole pages of n tokens, within the table
    const int p = static_cast<int>((static_cast<int64_t>(n) + mask) >> lg);
    return min(p, max_pages);
  };

  auto cached = [&](int r) { return max(old_lens[r], 0); };
  auto brings = [&](int r, int o) { return min(max(new_lens[r], 0), 0x7FFFFFFF - o); };

  // the page that request r's first new token shares with its last cached one, -1
  // if the table holds none (an earlier step found no page for it); 0 if it begins one
  auto shared_page = [&](int r, int o) {
    const int j = o >> lg;
    return (o & mask) && j < max_pages ? block_table[r * table_stride + j] : 0;
  };

  // every thread sums its run of requests, then a scan over the threads
  const int run = (R + PM_T - 1) / PM_T;
  const int r0 = min(tid * run, R), r1 = min(r0 + run, R);
  int tok = 0, need = 0;
  for (int r = r0; r < r1; ++r) {
    const int o = cached(r), n = brings(r, o);
    tok = add_sat(tok, n);
    need = add_sat(need, pages(o + n) - pages(o));
  }
  const int tok_in = wave_scan(tok), need_in = wave_scan(need);
  if (lane == 63) {
    s_part[wave] = tok_in;
    s_part[4 + wave] = need_in;
  }
  __syncthreads();
  // sums over the threads before this one: the lane below's in this wave, and
  // the waves below
  int a = __shfl_up(tok_in, 1), b = __shfl_up(need_in, 1), total = 0, all_need = 0;
  if (lane == 0) a = b = 0;
#pragma unroll
  for (int w = 0; w < PM_T / 64; ++w) {
    if (w < wave) {
      a = add_sat(a, s_part[w]);
      b = add_sat(b, s_part[4 + w]);
    }
    total = add_sat(total, s_part[w]);
    all_need = add_sat(all_need, s_part[4 + w]);
  }
  const bool first = blockIdx.x == 0;
  int unplaced = 0;
  for (int r = r0; r < r1; ++r) {
    const int o = cached(r), n = brings(r, o);
    const int have = pages(o), want = pages(o + n);
    s_cu[r] = a;
    s_need[r] = b;
    if (first) {
      cu[r] = a;
      lens[r] = o + n;
      // tokens past the pages this request gets
      const int64_t left = static_cast<int64_t>(num_free) - head - b;
      const int got = static_cast<int>(left < 0 ? 0 : left < want - have ? left : want - have);
      const int64_t room = static_cast<int64_t>(have + got) << lg;
      const int64_t from = room > o ? room : o;
      if (o + n > from) unplaced = add_sat(unplaced, static_cast<int>(o + n - from));
      if (n > 0 && shared_page(r, o) < 0) unplaced = add_sat(unplaced, min(n, mask + 1 - (o & mask)));
    }
    a = add_sat(a, n);
    b = add_sat(b, want - have);
  }
  if (tid == 0) s_cu[R] = total;
  if (first) {
    if (tid == 0) cu[R] = total;
    const int u = wave_scan(unplaced);
    if (lane == 63) s_part[8 + wave] = u;
  }
  __syncthreads();
  if (first && tid == 0) {
    const int64_t end = static_cast<int64_t>(head) + all_need;
    status[0] = static_cast<int>(end < num_free ? end : max(num_free, head));
    status[1] = add_sat(add_sat(s_part[8], s_part[9]), add_sat(s_part[10], s_part[11]));
  }

  // new table entries: one wave per request, requests dealt over the grid
  for (int r = static_cast<int>(blockIdx.x) * (PM_T / 64) + wave; r < R; r += gridDim.x * (PM_T / 64)) {
    const int o = cached(r), n = brings(r, o);
    const int have = pages(o), want = pages(o + n);
    const int64_t at = static_cast<int64_t>(head) + s_need[r];
    for (int j = lane; j < want - have; j += 64)
      if (at + j < num_free) block_table[r * table_stride + have + j] = free_pages[at + j];
  }

  // slots: entries that the table already held are read from it, new ones from
  // the free list (the table's own new entries belong to other workgroups)
  const int t0 = (static_cast<int>(blockIdx.x) * PM_T + tid) * PM_TOK;
  if (t0 >= T) return;
  int r = 0;
  if (t0 < total) {                // the last request that starts at or before t0
    int lo = 0, hi = R - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s_cu[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    r = lo;
  }
#pragma unroll
  for (int i = 0; i < PM_TOK; ++i) {
    const int t = t0 + i;
    if (t >= T) break;
    int pos = -1;
    int64_t slot = -1;
    if (t < total) {
      while (t >= s_cu[r + 1]) ++r;    // ends: t < total = s_cu[R]
      const int o = cached(r);
      pos = o + (t - s_cu[r]);
      const int j = pos >> lg, have = pages(o);
      int page = -1;
      if (j < have) {
        page = block_table[r * table_stride + j];
      } else if (j < max_pages) {
        const int64_t at = static_cast<int64_t>(head) + s_need[r] + (j - have);
        if (at < num_free) page = free_pages[at];
      }
      if (page >= 0) slot = (static_cast<int64_t>(page) << lg) | (pos & mask);
    }
    if (positions) positions[t] = pos;
    slots[t] = slot;
  }
}

hipError_t launch_page_map(const PageMapArgs& a) {
  const int per = PM_T * PM_TOK;
  const unsigned grid = a.T > 0 ? static_cast<unsigned>((static_cast<int64_t>(a.T) + per - 1) / per) : 1u;
  const size_t shmem = (2 * static_cast<size_t>(a.R) + 1 + 12) * sizeof(int);
  page_map_kernel<<<grid, PM_T, shmem, a.stream>>>(
      a.old_lens, a.new_lens, a.R, a.block_table, a.table_stride, a.max_pages, a.free_pages,
      a.num_free, a.free_head, a.page_lg, a.cu, a.lens, a.positions, a.slots, a.T, a.status);
  return hipGetLastError();
}

}  // namespace hyena
