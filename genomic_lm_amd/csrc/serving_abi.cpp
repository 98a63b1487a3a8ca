// serving_abi.cpp -- the extern "C" entry points of the serving operators
// declared in include/hyena.h: host validation, then a launcher (serving.hpp).
// Nothing here allocates, prints, throws or synchronises.
#include "hyena.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <limits>

#include "launch.hpp"
#include "serving.hpp"

namespace {

using hyena::aligned_to;

constexpr int64_t kMaxInt = std::numeric_limits<int>::max();
constexpr int64_t kMaxI64 = std::numeric_limits<int64_t>::max();

hyena_status_t from_hip(hipError_t e) { return e == hipSuccess ? HYENA_OK : HYENA_ERR_LAUNCH; }

bool valid_io(hyena_dtype_t io) { return io == HYENA_F32 || io == HYENA_BF16; }
size_t io_size(hyena_dtype_t io) { return io == HYENA_BF16 ? 2 : 4; }

// log2 of a page size, -1 if it is no power of two, -2 if it is out of range
int page_lg(int64_t page_size) {
  if (page_size < 1 || (page_size & (page_size - 1))) return -1;
  if (page_size < HYENA_MIN_PAGE || page_size > HYENA_MAX_PAGE) return -2;
  int lg = 0;
  while ((int64_t(1) << lg) < page_size) ++lg;
  return lg;
}

// a * b <= INT64_MAX for non-negative a, b
bool fits(int64_t a, int64_t b) { return b == 0 || a <= kMaxI64 / b; }

hyena_status_t norm_impl(const void* x, int64_t x_stride, const void* residual,
                         int64_t residual_stride, const float* weight, float eps, void* y,
                         int64_t y_stride, uint8_t* q, float* q_scale, int64_t group,
                         void* residual_out, int64_t residual_out_stride, int64_t T, int64_t D,
                         hyena_dtype_t io, bool fp8, hipStream_t stream) {
  if (!valid_io(io) || T < 0 || D < 0 || !(eps >= 0.0f) || std::isinf(eps)) return HYENA_ERR_INVALID_ARG;
  if (fp8 && group != 0 && group != HYENA_NORM_GROUP) return HYENA_ERR_INVALID_ARG;
  if (x_stride < 0 || residual_stride < 0 || y_stride < 0 || residual_out_stride < 0)
    return HYENA_ERR_INVALID_ARG;
  if (T == 0 || D == 0) return HYENA_OK;
  if (!x || (fp8 ? (!q || !q_scale) : !y) || (residual_out && !residual)) return HYENA_ERR_INVALID_ARG;
  // rows that are written must not overlap
  if (T > 1 && ((!fp8 && y_stride < D) || (residual_out && residual_out_stride < D)))
    return HYENA_ERR_INVALID_ARG;
  const size_t a = io_size(io);
  if (!aligned_to(x, a) || (residual && !aligned_to(residual, a)) || (weight && !aligned_to(weight, 4)) ||
      (y && !aligned_to(y, a)) || (q_scale && !aligned_to(q_scale, 4)) ||
      (residual_out && !aligned_to(residual_out, a)))
    return HYENA_ERR_INVALID_ARG;
  if (D > HYENA_MAX_NORM_DIM) return HYENA_ERR_UNSUPPORTED;
  const int64_t top = kMaxI64 / 8;
  if (T > top / D || T > top / (x_stride + 1) || T > top / (residual_stride + 1) ||
      T > top / (y_stride + 1) || T > top / (residual_out_stride + 1))
    return HYENA_ERR_UNSUPPORTED;
  hyena::NormArgs n{x, x_stride, residual, residual_stride, weight, eps, y, y_stride, q, q_scale,
                    static_cast<int>(group), residual_out, residual_out_stride, T,
                    static_cast<int>(D), io == HYENA_BF16, stream};
  return from_hip(hyena::launch_add_rmsnorm(n));
}

}  // namespace

extern "C" {

hyena_status_t hyena_add_rmsnorm(const void* x, int64_t x_stride, const void* residual,
                                 int64_t residual_stride, const float* weight, float eps, void* y,
                                 int64_t y_stride, void* residual_out,
                                 int64_t residual_out_stride, int64_t T, int64_t D,
                                 hyena_dtype_t io, hipStream_t stream) {
  return norm_impl(x, x_stride, residual, residual_stride, weight, eps, y, y_stride, nullptr,
                   nullptr, 0, residual_out, residual_out_stride, T, D, io, false, stream);
}

hyena_status_t hyena_add_rmsnorm_fp8(const void* x, int64_t x_stride, const void* residual,
                                     int64_t residual_stride, const float* weight, float eps,
                                     uint8_t* q, float* q_scale, int64_t group,
                                     void* residual_out, int64_t residual_out_stride, int64_t T,
                                     int64_t D, hyena_dtype_t io, hipStream_t stream) {
  return norm_impl(x, x_stride, residual, residual_stride, weight, eps, nullptr, 0, q, q_scale,
                   group, residual_out, residual_out_stride, T, D, io, true, stream);
}

hyena_status_t hyena_page_map(const int32_t* old_lens, const int32_t* new_lens, int64_t R,
                              int32_t* block_table, int64_t table_stride, int64_t max_pages,
                              const int32_t* free_pages, int64_t num_free,
                              const int32_t* free_head, int64_t page_size, int32_t* cu,
                              int32_t* lens, int32_t* positions, int64_t* slots, int64_t T,
                              int32_t* status, hipStream_t stream) {
  if (R < 0 || T < 0 || max_pages < 0 || num_free < 0 || table_stride < max_pages)
    return HYENA_ERR_INVALID_ARG;
  const int lg = page_lg(page_size);
  if (lg == -1) return HYENA_ERR_INVALID_ARG;
  if (!cu || !status || (R > 0 && (!old_lens || !new_lens || !lens)) || (T > 0 && !slots) ||
      (R > 0 && max_pages > 0 && !block_table) || (num_free > 0 && !free_pages))
    return HYENA_ERR_INVALID_ARG;
  if (!aligned_to(old_lens, 4) || !aligned_to(new_lens, 4) || !aligned_to(block_table, 4) ||
      !aligned_to(free_pages, 4) || !aligned_to(free_head, 4) || !aligned_to(cu, 4) ||
      !aligned_to(lens, 4) || !aligned_to(positions, 4) || !aligned_to(slots, 8) ||
      !aligned_to(status, 4))
    return HYENA_ERR_INVALID_ARG;
  if (lg < 0 || R > HYENA_MAX_REQUESTS || T > kMaxInt - 1024 || num_free > kMaxInt ||
      max_pages > (kMaxInt >> lg) || !fits(table_stride, 4 * R))
    return HYENA_ERR_UNSUPPORTED;
  hyena::PageMapArgs a{old_lens, new_lens, static_cast<int>(R), block_table, table_stride,
                       static_cast<int>(max_pages), free_pages, static_cast<int>(num_free),
                       free_head, lg, cu, lens, positions, slots, static_cast<int>(T), status,
                       stream};
  return from_hip(hyena::launch_page_map(a));
}

// The shape of a cache, shared by the two entries that take one.
static hyena_status_t check_cache(const uint8_t* k_cache, const uint8_t* v_cache,
                                  const float* k_scale, const float* v_scale, int64_t num_pages,
                                  int lg, int64_t H, int64_t DH) {
  if (!k_cache || !v_cache || !k_scale || !v_scale || num_pages < 1) return HYENA_ERR_INVALID_ARG;
  if (!aligned_to(k_cache, 16) || !aligned_to(v_cache, 16) || !aligned_to(k_scale, 4) ||
      !aligned_to(v_scale, 4))
    return HYENA_ERR_INVALID_ARG;
  if (num_pages > kMaxInt || !fits(num_pages, (H << lg) * DH)) return HYENA_ERR_UNSUPPORTED;
  return HYENA_OK;
}

hyena_status_t hyena_kv_append_fp8(const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                                   const void* v, int64_t v_tok_stride, int64_t v_head_stride,
                                   const int64_t* slots, uint8_t* k_cache, uint8_t* v_cache,
                                   float* k_scale, float* v_scale, int64_t num_pages,
                                   int64_t page_size, int64_t T, int64_t H, int64_t DH,
                                   hyena_dtype_t io, hipStream_t stream) {
  const int lg = page_lg(page_size);
  if (!valid_io(io) || T < 0 || H < 0 || DH < 0 || lg == -1) return HYENA_ERR_INVALID_ARG;
  if (k_tok_stride < 0 || k_head_stride < 0 || v_tok_stride < 0 || v_head_stride < 0)
    return HYENA_ERR_INVALID_ARG;
  if (lg < 0 || (DH != 64 && DH != 128) || H > HYENA_MAX_HEADS || T > kMaxInt)
    return HYENA_ERR_UNSUPPORTED;
  if (T == 0 || H == 0) return HYENA_OK;
  const size_t a = io_size(io);
  if (!k || !v || !slots || !aligned_to(k, a) || !aligned_to(v, a) || !aligned_to(slots, 8))
    return HYENA_ERR_INVALID_ARG;
  const hyena_status_t st = check_cache(k_cache, v_cache, k_scale, v_scale, num_pages, lg, H, DH);
  if (st != HYENA_OK) return st;
  // a workgroup per token group and head, less than 2^32 threads
  const int64_t most = kMaxI64 / 64;
  if (k_tok_stride > most / T || v_tok_stride > most / T || k_head_stride > most / H ||
      v_head_stride > most / H || !hyena::kv_append_fits(T, H))
    return HYENA_ERR_UNSUPPORTED;
  hyena::KvAppendArgs n{k, v, k_tok_stride, k_head_stride, v_tok_stride, v_head_stride, slots,
                        k_cache, v_cache, k_scale, v_scale, num_pages, lg, static_cast<int>(T),
                        static_cast<int>(H), static_cast<int>(DH), io == HYENA_BF16, stream};
  return from_hip(hyena::launch_kv_append(n));
}

// Sizes of an attention call that do not depend on its pointers.
static hyena_status_t check_attn(int64_t R, int64_t T, int64_t max_q, int64_t max_pages, int lg,
                                 int64_t Hq, int64_t Hkv, int64_t DH) {
  if (R < 0 || T < 0 || max_q < 0 || max_pages < 0 || Hq < 0 || Hkv < 1 || Hq % Hkv || DH < 0 || lg == -1)
    return HYENA_ERR_INVALID_ARG;
  if (lg < 0 || (DH != 64 && DH != 128) || R > HYENA_MAX_REQUESTS || Hq > HYENA_MAX_HEADS ||
      T > kMaxInt || max_q > kMaxInt || max_pages > ((kMaxInt - 1024) >> lg) ||
      (Hq > 0 && !hyena::attn_paged_fits(R, T, max_q, Hq, Hkv)))
    return HYENA_ERR_UNSUPPORTED;
  return HYENA_OK;
}

hyena_status_t hyena_attn_paged_fp8(const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                                    const uint8_t* k_cache, const uint8_t* v_cache,
                                    const float* k_scale, const float* v_scale, int64_t num_pages,
                                    int64_t page_size, const int32_t* block_table,
                                    int64_t table_stride, int64_t max_pages, const int32_t* lens,
                                    const int32_t* cu, int64_t R, int64_t T, int64_t max_q,
                                    int64_t Hq, int64_t Hkv, int64_t DH, float scale, void* out,
                                    hyena_dtype_t io, void* workspace, size_t ws_bytes,
                                    hipStream_t stream) {
  const int lg = page_lg(page_size);
  if (!valid_io(io) || !std::isfinite(scale) || q_tok_stride < 0 || q_head_stride < 0 ||
      table_stride < max_pages)
    return HYENA_ERR_INVALID_ARG;
  hyena_status_t st = check_attn(R, T, max_q, max_pages, lg, Hq, Hkv, DH);
  if (st != HYENA_OK) return st;
  if (R == 0 || T == 0 || max_q == 0 || Hq == 0) return HYENA_OK;
  const size_t a = io_size(io);
  if (!q || !out || !lens || !cu || (max_pages > 0 && !block_table)) return HYENA_ERR_INVALID_ARG;
  if (!aligned_to(q, a) || !aligned_to(out, a) || !aligned_to(lens, 4) || !aligned_to(cu, 4) ||
      !aligned_to(block_table, 4))
    return HYENA_ERR_INVALID_ARG;
  st = check_cache(k_cache, v_cache, k_scale, v_scale, num_pages, lg, Hkv, DH);
  if (st != HYENA_OK) return st;
  const int64_t most = kMaxI64 / 64;
  if (q_tok_stride > most / T || q_head_stride > most / Hq || !fits(T, Hq * DH * 4) ||
      !fits(table_stride, 4 * R))
    return HYENA_ERR_UNSUPPORTED;
  const size_t need = hyena::attn_paged_workspace(R, max_q, max_pages, lg, Hq, Hkv, static_cast<int>(DH));
  if (need > 0 && (!workspace || ws_bytes < need || !aligned_to(workspace, 16)))
    return HYENA_ERR_WORKSPACE;
  hyena::AttnArgs n{q, q_tok_stride, q_head_stride, k_cache, v_cache, k_scale, v_scale, num_pages,
                    lg, block_table, table_stride, static_cast<int>(max_pages), lens, cu,
                    static_cast<int>(R), static_cast<int>(T), static_cast<int>(max_q),
                    static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(DH), scale, out,
                    io == HYENA_BF16, workspace, stream};
  return from_hip(hyena::launch_attn_paged(n));
}

size_t hyena_attn_paged_workspace_size(int64_t R, int64_t T, int64_t max_q, int64_t max_pages,
                                       int64_t page_size, int64_t Hq, int64_t Hkv, int64_t DH) {
  const int lg = page_lg(page_size);
  if (check_attn(R, T, max_q, max_pages, lg, Hq, Hkv, DH) != HYENA_OK) return 0;
  if (R == 0 || T == 0 || max_q == 0 || Hq == 0) return 0;
  return hyena::attn_paged_workspace(R, max_q, max_pages, lg, Hq, Hkv, static_cast<int>(DH));
}

}  // extern "C"
