// serving.hpp -- internal host-side interface between serving_abi.cpp and the
// launchers of the serving kernels.  Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hyena {

// Residual addition and root-mean-square norm of T rows (norm.hip).  Strides
// are in elements between rows.  q / q_scale set: 8-bit output, group 0 (one
// scale per row) or the number of columns that share a scale; else y.
struct NormArgs {
  const void* x;
  int64_t x_stride;
  const void* residual;
  int64_t residual_stride;
  const float* weight;
  float eps;
  void* y;
  int64_t y_stride;
  uint8_t* q;
  float* q_scale;
  int group;
  void* residual_out;
  int64_t residual_out_stride;
  int64_t T;
  int D;
  bool bf16;
  hipStream_t stream;
};
hipError_t launch_add_rmsnorm(const NormArgs& a);

// Page tables and slots of one step (page_map.hip).
struct PageMapArgs {
  const int32_t* old_lens;
  const int32_t* new_lens;
  int R;
  int32_t* block_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* free_pages;
  int num_free;
  const int32_t* free_head;
  int page_lg;
  int32_t* cu;
  int32_t* lens;
  int32_t* positions;
  int64_t* slots;
  int T;
  int32_t* status;
  hipStream_t stream;
};
hipError_t launch_page_map(const PageMapArgs& a);

// New K and V rows into the 8-bit cache (kv_append.hip).  Strides in elements.
struct KvAppendArgs {
  const void* k;
  const void* v;
  int64_t k_tok, k_head, v_tok, v_head;
  const int64_t* slots;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;
  float* v_scale;
  int64_t num_pages;
  int page_lg;
  int T, H, DH;
  bool bf16;
  hipStream_t stream;
};
bool kv_append_fits(int64_t T, int64_t H);      // whether the launch grid exists
hipError_t launch_kv_append(const KvAppendArgs& a);

// Attention over the 8-bit cache (attn_paged.hip).  Strides in elements.
struct AttnArgs {
  const void* q;
  int64_t q_tok, q_head;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;
  const float* v_scale;
  int64_t num_pages;
  int page_lg;
  const int32_t* block_table;
  int64_t table_stride;
  int max_pages;
  const int32_t* lens;
  const int32_t* cu;
  int R, T, max_q, Hq, Hkv, DH;
  float scale;
  void* out;
  bool bf16;
  void* workspace;
  hipStream_t stream;
};
// Whether the launch grids of the shape exist, and the workspace it needs.
bool attn_paged_fits(int64_t R, int64_t T, int64_t max_q, int64_t Hq, int64_t Hkv);
size_t attn_paged_workspace(int64_t R, int64_t max_q, int64_t max_pages, int page_lg, int64_t Hq,
                            int64_t Hkv, int DH);
hipError_t launch_attn_paged(const AttnArgs& a);

}  // namespace hyena
