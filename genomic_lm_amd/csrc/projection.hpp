// projection.hpp -- internal host-side interface between projection_abi.cpp and
// the launchers of the 8-bit projections and their neighbours: the block-scaled
// e4m3 products (linear_tile.hip, linear_few.hip), the quantisation that makes
// their operands (quantize.hip) and the norms of query and key heads with the
// rotation (rope.hip).  Arguments arrive here already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace hyena {

enum Act { ACT_NONE = 0, ACT_GELU = 1, ACT_GELU_TANH = 2, ACT_SILU = 3 };
enum OutKind { OUT_F32 = 0, OUT_BF16 = 1, OUT_FP8 = 2 };

// y = x w0^T + bias, or (gated) act(x w0^T) * (x w1^T); strides in elements.  Weights of no
// columns may be null, the second one of a gated product too.
struct LinearArgs {
  const uint8_t* x;
  int64_t x_stride;
  const float* x_scale;
  int64_t xs_row;             // floats between the scales of two rows
  int xs_run;                 // and of two runs of 128 columns (0: one scale per row)
  const uint8_t* w0;
  const float* s0;
  const uint8_t* w1;
  const float* s1;
  const float* bias;
  bool gated;
  int act;
  void* y;                    // rows of fp32, bf16, or (gated) e4m3
  int64_t y_stride;
  float* q_scale;             // (T, ceil(N / 128)), OUT_FP8 only
  OutKind out;
  int64_t T;
  int N, K;
  hipStream_t stream;
  float* workspace = nullptr;   // (T, N), where linear_workspace asks for it
};
size_t linear_workspace(int64_t T, int64_t N);        // bytes, of OUT_FP8
bool linear_fits(int64_t T, int64_t N);               // whether the launch grid exists
hipError_t launch_linear(const LinearArgs& a);
hipError_t launch_linear_few(const LinearArgs& a);
hipError_t launch_linear_tile(const LinearArgs& a);
bool linear_dma_takes(const LinearArgs& a);            // alignment and strides
hipError_t launch_linear_dma(const LinearArgs& a);

// Codes and scales of T rows: a scale per row (group 0), per 128 columns
// (group 128, block 1) or per 128 rows by 128 columns (block 128).
struct QuantArgs {
  const void* x;
  int64_t x_stride;
  uint8_t* q;
  float* q_scale;
  int group, block;
  int64_t T;
  int D;
  bool bf16;
  hipStream_t stream;
};
hipError_t launch_quantize(const QuantArgs& a);

// Norms of heads and their rotation.  Strides in elements.
struct RopeArgs {
  const void* x[2];           // queries, keys
  int64_t tok[2], head[2];
  void* out[2];
  int64_t out_tok[2], out_head[2];
  const float* weight[2];
  int heads[2];
  const int32_t* positions;
  const float* inv_freq;
  int rotary;                 // columns that turn
  bool interleaved;
  bool norm;
  float eps;
  int64_t T;
  int DH;
  bool bf16;
  hipStream_t stream;
};
hipError_t launch_qk_norm_rope(const RopeArgs& a);

}  // namespace hyena
