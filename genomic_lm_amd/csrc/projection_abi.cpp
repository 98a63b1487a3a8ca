// projection_abi.cpp -- the extern "C" entry points of the 8-bit projections, the
// quantisation of their operands and the rotary positions declared in
// include/hyena.h: host validation, then a launcher (projection.hpp).  Nothing
// here allocates, prints, throws or synchronises.
#include "hyena.h"

#include <hip/hip_runtime.h>

#include <cmath>
#include <limits>

#include "launch.hpp"
#include "projection.hpp"

namespace {

using hyena::aligned_to;

constexpr int64_t kMaxInt = std::numeric_limits<int>::max();
constexpr int64_t kMost = std::numeric_limits<int64_t>::max() / 64;

hyena_status_t from_hip(hipError_t e) { return e == hipSuccess ? HYENA_OK : HYENA_ERR_LAUNCH; }
bool valid_io(hyena_dtype_t io) { return io == HYENA_F32 || io == HYENA_BF16; }
size_t io_size(hyena_dtype_t io) { return io == HYENA_BF16 ? 2 : 4; }

// Sizes, pointers and strides of a product.
hyena_status_t linear_impl(const hyena::LinearArgs& a, int64_t N, int64_t K, int64_t x_group,
                           size_t ws_bytes = 0) {
  if (a.T < 0 || N < 0 || K < 0 || a.x_stride < 0 || a.xs_row < 0 || a.y_stride < 0 ||
      (x_group != 0 && x_group != HYENA_NORM_GROUP))
    return HYENA_ERR_INVALID_ARG;
  if (a.T == 0 || N == 0) return HYENA_OK;
  if (!a.y || (a.out == hyena::OUT_FP8 && !a.q_scale) ||
      (K > 0 && (!a.x || !a.x_scale || !a.w0 || !a.s0 || (a.gated && (!a.w1 || !a.s1)))))
    return HYENA_ERR_INVALID_ARG;
  if (a.T > 1 && a.y_stride < N) return HYENA_ERR_INVALID_ARG;
  const size_t align = a.out == hyena::OUT_FP8 ? 1 : a.out == hyena::OUT_BF16 ? 2 : 4;
  if (!aligned_to(a.y, align) || !aligned_to(a.x_scale, 4) || !aligned_to(a.s0, 4) || !aligned_to(a.s1, 4) ||
      !aligned_to(a.bias, 4) || !aligned_to(a.q_scale, 4))
    return HYENA_ERR_INVALID_ARG;
  if (N > HYENA_MAX_PROJ_DIM || K > HYENA_MAX_PROJ_DIM || a.T > kMaxInt || a.x_stride > kMost / a.T ||
      a.xs_row > kMost / a.T || a.y_stride > kMost / a.T || !hyena::linear_fits(a.T, N))
    return HYENA_ERR_UNSUPPORTED;
  if (a.out == hyena::OUT_FP8) {
    const size_t need = hyena::linear_workspace(a.T, N);
    if (need && (!a.workspace || ws_bytes < need || !aligned_to(a.workspace, 16))) return HYENA_ERR_WORKSPACE;
  }
  hyena::LinearArgs b = a;
  b.N = static_cast<int>(N);
  b.K = static_cast<int>(K);
  b.xs_run = x_group ? 1 : 0;
  return from_hip(hyena::launch_linear(b));
}

hyena_status_t quantize_impl(const void* x, int64_t x_stride, uint8_t* q, float* q_scale, int64_t group,
                             int block, int64_t T, int64_t D, hyena_dtype_t io, hipStream_t stream) {
  if (!valid_io(io) || T < 0 || D < 0 || x_stride < 0 || (group != 0 && group != HYENA_NORM_GROUP))
    return HYENA_ERR_INVALID_ARG;
  if (T == 0 || (D == 0 && group)) return HYENA_OK;      // rows of no columns have a scale, but no runs
  if ((D > 0 && (!x || !q)) || !q_scale || !aligned_to(x, io_size(io)) || !aligned_to(q_scale, 4))
    return HYENA_ERR_INVALID_ARG;
  if (D > (group ? HYENA_MAX_PROJ_DIM : HYENA_MAX_NORM_DIM) || T > kMost / (D + 1) || x_stride > kMost / T)
    return HYENA_ERR_UNSUPPORTED;
  hyena::QuantArgs a{x, x_stride, q, q_scale, static_cast<int>(group), block, T, static_cast<int>(D),
                     io == HYENA_BF16, stream};
  return from_hip(hyena::launch_quantize(a));
}

// Whether the rows of DH at t tok + h head (t < T, h < H) do not overlap: they are written by
// different waves.  The strides times T and H fit 64 bits.
bool rows_apart(int64_t tok, int64_t head, int64_t T, int64_t H, int64_t DH) {
  if (H == 0 || (T == 1 && H == 1)) return true;
  if ((T > 1 && tok < DH) || (H > 1 && head < DH)) return false;
  if (T == 1 || H == 1 || tok >= (H - 1) * head + DH || head >= (T - 1) * tok + DH) return true;
  // neither axis lies within a step of the other: h heads on from some row, the rows of the tokens
  // to either side of that place
  for (int64_t h = 1; h < H; ++h) {
    const int64_t t = h * head / tok, past = h * head - t * tok;
    if ((t >= 1 && t < T && past < DH) || (t + 1 < T && tok - past < DH)) return false;
  }
  return true;
}

}  // namespace

extern "C" {

hyena_status_t hyena_linear_fp8(const uint8_t* x, int64_t x_stride, const float* x_scale,
                                int64_t x_scale_stride, int64_t x_group, const uint8_t* w,
                                const float* w_scale, const float* bias, void* y, int64_t y_stride,
                                int64_t T, int64_t N, int64_t K, hyena_dtype_t io,
                                hipStream_t stream) {
  if (!valid_io(io)) return HYENA_ERR_INVALID_ARG;
  hyena::LinearArgs a{x, x_stride, x_scale, x_scale_stride, 0, w, w_scale, nullptr, nullptr, bias,
                      false, hyena::ACT_NONE, y, y_stride, nullptr,
                      io == HYENA_BF16 ? hyena::OUT_BF16 : hyena::OUT_F32, T, 0, 0, stream};
  return linear_impl(a, N, K, x_group);
}

hyena_status_t hyena_gated_linear_fp8(const uint8_t* x, int64_t x_stride, const float* x_scale,
                                      int64_t x_scale_stride, int64_t x_group,
                                      const uint8_t* w_gate, const float* gate_scale,
                                      const uint8_t* w_up, const float* up_scale, hyena_act_t act,
                                      void* h, int64_t h_stride, int64_t T, int64_t I, int64_t K,
                                      hyena_dtype_t io, hipStream_t stream) {
  if (!valid_io(io) || act < HYENA_ACT_NONE || act > HYENA_ACT_SILU) return HYENA_ERR_INVALID_ARG;
  hyena::LinearArgs a{x, x_stride, x_scale, x_scale_stride, 0, w_gate, gate_scale, w_up, up_scale, nullptr,
                      true, static_cast<int>(act), h, h_stride, nullptr,
                      io == HYENA_BF16 ? hyena::OUT_BF16 : hyena::OUT_F32, T, 0, 0, stream};
  return linear_impl(a, I, K, x_group);
}

hyena_status_t hyena_gated_linear_fp8_quant(const uint8_t* x, int64_t x_stride,
                                            const float* x_scale, int64_t x_scale_stride,
                                            int64_t x_group, const uint8_t* w_gate,
                                            const float* gate_scale, const uint8_t* w_up,
                                            const float* up_scale, hyena_act_t act, uint8_t* q,
                                            float* q_scale, int64_t T, int64_t I, int64_t K,
                                            void* workspace, size_t ws_bytes, hipStream_t stream) {
  if (act < HYENA_ACT_NONE || act > HYENA_ACT_SILU) return HYENA_ERR_INVALID_ARG;
  hyena::LinearArgs a{x, x_stride, x_scale, x_scale_stride, 0, w_gate, gate_scale, w_up, up_scale, nullptr,
                      true, static_cast<int>(act), q, I, q_scale, hyena::OUT_FP8, T, 0, 0, stream,
                      static_cast<float*>(workspace)};
  return linear_impl(a, I, K, x_group, ws_bytes);
}

size_t hyena_gated_linear_fp8_workspace_size(int64_t T, int64_t I, int64_t K) {
  if (T < 1 || I < 1 || K < 0 || I > HYENA_MAX_PROJ_DIM || K > HYENA_MAX_PROJ_DIM || T > kMaxInt ||
      !hyena::linear_fits(T, I))
    return 0;
  return hyena::linear_workspace(T, I);
}

hyena_status_t hyena_quantize_fp8(const void* x, int64_t x_stride, uint8_t* q, float* q_scale,
                                  int64_t group, int64_t T, int64_t D, hyena_dtype_t io,
                                  hipStream_t stream) {
  return quantize_impl(x, x_stride, q, q_scale, group, 1, T, D, io, stream);
}

hyena_status_t hyena_quantize_weight_fp8(const void* w, int64_t w_stride, uint8_t* q, float* scale,
                                         int64_t N, int64_t K, hyena_dtype_t io,
                                         hipStream_t stream) {
  return quantize_impl(w, w_stride, q, scale, HYENA_NORM_GROUP, 128, N, K, io, stream);
}

hyena_status_t hyena_qk_norm_rope(const void* q, int64_t q_tok_stride, int64_t q_head_stride,
                                  const void* k, int64_t k_tok_stride, int64_t k_head_stride,
                                  const int32_t* positions, const float* inv_freq,
                                  int64_t rotary_dim, int32_t interleaved, int32_t norm, float eps,
                                  const float* q_weight, const float* k_weight, void* q_out,
                                  int64_t qo_tok_stride, int64_t qo_head_stride, void* k_out,
                                  int64_t ko_tok_stride, int64_t ko_head_stride, int64_t T,
                                  int64_t Hq, int64_t Hk, int64_t DH, hyena_dtype_t io,
                                  hipStream_t stream) {
  if (!valid_io(io) || T < 0 || Hq < 0 || Hk < 0 || DH < 0 || rotary_dim < 0 || rotary_dim > DH || (rotary_dim & 1) ||
      (norm && (!(eps >= 0.0f) || std::isinf(eps))) || q_tok_stride < 0 || q_head_stride < 0 ||
      k_tok_stride < 0 || k_head_stride < 0 || qo_tok_stride < 0 || qo_head_stride < 0 || ko_tok_stride < 0 ||
      ko_head_stride < 0)
    return HYENA_ERR_INVALID_ARG;
  if (T == 0 || DH == 0 || Hq + Hk == 0) return HYENA_OK;
  if ((Hq && (!q || !q_out)) || (Hk && (!k || !k_out)) || (rotary_dim && (!positions || !inv_freq)))
    return HYENA_ERR_INVALID_ARG;
  const size_t s = io_size(io);
  if (!aligned_to(q, s) || !aligned_to(k, s) || !aligned_to(q_out, s) || !aligned_to(k_out, s) ||
      !aligned_to(positions, 4) || !aligned_to(inv_freq, 4) || !aligned_to(q_weight, 4) || !aligned_to(k_weight, 4))
    return HYENA_ERR_INVALID_ARG;
  if (DH > HYENA_MAX_ROPE_DIM || Hq > HYENA_MAX_HEADS || Hk > HYENA_MAX_HEADS || T > (int64_t(1) << 25))
    return HYENA_ERR_UNSUPPORTED;
  for (const int64_t st : {q_tok_stride, k_tok_stride, qo_tok_stride, ko_tok_stride})
    if (st > kMost / T) return HYENA_ERR_UNSUPPORTED;
  for (const int64_t st : {q_head_stride, k_head_stride, qo_head_stride, ko_head_stride})
    if (st > kMost / HYENA_MAX_HEADS) return HYENA_ERR_UNSUPPORTED;
  if (!rows_apart(qo_tok_stride, qo_head_stride, T, Hq, DH) || !rows_apart(ko_tok_stride, ko_head_stride, T, Hk, DH))
    return HYENA_ERR_INVALID_ARG;
  hyena::RopeArgs a{{q, k}, {q_tok_stride, k_tok_stride}, {q_head_stride, k_head_stride}, {q_out, k_out},
                    {qo_tok_stride, ko_tok_stride}, {qo_head_stride, ko_head_stride}, {q_weight, k_weight},
                    {static_cast<int>(Hq), static_cast<int>(Hk)}, positions, inv_freq,
                    static_cast<int>(rotary_dim), interleaved != 0, norm != 0, eps, T, static_cast<int>(DH),
                    io == HYENA_BF16, stream};
  return from_hip(hyena::launch_qk_norm_rope(a));
}

}  // extern "C"
