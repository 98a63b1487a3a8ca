// quantize.hip -- e4m3 codes and scales of activations (a scale per row or per
// 128 columns) and of weights (per 128 x 128 block).
//
// The operands of the 8-bit projections that no norm makes: a mixer's output in
// front of out_proj (evo2_flash README, layer_names table), and the weights.
// Over a run or block,
//     scale = max(max|x| / 448, 2^-140) (1 where x is 0),   q = e4m3(x * (1 / scale)).
//
// One pass over memory, which bounds all of them: a run, row or block stays in registers between
// its maximum and its codes.  Measured: 32768 x 4096 bf16 per 128 columns 75 to 80 us, 5.1 to 5.4 TB/s;
// weights of 11008 x 4096 fp32 41.5 us, 5.4 TB/s; 16 x 4096 2.6 to 3.4 us in a graph, the launch; rows of 64
// columns, a workgroup each, 262144 of them 75 us, 0.7 TB/s.
#include "linear_common.hpp"

namespace hyena {

// codes of eight values, of which n exist
__device__ __forceinline__ void put8(uint8_t* p, int64_t n, const float (&x)[8], float scale) {
  uint32_t w[2];
  to_codes<8>(x, scale, w);
  if (n >= 8) {
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n) p[e] = static_cast<uint8_t>(w[e >> 2] >> (8 * (e & 3)));
  }
}

__device__ __forceinline__ uint32_t top8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t b = mag_bits(x[e]);
    m = b > m ? b : m;
  }
  return m;
}

// A scale per 128 columns: 16 lanes per run, V runs per lane set; consecutive
// runs of a row, then of the next, so that a wave's loads are contiguous.
template <typename IO, int V>
__global__ __launch_bounds__(256) void quantize_runs_kernel(const IO* x, int64_t x_stride, uint8_t* q,
                                                            float* q_scale, int64_t T, int D, int runs) {
  const int sub = static_cast<int>(threadIdx.x) >> 4, c0 = (static_cast<int>(threadIdx.x) & 15) * 8;
  const int64_t total = T * runs;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (16 * V) + sub;
  float v[V][8];
  int64_t row[V];
  int col[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t g = first + i * 16;
    row[i] = g < total ? g / runs : T;
    col[i] = static_cast<int>(g - row[i] * runs) * RUN + c0;
    if (g < total) load8(x + row[i] * x_stride + col[i], static_cast<int64_t>(D) - col[i], v[i]);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (row[i] >= T) return;            // a run's 16 lanes together
    const float scale = run_scale(max16(top8(v[i])));
    if (c0 == 0) q_scale[first + i * 16] = scale;
    put8(q + row[i] * D + col[i], static_cast<int64_t>(D) - col[i], v[i], scale);
  }
}

// A scale per row: W waves hold it, NV steps of 512 W columns.
template <typename IO, int W, int NV>
__global__ __launch_bounds__(W * 64) void quantize_rows_kernel(const IO* x, int64_t x_stride, uint8_t* q,
                                                               float* q_scale, int D) {
  __shared__ uint32_t sh[W];
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const IO* xr = x + row * x_stride;
  float v[NV][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = ((i * W + wave) * 64 + lane) * 8;
    load8(xr + c, static_cast<int64_t>(D) - c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const uint32_t t = top8(v[i]);
    m = t > m ? t : m;
  }
  m = max64(m);
  if constexpr (W > 1) {
    if (lane == 0) sh[wave] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) m = sh[i] > m ? sh[i] : m;
  }
  const float scale = run_scale(m);
  if (threadIdx.x == 0) q_scale[row] = scale;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = ((i * W + wave) * 64 + lane) * 8;
    put8(q + row * D + c, static_cast<int64_t>(D) - c, v[i], scale);
  }
}

// A scale per 128 x 128 block: a workgroup holds it, eight rows per thread.
template <typename IO>
__global__ __launch_bounds__(256) void quantize_blocks_kernel(const IO* x, int64_t x_stride, uint8_t* q,
                                                              float* q_scale, int64_t T, int D, int runs) {
  __shared__ uint32_t sh[4];
  const int col = static_cast<int>(blockIdx.x % runs) * RUN + (static_cast<int>(threadIdx.x) & 15) * 8;
  const int64_t row = static_cast<int64_t>(blockIdx.x / runs) * RUN + (threadIdx.x >> 4);
  float v[8][8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8(x + (row + 16 * i) * x_stride + col, row + 16 * i < T ? static_cast<int64_t>(D) - col : 0, v[i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t t = top8(v[i]);
    m = t > m ? t : m;
  }
  m = max64(m);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i) m = sh[i] > m ? sh[i] : m;
  const float scale = run_scale(m);
  if (threadIdx.x == 0) q_scale[blockIdx.x] = scale;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (row + 16 * i < T) put8(q + (row + 16 * i) * D + col, static_cast<int64_t>(D) - col, v[i], scale);
}

template <typename IO>
static void quantize_go(const QuantArgs& a) {
  const IO* x = static_cast<const IO*>(a.x);
  const int runs = (a.D + RUN - 1) / RUN;
  if (a.block > 1) {
    const int64_t n = (a.T + RUN - 1) / RUN * runs;
    quantize_blocks_kernel<IO><<<static_cast<unsigned>(n), 256, 0, a.stream>>>(x, a.x_stride, a.q, a.q_scale, a.T,
                                                                             a.D, runs);
  } else if (a.group) {
    const int64_t n = a.T * runs;
    constexpr int V = sizeof(IO) == 2 ? 4 : 2;
    quantize_runs_kernel<IO, V><<<static_cast<unsigned>((n + 16 * V - 1) / (16 * V)), 256, 0, a.stream>>>(
        x, a.x_stride, a.q, a.q_scale, a.T, a.D, runs);
  } else {
    auto go = [&](auto kernel, int waves) {
      kernel<<<static_cast<unsigned>(a.T), waves * 64, 0, a.stream>>>(x, a.x_stride, a.q, a.q_scale, a.D);
    };
    if (a.D <= 512) go(quantize_rows_kernel<IO, 1, 1>, 1);
    else if (a.D <= 1024) go(quantize_rows_kernel<IO, 1, 2>, 1);
    else if (a.D <= 2048) go(quantize_rows_kernel<IO, 4, 1>, 4);
    else if (a.D <= 4096) go(quantize_rows_kernel<IO, 4, 2>, 4);
    else if (a.D <= 8192) go(quantize_rows_kernel<IO, 4, 4>, 4);
    else go(quantize_rows_kernel<IO, 16, 4>, 16);
  }
}

hipError_t launch_quantize(const QuantArgs& a) {
  // a grid holds less than 2^32 threads; rows go in pieces (whole blocks of them)
  const int64_t runs = (a.D + RUN - 1) / RUN;
  int64_t most = int64_t(1) << 21;
  if (a.group) {
    const int64_t per = (int64_t(1) << 24) / runs;       // 16 lanes a run, 2 lanes per row and run of a block
    most = per < RUN ? RUN : per / RUN * RUN;
  }
  const int64_t size = a.bf16 ? 2 : 4;
  for (int64_t t = 0; t < a.T; t += most) {
    QuantArgs b = a;
    b.T = a.T - t < most ? a.T - t : most;
    b.x = static_cast<const char*>(a.x) + t * a.x_stride * size;
    b.q = a.q + t * a.D;
    b.q_scale = a.q_scale + (a.block > 1 ? t / RUN * runs : a.group ? t * runs : t);
    if (a.bf16) quantize_go<bf16_t>(b);
    else quantize_go<float>(b);
  }
  return hipGetLastError();
}

}  // namespace hyena
