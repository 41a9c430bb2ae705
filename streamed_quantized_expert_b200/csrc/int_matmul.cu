// Product of 8-bit integer rows with a scale per token and per output
// (moe_int_matmul): y[t][n] = add[t][n] + row_w[t] xs[t] ws[n] sum_k xq[t][k] wq[n][k].
//
// The sum is a whole number below 2^31 (K <= 65,536), so int32 accumulation
// is exact in any order; the scales are applied once to each sum.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kTile = 64, kKc = 64;  // outputs and tokens of a block; inputs of a step

__global__ void __launch_bounds__(256) int_matmul_kernel(const IntMatmulArgs a) {
  __shared__ int s_w[kTile][kKc / 4 + 1], s_x[kTile][kKc / 4 + 1];
  pdl_wait();
  pdl_launch_dependents();
  const int n0 = blockIdx.x * kTile, t0 = blockIdx.y * kTile;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  int acc[4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += kKc) {
    for (int i = threadIdx.x; i < kTile * (kKc / 4); i += 256) {
      const int r = i / (kKc / 4), c = i % (kKc / 4), k = k0 + 4 * c;
      const bool in = k < a.K;
      s_w[r][c] = in && n0 + r < a.N ? *reinterpret_cast<const int*>(a.wq + (int64_t)(n0 + r) * a.K + k) : 0;
      s_x[r][c] = in && t0 + r < a.T ? *reinterpret_cast<const int*>(a.xq + (int64_t)(t0 + r) * a.K + k) : 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kKc / 4; ++c)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(s_x[ty + 16 * i][c], s_w[tx + 16 * j][c], acc[i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int t = t0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (t >= a.T || n >= a.N) continue;
      const int64_t at = (int64_t)t * a.N + n;
      const float xs = a.row_w ? a.xs[t] * a.row_w[t] : a.xs[t];
      float v = (float)acc[i][j] * (xs * a.ws[n]);
      if (a.add) v += a.add[at];
      if (a.y_f32)
        static_cast<float*>(a.y)[at] = v;
      else
        static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rne(v);
    }
}

}  // namespace

cudaError_t launch_int_matmul(const IntMatmulArgs& a, int num_sms, cudaStream_t st) {
  (void)num_sms;
  const dim3 grid((unsigned)((a.N + kTile - 1) / kTile), (unsigned)((a.T + kTile - 1) / kTile));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int_matmul_kernel, a);
}

}  // namespace moe
