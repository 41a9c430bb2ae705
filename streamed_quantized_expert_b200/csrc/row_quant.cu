// Rows quantised to 8-bit integers with one scale per row: plain rows
// (moe_quantize_channels), the sum and root-mean-square norm in front of a
// layer (moe_add_norm_quant), and SwiGLU (moe_swiglu_quant).
//
// Mathematics: for a row p with a = max |p_i|, q_i = rint(127 p_i / a) (ties
// to even) and scale = a / 127.  The norm's factor r = 1 / sqrt(mean h^2 +
// eps) multiplies the whole row, so the codes need only p_i = h_i g_i (rounded
// to 32 bits, exact for bf16 h) and r joins the scale: a code does not depend
// on the order in which the squares were summed.
#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr int kRowThreads = 256;

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t i, float (&v)[8]) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + i);
    v[0] = bf16_lo(a.x), v[1] = bf16_hi(a.x), v[2] = bf16_lo(a.y), v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z), v[5] = bf16_hi(a.z), v[6] = bf16_lo(a.w), v[7] = bf16_hi(a.w);
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  return (uint32_t)f32_to_bf16_rne(lo) | ((uint32_t)f32_to_bf16_rne(hi) << 16);
}

__device__ __forceinline__ void store8_bf16(uint16_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <bool F32>
__device__ __forceinline__ void store8(void* base, int64_t i, const float (&v)[8]) {
  if constexpr (F32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    store8_bf16(static_cast<uint16_t*>(base) + i, v);
  }
}

// Bits of |p|: as unsigned numbers they order like the magnitudes, with
// infinities and then NaN above every finite one.
__device__ __forceinline__ uint32_t abs_bits(float p) { return __float_as_uint(p) & 0x7fffffffu; }

// rint(127 p / a) exactly: the quotient of two 32-bit floats is no nearer to
// a tie than 2^-40 of its size unless it is one, so the 64-bit quotient
// rounds to the same integer.
__device__ __forceinline__ int code_of(float p, float a) { return (int)rint(127.0 * (double)p / (double)a); }

__device__ __forceinline__ void store8_codes(int8_t* p, const float (&v)[8], uint32_t amax) {
  uint32_t w[2] = {0u, 0u};
  if (amax != 0u && amax < 0x7f800000u) {  // a row of zeros, or with an infinity or NaN, has codes 0
    const float a = __uint_as_float(amax);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)code_of(v[i], a) & 0xffu) << (8 * (i & 3));
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

// Sum and largest magnitude over the block, in a fixed order.
__device__ __forceinline__ void block_reduce(float& sum, uint32_t& amax) {
  __shared__ float s_sum[kRowThreads / 32];
  __shared__ uint32_t s_max[kRowThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  amax = __reduce_max_sync(0xffffffffu, amax);
  if ((threadIdx.x & 31) == 0) {
    s_sum[threadIdx.x >> 5] = sum;
    s_max[threadIdx.x >> 5] = amax;
  }
  __syncthreads();
  sum = 0.0f;
  amax = 0u;
#pragma unroll
  for (int w = 0; w < kRowThreads / 32; ++w) {
    sum += s_sum[w];
    amax = max(amax, s_max[w]);
  }
}

// The row's scale: a r / 127; NaN for a row with an infinity or NaN, so that
// what is computed from its codes shows it.
__device__ __forceinline__ float scale_of(uint32_t amax, float r) {
  return amax < 0x7f800000u ? __fdiv_rn(__fmul_rn(__uint_as_float(amax), r), 127.0f) : __uint_as_float(0x7fffffffu);
}

// The eight values of row `row` at column c: what is quantised, or (norm) the
// residual sum in its own type.
template <int OP, bool HF32, bool DF32>
__device__ __forceinline__ void row_values(const RowQuantArgs& a, int64_t row, int c, float (&v)[8]) {
  if constexpr (OP == kRowSwiglu) {
    float u[8];
    load8<HF32>(a.in, row * 2 * a.H + c, v);
    load8<HF32>(a.in, row * 2 * a.H + a.H + c, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __fdiv_rn(v[i], 1.0f + expf(-v[i])) * u[i];
  } else {
    load8<HF32>(a.in, row * a.H + c, v);
    if (OP == kRowNorm && a.delta) {
      float d[8];
      load8<DF32>(a.delta, row * a.H + c, d);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] += d[i];
        if (!HF32) v[i] = __uint_as_float((uint32_t)f32_to_bf16_rne(v[i]) << 16);
      }
    }
  }
}

template <int OP, bool HF32, bool DF32>
__global__ void __launch_bounds__(kRowThreads) row_quant_kernel(const RowQuantArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t row = blockIdx.x;
  float sum = 0.0f;
  uint32_t amax = 0u;
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * kRowThreads) {
    float v[8], g[8];
    row_values<OP, HF32, DF32>(a, row, c, v);
    if constexpr (OP == kRowNorm) {
      if (a.h_out) store8<HF32>(a.h_out, row * a.H + c, v);
      load8<false>(a.gamma, c, g);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (OP == kRowNorm) {
        sum = fmaf(v[i], v[i], sum);
        v[i] *= g[i];
      }
      amax = max(amax, abs_bits(v[i]));
    }
  }
  block_reduce(sum, amax);
  const float r = OP == kRowNorm ? rsqrtf(sum / (float)a.H + a.eps) : 1.0f;
  if (a.scale && threadIdx.x == 0) a.scale[row] = scale_of(amax, r);
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * kRowThreads) {
    float v[8], g[8], x[8];
    if (OP == kRowNorm && a.h_out)
      load8<HF32>(a.h_out, row * a.H + c, v);  // this thread's own writes (h_out may be the input)
    else
      row_values<OP, HF32, DF32>(a, row, c, v);
    if constexpr (OP == kRowNorm) {
      load8<false>(a.gamma, c, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = v[i] * r * g[i];
        v[i] *= g[i];
      }
      if (a.x) store8_bf16(a.x + row * a.H + c, x);
    }
    if (a.q) store8_codes(a.q + row * a.H + c, v, amax);
  }
}

template <int OP>
const void* row_kernel(bool hf32, bool df32) {
  if constexpr (OP == kRowNorm) {
    if (df32)
      return hf32 ? reinterpret_cast<const void*>(row_quant_kernel<OP, true, true>)
                  : reinterpret_cast<const void*>(row_quant_kernel<OP, false, true>);
  }
  return hf32 ? reinterpret_cast<const void*>(row_quant_kernel<OP, true, false>)
              : reinterpret_cast<const void*>(row_quant_kernel<OP, false, false>);
}

}  // namespace

cudaError_t launch_row_quant(const RowQuantArgs& a, int op, bool in_f32, bool delta_f32, int T, cudaStream_t st) {
  const void* kern = op == kRowNorm    ? row_kernel<kRowNorm>(in_f32, delta_f32)
                     : op == kRowSwiglu ? row_kernel<kRowSwiglu>(in_f32, false)
                                        : row_kernel<kRowPlain>(in_f32, false);
  return launch_pdl(kern, T, kRowThreads, 0, st, a);
}

}  // namespace moe
