// Rows quantised to 8-bit integers with one scale per row: plain rows
// (moe_quantize_channels), the sum and root-mean-square norm in front of a
// layer (moe_add_norm_quant), and SwiGLU (moe_swiglu_quant).
//
// Mathematics: for a row p with a = max |p_i|, q_i = rint(127 p_i / a) (ties
// to even) and scale = a / 127.  The norm's factor r = 1 / sqrt(mean h^2 +
// eps) multiplies the whole row, so the codes need only p_i = h_i g_i (rounded
// to 32 bits, exact for bf16 h) and r joins the scale: a code does not depend
// on the order in which the squares were summed.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Two fp32 lanes to an instruction: each rounds as its scalar counterpart.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 split2(F2 a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 bf16_pair(uint32_t w) { return pack2(bf16_lo(w), bf16_hi(w)); }
__device__ __forceinline__ uint32_t to_bf16_pair(F2 a) {
  const float2 f = split2(a);
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// max(m, |a|, |b|), NaN if one of them is.
__device__ __forceinline__ float max_abs(float m, F2 a) {
  const float2 f = split2(a);
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(f.x), "f"(f.y));
  return r;
}

// Eight values: 16 bytes of bf16, or 32 of fp32.
template <bool F32>
__host__ __device__ constexpr int raw_words() {
  return F32 ? 2 : 1;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const uint4* w, F2 (&v)[4]) {
  if constexpr (F32) {
    v[0] = pack2(__uint_as_float(w[0].x), __uint_as_float(w[0].y));
    v[1] = pack2(__uint_as_float(w[0].z), __uint_as_float(w[0].w));
    v[2] = pack2(__uint_as_float(w[1].x), __uint_as_float(w[1].y));
    v[3] = pack2(__uint_as_float(w[1].z), __uint_as_float(w[1].w));
  } else {
    v[0] = bf16_pair(w[0].x), v[1] = bf16_pair(w[0].y), v[2] = bf16_pair(w[0].z), v[3] = bf16_pair(w[0].w);
  }
}
__device__ __forceinline__ uint4 pack8_bf16(const F2 (&v)[4]) {
  return make_uint4(to_bf16_pair(v[0]), to_bf16_pair(v[1]), to_bf16_pair(v[2]), to_bf16_pair(v[3]));
}
template <bool F32>
__device__ __forceinline__ const uint4* raw_at(const void* base, int64_t i) {
  return reinterpret_cast<const uint4*>(static_cast<const char*>(base) + i * (F32 ? 4 : 2));
}

// The largest magnitude over the warp.  Bits of magnitudes order like the
// magnitudes, infinities and then NaN above every finite one.
__device__ __forceinline__ float warp_max(float m) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// How a row's values p become codes, rint(127 p / a) exactly.
//
// NARROW (p and a have at most 16 bits: bf16 values, and their products with a
// bf16 gamma): 127 p has 23 bits, and a quotient of such numbers that is not a
// tie is at least one fp32 step away from every tie (2^-16 next to numbers up
// to 127, whose step is 2^-17, and so on down).  So the fp32 quotient, made
// correct by one step from the reciprocal, rounds to the right integer, ties
// included.
//
// Otherwise: inv = 127 / a carries the errors of a reciprocal (2^-23) and of a
// product (2^-24), so p inv is within 127 x 1.5 x 2^-23 < 2.3e-5 of 127 p / a
// and rounds to the same integer unless it is within 3e-5 of a tie.  There the
// sign of 254 p - (2 k +- 1) a decides, whose terms have 32 bits: exact in 64.
template <bool NARROW>
struct RowCoder {
  static constexpr float kMagic = 12582912.0f;  // 1.5 x 2^23: adding it leaves the rounded integer in the low bits
  float a, inv, times;
  bool none;
  __device__ explicit RowCoder(float amax) {
    none = !(amax > 0.0f && amax < INFINITY);  // a row of zeros, or with an infinity or NaN: codes 0
    // where 127 / a or 1 / a would leave the normal numbers, the row is taken
    // times 2^+-100 (exactly, but for values far below half a code)
    times = amax < 0x1p-100f ? 0x1p100f : amax > 0x1p100f ? 0x1p-100f : 1.0f;
    a = amax * times;
    inv = none ? 0.0f : (NARROW ? 1.0f : 127.0f) * rcp(a);
  }
  // code k next to the tie in the direction of d = p inv - k
  __device__ __forceinline__ uint32_t beside_tie(float p, float d, uint32_t bits) const {
    if (fabsf(d) <= 0.5f - 3e-5f) return bits;
    const int k = (int)(int8_t)bits, s = d > 0.0f ? 1 : -1;
    const double e = (double)s * fma((double)-(2 * k + s), (double)a, 254.0 * (double)p);
    return (uint32_t)(e > 0.0 || (e == 0.0 && (k & 1)) ? k + s : k);
  }
  __device__ __forceinline__ uint2 codes(const F2 (&q)[4]) const {
    const F2 magic = pack2(kMagic, kMagic), i2 = pack2(inv, inv);
    F2 p[4];
    uint32_t c[8];
    if (none) return make_uint2(0u, 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = q[i];
    if (times != 1.0f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = mul2(p[i], pack2(times, times));
    }
    if constexpr (NARROW) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 n = mul2(p[i], pack2(127.0f, 127.0f)), t = mul2(n, i2);
        const float2 f = split2(add2(fma2(fma2(t, pack2(-a, -a), n), i2, t), magic));
        c[2 * i] = __float_as_uint(f.x);
        c[2 * i + 1] = __float_as_uint(f.y);
      }
    } else {
      F2 d[4];
      float off = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const F2 m = fma2(p[i], i2, magic);
        d[i] = fma2(p[i], i2, fma2(m, pack2(-1.0f, -1.0f), magic));
        off = max_abs(off, d[i]);
        const float2 f = split2(m);
        c[2 * i] = __float_as_uint(f.x);
        c[2 * i + 1] = __float_as_uint(f.y);
      }
      if (off > 0.5f - 3e-5f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 pf = split2(p[i]), df = split2(d[i]);
          c[2 * i] = beside_tie(pf.x, df.x, c[2 * i]);
          c[2 * i + 1] = beside_tie(pf.y, df.y, c[2 * i + 1]);
        }
      }
    }
    return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                      __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
  }
};

// Sum and largest magnitude over the row's threads (a warp, or the block), in a fixed order.
template <bool WARP>
__device__ __forceinline__ void row_reduce(float& sum, float& amax) {
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  amax = warp_max(amax);
  if constexpr (!WARP) {
    __shared__ float2 s[32];
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    if (lane == 0) s[threadIdx.x >> 5] = make_float2(sum, amax);
    __syncthreads();
    const float2 v = lane < warps ? s[lane] : make_float2(0.0f, 0.0f);
    sum = v.x;
    amax = warp_max(v.y);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  }
}

// The row's scale: a r / 127; NaN for a row with an infinity or NaN, so that
// what is computed from its codes shows it.
__device__ __forceinline__ float scale_of(float amax, float r) {
  return amax < INFINITY ? __fdiv_rn(__fmul_rn(amax, r), 127.0f) : __uint_as_float(0x7fffffffu);
}

__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// silu(g) u.  With s = exp(-|g|) in [0, 1], silu(g) is g (1 or s) / (1 + s),
// whose denominator never overflows; the quotient is corrected once, which
// leaves one rounding.  s = 2^(t + e): t = -|g| log2 e rounded, e what the
// rounding and the constant's tail leave out, 2^e = 1 + e ln 2 (e < 2^-15).
// |g| above 128 gives 0 like 128 does.  24 instructions a value with its code,
// two lanes to an instruction, are 22 us of issue at 4000 x 8200; at 27 warps an
// SM, which all load, meet a barrier and then code, 2.5 of 4 slots issue: bf16
// takes 38-41 us (4.0-4.3 TB/s), fp32 73 us (4.0 TB/s).
__device__ __forceinline__ F2 swiglu_of(F2 g2, F2 u) {
  const float2 g = split2(g2);
  const F2 m = pack2(fminf(fabsf(g.x), 128.0f), fminf(fabsf(g.y), 128.0f)), one = pack2(1.0f, 1.0f);
  const F2 t = mul2(m, pack2(0x1.715476p+0f, 0x1.715476p+0f));  // -t above
  const F2 e = fma2(m, pack2(-0x1.4ae0cp-26f, -0x1.4ae0cp-26f), fma2(m, pack2(-0x1.715476p+0f, -0x1.715476p+0f), t));
  const float2 tf = split2(t);
  const F2 p = pack2(exp2_of(-tf.x), exp2_of(-tf.y));
  const F2 s2 = fma2(mul2(e, pack2(0x1.62e43p-1f, 0x1.62e43p-1f)), p, p), d2 = add2(s2, one);
  const float2 s = split2(s2), d = split2(d2);
  // with n = -g (1 or s) and r = -1 / (1 + s) rounded: q = n r, then q + (q (1 + s) + n) r
  const F2 n = mul2(g2, pack2(g.x < 0.0f ? -s.x : -1.0f, g.y < 0.0f ? -s.y : -1.0f));
  const F2 r = pack2(rcp(-d.x), rcp(-d.y)), q = mul2(n, r);
  return mul2(fma2(fma2(d2, q, n), r, q), u);
}

// What a thread reads for eight columns of a row: one or two arrays of eight values.
template <int OP, bool HF32, bool DF32>
struct RowRaw {
  static constexpr bool kTwo = OP != kRowPlain, kSecondF32 = OP == kRowSwiglu ? HF32 : DF32;
  static constexpr int kFirst = raw_words<HF32>(), kWords = kFirst + (kTwo ? raw_words<kSecondF32>() : 0);
  static __device__ __forceinline__ const uint4* first(const RowQuantArgs& a, int64_t row, int c) {
    return raw_at<HF32>(a.in, row * (OP == kRowSwiglu ? 2 * a.H : a.H) + c);
  }
  static __device__ __forceinline__ const uint4* second(const RowQuantArgs& a, int64_t row, int c) {
    if constexpr (OP == kRowSwiglu) return raw_at<HF32>(a.in, (row * 2 + 1) * a.H + c);
    return raw_at<DF32>(a.delta, row * a.H + c);
  }
  static __device__ __forceinline__ bool two(const RowQuantArgs& a) {
    return OP == kRowSwiglu || (OP == kRowNorm && a.delta);
  }
  // What is quantised, or (norm) the residual sum in its own type, which goes
  // to h_out.  Two bf16 numbers are added as such: their sum rounded once is
  // their fp32 sum rounded (that one is exact unless one of them is below
  // 2^-16 of the other, and then both round to the larger).
  static __device__ __forceinline__ void values(const RowQuantArgs& a, int64_t row, int c, uint4 (&w)[kWords],
                                                F2 (&v)[4]) {
    if constexpr (OP == kRowNorm) {
      if (a.delta) {
        if constexpr (!HF32 && !DF32) {
          __nv_bfloat162* x = reinterpret_cast<__nv_bfloat162*>(&w[0]);
          const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(&w[1]);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[i] = __hadd2_rn(x[i], y[i]);
          unpack8<false>(w, v);
        } else {
          F2 d[4];
          unpack8<HF32>(w, v);
          unpack8<DF32>(w + kFirst, d);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = add2(v[i], d[i]);
          if constexpr (HF32) {
            const float2 f0 = split2(v[0]), f1 = split2(v[1]), f2 = split2(v[2]), f3 = split2(v[3]);
            w[0] = make_uint4(__float_as_uint(f0.x), __float_as_uint(f0.y), __float_as_uint(f1.x), __float_as_uint(f1.y));
            w[1] = make_uint4(__float_as_uint(f2.x), __float_as_uint(f2.y), __float_as_uint(f3.x), __float_as_uint(f3.y));
          } else {
            w[0] = pack8_bf16(v);
            unpack8<false>(w, v);
          }
        }
      } else {
        unpack8<HF32>(w, v);
      }
      if (a.h_out) {
        uint4* h = const_cast<uint4*>(raw_at<HF32>(a.h_out, row * a.H + c));
#pragma unroll
        for (int k = 0; k < kFirst; ++k) h[k] = w[k];
      }
    } else {
      unpack8<HF32>(w, v);
      if constexpr (OP == kRowSwiglu) {
        F2 u[4];
        unpack8<HF32>(w + kFirst, u);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = swiglu_of(v[i], u[i]);
      }
    }
  }
  static __device__ __forceinline__ void load(const RowQuantArgs& a, int64_t row, int c, uint4 (&w)[kWords]) {
#pragma unroll
    for (int k = 0; k < kFirst; ++k) w[k] = first(a, row, c)[k];
    if (kTwo && two(a)) {
#pragma unroll
      for (int k = kFirst; k < kWords; ++k) w[k] = second(a, row, c)[k - kFirst];
    }
  }
};

// Of the eight values: the squares' sum, p in their place, and p's largest magnitude.
template <int OP>
__device__ __forceinline__ void row_stats(const uint4& gamma, F2 (&v)[4], F2& sum, float& amax) {
  F2 g[4];
  if constexpr (OP == kRowNorm) unpack8<false>(&gamma, g);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (OP == kRowNorm) {
      sum = fma2(v[i], v[i], sum);
      v[i] = mul2(v[i], g[i]);
    }
    amax = max_abs(amax, v[i]);
  }
}

template <int OP, bool NARROW>
__device__ __forceinline__ void row_out(const RowQuantArgs& a, int64_t row, int c, const F2 (&p)[4], float r,
                                        const RowCoder<NARROW>& coder) {
  if constexpr (OP == kRowNorm) {
    if (a.x) {
      F2 x[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = mul2(p[i], pack2(r, r));
      *reinterpret_cast<uint4*>(a.x + row * a.H + c) = pack8_bf16(x);
    }
    if (!a.q) return;
  }
  *reinterpret_cast<uint2*>(a.q + row * a.H + c) = coder.codes(p);
}

// One value of the residual: read back from h_out (the caller's own writes;
// h_out may be the input), or summed again.
template <bool HF32, bool DF32>
__device__ __forceinline__ float residual_at(const RowQuantArgs& a, int64_t at) {
  auto load = [](const void* p, bool f32, int64_t i) {
    return f32 ? static_cast<const float*>(p)[i] : __uint_as_float((uint32_t) static_cast<const uint16_t*>(p)[i] << 16);
  };
  const float h = load(a.h_out ? a.h_out : a.in, HF32, at);
  if (a.h_out || !a.delta) return h;
  const float sum = __fadd_rn(h, load(a.delta, DF32, at));
  return HF32 ? sum : __uint_as_float((uint32_t)f32_to_bf16_rne(sum) << 16);
}

// The row's factor r, from the sum of its squares.  Where that left fp32's
// range (512 squares of 1e18 do), or where next to a tiny eps the squares lost
// bits below it (mean + eps under 2^-80, of which the 2^-150 that a square may
// lose is more than 2^-70), the row is read again and summed times 2^-80 or
// 2^60, whose squares stay below 2^96 and 2^56: powers of two, which round
// nothing else.  i, n: this thread and the row's threads.  One value at a time,
// so that ordinary rows, which never come here, keep their registers.
template <int OP, bool HF32, bool DF32, bool WARP>
__device__ __forceinline__ float row_factor(const RowQuantArgs& a, int64_t row, int i, int n, float sum) {
  if constexpr (OP != kRowNorm) return 1.0f;
  const float mean = fmaf(sum, a.inv_h, a.eps);
  if (mean >= 0x1p-80f && mean < INFINITY) return rsqrtf(mean);
  const float times = mean < 1.0f ? 0x1p60f : 0x1p-80f;
  float amax = 0.0f;
  sum = 0.0f;
#pragma unroll 1
  for (int c = 8 * i; c < a.H; c += c % 8 == 7 ? 8 * n - 7 : 1) {
    const float v = times * residual_at<HF32, DF32>(a, row * a.H + c);
    sum = fmaf(v, v, sum);
  }
  if (!WARP) __syncthreads();  // the first sums have been read
  row_reduce<WARP>(sum, amax);
  return times * rsqrtf(fmaf(sum, a.inv_h, a.eps * times * times));
}

// Threads of a block at most, and blocks that an SM is to hold.  The norm of
// short bf16 rows keeps 32 registers, so that its cold path costs no occupancy.
__host__ __device__ constexpr int row_threads(int op, int ch, bool warp) {
  return warp || (op == kRowNorm && ch == 1) ? 256 : ch == 4 ? 512 : 1024;
}
__host__ __device__ constexpr int row_blocks(int op, bool hf32, int ch, bool warp) {
  return ch == 4 ? 2 : op == kRowNorm && ch == 1 ? (hf32 ? 6 : 8) : 1;
}

// Rows held in registers, CH pieces of eight columns a thread: one pass over
// the data.  A row is a warp's (WARP: eight rows to a block) or a block's.
template <int OP, bool HF32, bool DF32, int CH, bool WARP>
__global__ void __launch_bounds__(row_threads(OP, CH, WARP), row_blocks(OP, HF32, CH, WARP))
    row_quant_kernel(const RowQuantArgs a) {
  using Raw = RowRaw<OP, HF32, DF32>;
  const int n = WARP ? 32 : blockDim.x, i = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row = WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (WARP && row >= a.T) return;
  uint4 w[CH][Raw::kWords], gamma[CH];
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = 8 * (i + j * n);
    if (c < a.H) {
      Raw::load(a, row, c, w[j]);
      if constexpr (OP == kRowNorm) gamma[j] = *raw_at<false>(a.gamma, c);
    }
  }
  F2 v[CH][4], sum2 = pack2(0.0f, 0.0f);
  float amax = 0.0f;
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = 8 * (i + j * n);
    if (c < a.H) {
      Raw::values(a, row, c, w[j], v[j]);
      row_stats<OP>(gamma[j], v[j], sum2, amax);
    }
  }
  const float2 half = split2(sum2);
  float sum = half.x + half.y;
  row_reduce<WARP>(sum, amax);
  const float r = row_factor<OP, HF32, DF32, WARP>(a, row, i, n, sum);
  const RowCoder<OP != kRowSwiglu && !HF32> coder(amax);
  if (i == 0 && a.scale) a.scale[row] = scale_of(amax, r);
#pragma unroll
  for (int j = 0; j < CH; ++j) {
    const int c = 8 * (i + j * n);
    if (c < a.H) row_out<OP>(a, row, c, v[j], r, coder);
  }
}

// Longer rows: read a second time, from L2 (a row of 65,536 fp32 values is 256 KB).
template <int OP, bool HF32, bool DF32>
__global__ void __launch_bounds__(1024) row_quant_long_kernel(RowQuantArgs a) {
  using Raw = RowRaw<OP, HF32, DF32>;
  const int64_t row = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  F2 sum2 = pack2(0.0f, 0.0f), unused_sum = sum2;
  float amax = 0.0f, unused_max = 0.0f;
  uint4 w[Raw::kWords], g = make_uint4(0u, 0u, 0u, 0u);
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * blockDim.x) {
    F2 v[4];
    Raw::load(a, row, c, w);
    Raw::values(a, row, c, w, v);
    if constexpr (OP == kRowNorm) g = *raw_at<false>(a.gamma, c);
    row_stats<OP>(g, v, sum2, amax);
  }
  const float2 half = split2(sum2);
  float sum = half.x + half.y;
  row_reduce<false>(sum, amax);
  const float r = row_factor<OP, HF32, DF32, false>(a, row, threadIdx.x, blockDim.x, sum);
  const RowCoder<OP != kRowSwiglu && !HF32> coder(amax);
  if (threadIdx.x == 0 && a.scale) a.scale[row] = scale_of(amax, r);
  if (OP == kRowNorm && a.h_out) {  // from here on the residual is this thread's own writes (h_out may be the input)
    a.in = a.h_out;
    a.h_out = nullptr;
    a.delta = nullptr;
  }
  for (int c = 8 * threadIdx.x; c < a.H; c += 8 * blockDim.x) {
    F2 v[4];
    Raw::load(a, row, c, w);
    Raw::values(a, row, c, w, v);
    if constexpr (OP == kRowNorm) g = *raw_at<false>(a.gamma, c);
    row_stats<OP>(g, v, unused_sum, unused_max);
    row_out<OP>(a, row, c, v, r, coder);
  }
}

struct RowPlan {
  const void* fn;
  int threads, rows;  // of a block
};

template <int OP, bool HF32, bool DF32, int CH, bool WARP>
RowPlan row_plan_of(int threads) {
  return {reinterpret_cast<const void*>(row_quant_kernel<OP, HF32, DF32, CH, WARP>), threads, WARP ? 8 : 1};
}

// By the row's length alone, so that a row's results do not depend on how many
// rows there are.  Short rows are a warp's.  More pieces a thread mean fewer
// threads at a row's barrier and more loads on the way, but a longer wait for
// a single row: 16384 x 4096 bf16 + bf16 takes 90.0 / 89.0 / 90.3 us with 1 /
// 2 / 4 pieces, one row of it 1.7 / 1.9 / 2.4, 16384 x 4104 99.5 / 92.6 with 2 /
// 4, 8192 x 7168 90.9 / 79.6; 4096 x 7168 plain bf16 29.1 / 20.6 / 17.4, fp32
// 49.8 / 29.0 / 34.8.
template <int OP, bool HF32, bool DF32>
RowPlan row_plan(int H) {
  constexpr int kLong = OP == kRowNorm ? 2048 : 1024;  // one piece a thread up to here
  constexpr bool kFour = RowRaw<OP, HF32, DF32>::kWords <= 2 && !HF32;
  auto threads = [&](int ch) { return (H / 8 + ch * 32 - 1) / (ch * 32) * 32; };
  if (H <= 256) return row_plan_of<OP, HF32, DF32, 1, true>(256);
  if (H <= 512) return row_plan_of<OP, HF32, DF32, 2, true>(256);
  if (H <= kLong) return row_plan_of<OP, HF32, DF32, 1, false>(threads(1));
  if (H > 16384) return {reinterpret_cast<const void*>(row_quant_long_kernel<OP, HF32, DF32>), 1024, 1};
  if constexpr (kFour) {
    if (H >= 4096 + (OP == kRowNorm)) return row_plan_of<OP, HF32, DF32, 4, false>(threads(4));
  }
  return row_plan_of<OP, HF32, DF32, 2, false>(threads(2));
}

template <int OP>
RowPlan row_plan(int H, bool hf32, bool df32) {
  if constexpr (OP == kRowNorm) {
    if (df32) return hf32 ? row_plan<OP, true, true>(H) : row_plan<OP, false, true>(H);
  }
  return hf32 ? row_plan<OP, true, false>(H) : row_plan<OP, false, false>(H);
}

}  // namespace

cudaError_t launch_row_quant(const RowQuantArgs& a, int op, bool in_f32, bool delta_f32, cudaStream_t st) {
  const RowPlan k = op == kRowNorm     ? row_plan<kRowNorm>(a.H, in_f32, delta_f32)
                    : op == kRowSwiglu ? row_plan<kRowSwiglu>(a.H, in_f32, false)
                                       : row_plan<kRowPlain>(a.H, in_f32, false);
  return launch_pdl(k.fn, (int)(((int64_t)a.T + k.rows - 1) / k.rows), k.threads, 0, st, a);
}

}  // namespace moe
