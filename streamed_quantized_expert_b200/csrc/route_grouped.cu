// Stage 1 for routers that score their experts by softmax or sigmoid, choose
// by biased scores and may keep only some groups of experts
// (moe_route_grouped; include/moe.h has the definition).
//
// Mathematics: s_e = sigmoid(l_e) or softmax(l)_e; c_e = s_e + b_e, raised by
// L (max c - min c) for resident experts; a group's score is the sum of its
// one or two best c; the best groups' experts are ranked by (c desc, l desc,
// e asc); the weights are the chosen experts' s.  The choice is a comparison
// of reals, so it is computed in 64 bits: scores that differ in the 25th bit
// are told apart, and equal ones go to the lower expert.
//
// One warp per token, lane i holding experts i, 32 + i, ...
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ double warp_min(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmin(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// (c desc, l desc, e asc)
__device__ __forceinline__ bool before(double ac, float al, int ae, double bc, float bl, int be) {
  return ac > bc || (ac == bc && (al > bl || (al == bl && ae < be)));
}

// The best expert among those whose bit of `out` is clear; its score too.
template <int NPL>
__device__ __forceinline__ int warp_best(const double (&c)[NPL], const float (&l)[NPL], uint32_t out, int E) {
  const int lane = threadIdx.x & 31;
  double bc = -INFINITY;
  float bl = -INFINITY;
  int be = INT_MAX;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = 32 * i + lane;
    if (e < E && !((out >> i) & 1u) && before(c[i], l[i], e, bc, bl, be)) {
      bc = c[i];
      bl = l[i];
      be = e;
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const double oc = __shfl_xor_sync(0xffffffffu, bc, o);
    const float ol = __shfl_xor_sync(0xffffffffu, bl, o);
    const int oe = __shfl_xor_sync(0xffffffffu, be, o);
    if (before(oc, ol, oe, bc, bl, be)) {
      bc = oc;
      bl = ol;
      be = oe;
    }
  }
  return be;
}

template <int NPL>
__global__ void __launch_bounds__(128) route_grouped_kernel(const RouteGroupedArgs a) {
  const int lane = threadIdx.x & 31;
  const int t = (int)((blockIdx.x * (unsigned)blockDim.x + threadIdx.x) >> 5);
  pdl_wait();
  pdl_launch_dependents();
  if (t >= a.T) return;
  const float* row = a.logits + (size_t)t * a.E;
  const int E = a.E, m = E / a.G;
  float l[NPL];
  double s[NPL], c[NPL];
  float lmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = 32 * i + lane;
    l[i] = e < E ? row[e] : -INFINITY;
    if (!(l[i] == l[i])) l[i] = -INFINITY;  // a NaN counts as an expert that is off
    lmax = fmaxf(lmax, l[i]);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) lmax = fmaxf(lmax, __shfl_xor_sync(0xffffffffu, lmax, o));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    // an expert that is off scores 0, also where every expert is
    s[i] = l[i] == -INFINITY ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-(double)l[i])) : exp((double)l[i] - (double)lmax);
    sum += s[i];
  }
  if (!a.sigmoid) {
    sum = warp_sum(sum);
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = sum > 0.0 ? s[i] / sum : 0.0;
  }
  double cmax = -INFINITY, cmin = INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; ++i) {
    const int e = 32 * i + lane;
    c[i] = -INFINITY;
    if (e < E && l[i] != -INFINITY) {
      c[i] = a.bias ? s[i] + (double)a.bias[e] : s[i];
      if (!(c[i] == c[i])) c[i] = -INFINITY;
      if (c[i] != -INFINITY) {
        cmax = fmax(cmax, c[i]);
        cmin = fmin(cmin, c[i]);
      }
    }
  }
  if (a.L > 0.0f && a.table) {
    cmax = warp_max(cmax);
    cmin = warp_min(cmin);
    const double lift = cmax > cmin ? __dmul_rn((double)a.L, cmax - cmin) : 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = 32 * i + lane;
      if (e < E && c[i] != -INFINITY && a.table[e] >= 0) c[i] = __dadd_rn(c[i], lift);
    }
  }
  uint32_t out = 0;  // experts taken, or in a group that is not kept
  if (a.top < a.G) {
    double mine = -INFINITY;  // lane g: group g's score
    for (int g = 0; g < a.G; ++g) {
      uint32_t other = 0;
#pragma unroll
      for (int i = 0; i < NPL; ++i) other |= ((32 * i + lane) / m != g ? 1u : 0u) << i;
      double v = 0.0;
      for (int j = 0; j < a.gtop; ++j) {
        const int b = warp_best<NPL>(c, l, other, E);
        double cb = -INFINITY;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (32 * i + lane == b) {
            cb = c[i];
            other |= 1u << i;
          }
        v += warp_max(cb);
      }
      if (lane == g) mine = v;
    }
    int better = 0;
    for (int g = 0; g < a.G; ++g) {
      const double v = __shfl_sync(0xffffffffu, mine, g);
      better += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    const uint32_t keep = __ballot_sync(0xffffffffu, lane < a.G && better < a.top);
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
      const int e = 32 * i + lane;
      if (e < E && !((keep >> (e / m)) & 1u)) out |= 1u << i;
    }
  }
  int my_e = 0;
  double my_s = 0.0;
  for (int j = 0; j < a.k; ++j) {
    const int b = warp_best<NPL>(c, l, out, E);
    double sb = 0.0;
#pragma unroll
    for (int i = 0; i < NPL; ++i)
      if (32 * i + lane == b) {
        sb = s[i];
        out |= 1u << i;
      }
    sb = warp_max(sb);
    if (lane == j) {
      my_e = b;
      my_s = sb;
    }
  }
  double den = 1.0;
  if (a.renorm) den = warp_sum(my_s);
  const int ks = a.k + a.ns;  // output row: the top-k, then the shared experts
  if (lane < a.k) {
    a.ids[(size_t)t * ks + lane] = my_e;
    a.w[(size_t)t * ks + lane] = den > 0.0 ? (float)((double)a.scale * (my_s / den)) : 0.0f;
  }
  if (lane < a.ns) {
    a.ids[(size_t)t * ks + a.k + lane] = E + lane;
    a.w[(size_t)t * ks + a.k + lane] = a.shared_w ? a.shared_w[t] : 1.0f;
  }
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGroupedArgs& a, cudaStream_t st) {
  const void* kern = a.E <= 128   ? reinterpret_cast<const void*>(route_grouped_kernel<4>)
                     : a.E <= 256 ? reinterpret_cast<const void*>(route_grouped_kernel<8>)
                     : a.E <= 512 ? reinterpret_cast<const void*>(route_grouped_kernel<16>)
                                  : reinterpret_cast<const void*>(route_grouped_kernel<32>);
  return launch_pdl(kern, (a.T + 3) / 4, 128, 0, st, a);
}

}  // namespace moe
