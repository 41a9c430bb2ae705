// Stage 1 for routers that score their experts by softmax or sigmoid, choose
// by biased scores and may keep only some groups of experts
// (moe_route_grouped; include/moe.h has the definition).
//
// Mathematics: s_e = sigmoid(l_e) or softmax(l)_e; c_e = s_e + b_e, raised by
// L (max c - min c) for resident experts; a group's score is the sum of its
// one or two best c; the best groups' experts are ranked by (c desc, l desc,
// e asc); the weights are the chosen experts' s.  The choice compares reals.
// It is first made in fp32, with a bound D on how far any c may be off: where
// every pair of neighbours among the k + 1 best, and the lowest kept and the
// highest dropped group, are further apart than the bounds allow, the fp32
// choice is the choice over reals.  Otherwise (about one token in six thousand
// of N(0, 1) logits with a bias: 256 experts, 4 of 8 groups) its candidates, or
// where the groups are in doubt all its experts, are compared again in 64 bits.
// Without bias and substitution the order is the logits' own, which needs no
// bound.
//
// One warp per token, lane i holding experts i, 32 + i, ...  The k + 1 best are
// found through a threshold: the (k + 1)-th largest of the 32 lanes' own
// maxima has at least k + 1 experts at or above it, and few more; those are
// ranked by counting.
//
// What bounds it: a warp's chain of dependent instructions (545 a token of 512
// plain experts, 980 of 256 with bias and groups), at 2.0 to 2.6 of 4 issue
// slots a cycle; the bytes would take 0.3 ns a token at 6.6 TB/s.  16384 tokens
// x 512 experts, softmax, k 10: 13.4 us.  4096 x 256, sigmoid with bias and 4
// of 8 groups, k 8, one wave that lasts as long as its slowest warp: 6.8 us
// where no token goes to 64 bits, 8.4 on the average of N(0, 1) logits (0.7 of
// a call's tokens go there).  One token of 512 with all of it: 4.1 us (243, 53
// and 41 us where every score and choice is made in 64 bits with a search of
// all experts per rank); with its sort and slot lookup in the launch 7.3.
#include <cfloat>
#include <climits>

#include "common.cuh"
#include "kernels.h"
#include "route_tail.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kCand = 64;  // experts ranked by counting, at most
constexpr float kLog2e = 0x1.715476p+0f;

__device__ __forceinline__ double warp_max(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v = fmax(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
// Floats as unsigned numbers of the same order.
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t b = __float_as_uint(f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ float warp_max(float v) { return unordered(__reduce_max_sync(kAll, ordered(v))); }
__device__ __forceinline__ float warp_min(float v) { return unordered(__reduce_min_sync(kAll, ordered(v))); }

__device__ __forceinline__ float exp2_of(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// (c desc, l desc, e asc)
__device__ __forceinline__ bool before(double ac, float al, int ae, double bc, float bl, int be) {
  return ac > bc || (ac == bc && (al > bl || (al == bl && ae < be)));
}

// A token's logit: NaN counts as an expert that is off.
__device__ __forceinline__ float logit(const float* row, int e) {
  const float l = row[e];
  return l == l ? l : -INFINITY;
}

// c + L (hi - lo) of a resident expert, or the sum c of n of them.  At L = 1
// the lowest meets the highest score over the reals; summed from hi downwards
// that tie is exact in 64 bits too and goes to the larger logit, not to the
// way the sum rounds.
__device__ __forceinline__ double lift_of(double c, float L, double hi, double lo, double n = 1.0) {
  if (!(hi > lo)) return c;
  const double down = __dmul_rn((double)L - 1.0, __dsub_rn(hi, lo));
  return __dadd_rn(n * hi, __dadd_rn(__dsub_rn(c, n * lo), n * down));  // n times: exact
}

// The token's choice in 64 bits: lane j (< k) gets rank j's expert and score.
// c: E doubles of shared memory of this warp.
__device__ __noinline__ void route_exact(const RouteGroupedArgs& a, const float* row, double* c, int& my_e,
                                         double& my_s) {
  const int lane = threadIdx.x & 31, E = a.E, m = E / a.G;
  double lmax = -INFINITY, sum = 0.0;
  for (int e = lane; e < E; e += 32) lmax = fmax(lmax, (double)logit(row, e));
  lmax = warp_max(lmax);
  // an expert that is off scores 0, also where every expert is
  auto score = [&](float l) -> double {
    if (l == -INFINITY) return 0.0;
    return a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - lmax);
  };
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    const double v = score(logit(row, e));
    c[e] = v;
    sum += v;
  }
  if (!a.sigmoid) sum = warp_sum(sum);
  const double scale = a.sigmoid ? 1.0 : sum > 0.0 ? 1.0 / sum : 0.0;
  double hi = -INFINITY, lo = -INFINITY;  // lo: of -c
#pragma unroll 4
  for (int e = lane; e < E; e += 32) {
    double v = c[e] * scale;
    if (a.bias) v += (double)a.bias[e];
    if (logit(row, e) == -INFINITY || !(v == v)) v = -INFINITY;
    if (v != -INFINITY) {
      hi = fmax(hi, v);
      lo = fmax(lo, -v);
    }
    c[e] = v;
  }
  bool lifted = a.L > 0.0f && a.table;
  if (lifted) {
    hi = warp_max(hi);
    lo = -warp_max(lo);
    lifted = hi > lo;
    for (int e = lane; e < E; e += 32)
      if (c[e] != -INFINITY && a.table[e] >= 0) c[e] = lift_of(c[e], a.L, hi, lo);
  }
  __syncwarp();
  if (a.top < a.G) {
    // 32 / P lanes to a group (P: groups rounded up to a power of two)
    const int lg = 5 - (a.G > 1 ? 32 - __clz(a.G - 1) : 0), lanes = 1 << lg;
    double t1 = -INFINITY, t2 = -INFINITY;
    if ((lane >> lg) < a.G) {
      const double* group = c + (lane >> lg) * m;
#pragma unroll 4
      for (int j = lane & (lanes - 1); j < m; j += lanes) {
        t2 = fmax(t2, fmin(t1, group[j]));
        t1 = fmax(t1, group[j]);
      }
    }
    for (int o = lanes >> 1; o; o >>= 1) {
      const double o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
      t2 = fmax(fmin(t1, o1), fmax(t2, o2));
      t1 = fmax(t1, o1);
    }
    double mine = t1;
    if (a.gtop == 2) {
      // Scores, biases and lifts are summed each for itself: two groups whose
      // sums are equal over the reals because they share them out differently
      // (the same logits, one expert of each resident) are equal here too.
      const int g0 = (lane >> lg) * m;
      int e1 = INT_MAX, e2 = INT_MAX;  // the lowest experts with these values
      if ((lane >> lg) < a.G)
        for (int j = lane & (lanes - 1); j < m && e1 == INT_MAX; j += lanes)
          if (c[g0 + j] == t1) e1 = g0 + j;
      for (int o = lanes >> 1; o; o >>= 1) e1 = min(e1, __shfl_xor_sync(kAll, e1, o));
      if ((lane >> lg) < a.G)
        for (int j = lane & (lanes - 1); j < m && e2 == INT_MAX; j += lanes)
          if (c[g0 + j] == t2 && g0 + j != e1) e2 = g0 + j;
      for (int o = lanes >> 1; o; o >>= 1) e2 = min(e2, __shfl_xor_sync(kAll, e2, o));
      mine = -INFINITY;  // where one of the two is off
      if (t2 > -INFINITY && e1 < E && e2 < E) {
        mine = __dadd_rn(__dmul_rn(score(logit(row, e1)), scale), __dmul_rn(score(logit(row, e2)), scale));
        if (a.bias) mine = __dadd_rn(mine, __dadd_rn((double)a.bias[e1], (double)a.bias[e2]));
        const int n = lifted ? (a.table[e1] >= 0 ? 1 : 0) + (a.table[e2] >= 0 ? 1 : 0) : 0;
        if (n) mine = lift_of(mine, a.L, hi, lo, (double)n);
      }
    }
    mine = __shfl_sync(kAll, mine, (lane << lg) & 31);  // lane g: group g's score
    int better = 0;
    for (int g = 0; g < a.G; ++g) {
      const double v = __shfl_sync(kAll, mine, g);
      better += (v > mine || (v == mine && g < lane)) ? 1 : 0;
    }
    const uint32_t keep = __ballot_sync(kAll, lane < a.G && better < a.top);
    __syncwarp();
    for (int e = lane; e < E; e += 32)
      if (!((keep >> (e / m)) & 1u)) c[e] = NAN;  // out of the choice
  }
  // each lane's best of its experts, looked for again only where it was taken
  double mc;
  float ml;
  int me;
  auto best = [&]() {
    mc = -INFINITY;
    me = INT_MAX;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) {
      const double v = c[e];  // NaN: out of the choice
      const bool first = me == INT_MAX && v == v;
      if (first || v > mc || (v == mc && logit(row, e) > logit(row, me))) {
        mc = v;
        me = e;
      }
    }
    ml = me < E ? logit(row, me) : -INFINITY;
  };
  best();
  for (int j = 0; j < a.k; ++j) {
    double bc = mc;
    float bl = ml;
    int be = me;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const double oc = __shfl_xor_sync(kAll, bc, o);
      const float ol = __shfl_xor_sync(kAll, bl, o);
      const int oe = __shfl_xor_sync(kAll, be, o);
      if (before(oc, ol, oe, bc, bl, be)) {
        bc = oc;
        bl = ol;
        be = oe;
      }
    }
    if (be == me) {  // k experts are left in the kept groups: be is one of them
      c[be] = NAN;
      best();
    }
    if (lane == j) {
      my_e = be;
      my_s = score(logit(row, be)) * scale;
    }
    __syncwarp();
  }
}

// Where a warp keeps the c of expert e for the groups' scores: four words
// after every 32, so that the lanes of eight groups of 32 read apart.
__host__ __device__ constexpr int spread(int e) { return e + 4 * (e >> 5); }

// An expert to be ranked.
struct Cand {
  double c;
  float l;
  int e;
};

// Shared memory of a warp: the c (spread fp32, or 64 bits), or the candidates in 64 bits; then what is ranked.
__host__ __device__ constexpr size_t c_bytes(int E) { return 8 * E > 16 * kCand ? (size_t)round_up(8 * E, 16) : 16 * kCand; }
__host__ __device__ constexpr size_t warp_bytes(int E) { return c_bytes(E) + 12 * kCand; }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max_abs3(float m, float a, float b) {  // NaN if one of them is
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}

// The token's choice in fp32, or of the candidates that fp32 leaves in 64
// bits; false where that does not settle it.  my_e: lane j's expert (rank j);
// lmax, sum: the largest logit and the softmax's denominator.  FULL: E = 32 NPL,
// and the lanes hold four experts side by side.  PLAIN: no bias, substitution
// or groups (code and registers of their own: 16384 x 512 takes 13.4 us, 16.1
// with all of it in one kernel).
template <int NPL, bool FULL, bool PLAIN>
__device__ __forceinline__ bool route_fast(const RouteGroupedArgs& a, const float* row, char* sm, int& my_e, float& lmax,
                                           float& sum) {
  const int lane = threadIdx.x & 31, E = a.E, k = a.k;
  const bool lifted = !PLAIN && a.L > 0.0f && a.table, by_l = PLAIN || (!a.bias && !lifted);
  const bool groups = !PLAIN && a.top < a.G;
  float* const sc = reinterpret_cast<float*>(sm);
  Cand* const wide = reinterpret_cast<Cand*>(sm);
  float* const skey = reinterpret_cast<float*>(sm + c_bytes(E));
  int* const sid = reinterpret_cast<int*>(skey + kCand);
  int* const cand = sid + kCand;
  auto expert = [&](int i) { return FULL ? 128 * (i >> 2) + 4 * lane + (i & 3) : 32 * i + lane; };
  auto have = [&](int i) { return FULL || 32 * i + lane < E; };
  float key[NPL], bias[NPL];
  uint32_t resident = 0;
  if constexpr (FULL) {
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(row + 32 * i + 4 * lane);
      key[i] = v.x, key[i + 1] = v.y, key[i + 2] = v.z, key[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NPL; ++i) key[i] = have(i) ? row[expert(i)] : -INFINITY;
  }
  if (!PLAIN && a.bias) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) bias[i] = have(i) ? a.bias[expert(i)] : 0.0f;
  }
  if (lifted) {
#pragma unroll
    for (int i = 0; i < NPL; ++i) resident |= (have(i) && a.table[expert(i)] >= 0 ? 1u : 0u) << i;
  }
  float big = 0.0f;
  lmax = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; i += 2) {
    big = max_abs3(big, have(i) ? key[i] : 0.0f, have(i + 1) ? key[i + 1] : 0.0f);
    lmax = max3(lmax, key[i], key[i + 1]);
  }
  if (__any_sync(kAll, !(big < INFINITY))) return false;  // an expert that is off, or a logit without order
  sum = 0.0f;
  float D = 0.0f, inv = 1.0f, lift = 0.0f, most = 0.0f, hi = -INFINITY, lo = -INFINITY;  // lo: of -c at first
  if (!a.sigmoid) lmax = warp_max(lmax);
  // a score before the softmax's quotient; every rounding is spelled out, so
  // that the candidates' c are the same numbers when they are computed again
  auto term = [&](float l) {
    return a.sigmoid ? rcp(__fadd_rn(1.0f, exp2_of(__fmul_rn(l, -kLog2e))))
                     : exp2_of(__fmul_rn(__fsub_rn(l, lmax), kLog2e));
  };
  if (by_l && !groups) {
    if (!a.sigmoid && !a.renorm) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) sum += term(key[i]);  // 0 past E
      sum = warp_sum(sum);
    }
  } else {
    // How far a score may be off, in 2^-24: 1 / (1 + 2^x) with x rounded once
    // and 2^x off by 2^-22: 1 (of 2^x, halved twice) + 1/4 (of x) + 1 + 2 (the
    // sum, the reciprocal).  A softmax's terms are off by 4 + 1.4 |x| (|x| 2^x
    // stays below 1), its sum by as much, |x| below log2 E on the average, and
    // by a tree of additions, its quotient by 3: 40 of the largest.  The sum's
    // error is every score's and does not count where no bias is added: 8.
    float s[NPL], unit = 5.0f * 0x1p-24f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) s[i] = term(key[i]);
    if (!a.sigmoid) {
      float part[NPL];  // 0 past E
#pragma unroll
      for (int i = 0; i < NPL; ++i) part[i] = s[i];
#pragma unroll
      for (int o = NPL / 2; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) part[i] += part[i + o];
      sum = warp_sum(part[0]);
      inv = rcp(sum);
#pragma unroll
      for (int i = 0; i < NPL; ++i) s[i] = __fmul_rn(s[i], inv);
      unit = (a.bias ? 40.0f : 8.0f) * 0x1p-24f * inv;
    }
    if (a.bias) {  // c, before the lift
#pragma unroll
      for (int i = 0; i < NPL; ++i) s[i] = __fadd_rn(s[i], bias[i]);
    }
#pragma unroll
    for (int i = 0; i < NPL; i += 2) {
      hi = max3(hi, have(i) ? s[i] : -INFINITY, have(i + 1) ? s[i + 1] : -INFINITY);
      lo = max3(lo, have(i) ? -s[i] : -INFINITY, have(i + 1) ? -s[i + 1] : -INFINITY);
    }
    hi = warp_max(hi);
    lo = -warp_max(lo);
    if (!(hi < INFINITY && lo > -INFINITY)) return false;
    if (lifted) {
      lift = a.L * (hi - lo);
#pragma unroll
      for (int i = 0; i < NPL; ++i)
        if ((resident >> i) & 1u) s[i] = __fadd_rn(s[i], lift);
    }
    // the sums with the bias and the lift round to steps of the largest of them
    most = fmaxf(fabsf(hi), fabsf(lo));
    D = lifted ? unit * (1.0f + 2.0f * a.L) + 0x1p-22f * (most + lift) : unit + 0x1.1p-24f * most;
    if (groups) {
      if constexpr (FULL) {
#pragma unroll
        for (int i = 0; i < NPL; i += 4)
          *reinterpret_cast<float4*>(sc + spread(expert(i))) = make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i)
          if (have(i)) sc[spread(expert(i))] = s[i];
      }
    }
    if (!by_l) {
#pragma unroll
      for (int i = 0; i < NPL; ++i) key[i] = have(i) ? s[i] : -INFINITY;
    }
  }
  if (groups) {
    // 32 / P lanes to a group (P: groups rounded up to a power of two)
    const int m = E / a.G, lg = 5 - (a.G > 1 ? 32 - __clz(a.G - 1) : 0), lanes = 1 << lg;
    const int g = lane >> lg;
    float t1 = -INFINITY, t2 = -INFINITY;
    __syncwarp();
    if (g < a.G)
      for (int j = lane & (lanes - 1); j < m; j += lanes) {
        const float v = sc[spread(g * m + j)];
        t2 = fmaxf(t2, fminf(t1, v));
        t1 = fmaxf(t1, v);
      }
    for (int o = lanes >> 1; o; o >>= 1) {
      const float o1 = __shfl_xor_sync(kAll, t1, o), o2 = __shfl_xor_sync(kAll, t2, o);
      t2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
      t1 = fmaxf(t1, o1);
    }
    const float mine = a.gtop == 2 ? t1 + t2 : t1;
    int better = 0;
    for (int h = 0; h < a.G; ++h) {
      const float v = __shfl_sync(kAll, mine, h << lg);
      better += (v > mine || (v == mine && h < g)) ? 1 : 0;
    }
    const bool kept = g < a.G && better < a.top;
    const uint32_t lanes_kept = __ballot_sync(kAll, kept);
    const float low = warp_min(kept ? mine : INFINITY), high = warp_max(g < a.G && !kept ? mine : -INFINITY);
    // the sum of two c is off by 2 D and its own rounding
    if (!(low - high > 4.0f * D + 0x1p-22f * (most + lift))) return false;
    const uint32_t inv_m = ((1u << 22) + m - 1) / m;  // e / m = e inv_m >> 22 for e < 1024
    const bool fours = FULL && (m & 3) == 0;          // four experts side by side share a group
#pragma unroll
    for (int i = 0; i < NPL; i += 4) {
      bool in = (lanes_kept >> ((((uint32_t)expert(i) * inv_m >> 22) << lg) & 31u)) & 1u;
      if (!in) key[i] = -INFINITY;
#pragma unroll
      for (int j = 1; j < 4; ++j) {
        if (!fours) in = (lanes_kept >> ((((uint32_t)expert(i + j) * inv_m >> 22) << lg) & 31u)) & 1u;
        if (!in) key[i + j] = -INFINITY;
      }
    }
  }
  // threshold: of the lanes' maxima, the largest that is left after k have
  // been taken away (equal ones together: then it is lower, which does no harm)
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < NPL; i += 2) top = max3(top, key[i], key[i + 1]);
  uint32_t rest = ordered(top), most_left = 0u;
  for (int j = 0; j <= k; ++j) {
    most_left = __reduce_max_sync(kAll, rest);
    if (rest == most_left) rest = 0u;
  }
  const float tau = most_left > ordered(-FLT_MAX) ? unordered(most_left) : -FLT_MAX;
  uint32_t in = 0;
#pragma unroll
  for (int i = 0; i < NPL; ++i) in |= (key[i] >= tau ? 1u : 0u) << i;
  int cnt = 0;
  while (const uint32_t who = __ballot_sync(kAll, in != 0)) {  // every lane's next expert
    const int at = cnt + __popc(who & ((1u << lane) - 1u));
    if (in && at < kCand) cand[at] = expert(__ffs(in) - 1);
    in &= in - 1;
    cnt += __popc(who);
  }
  if (cnt > kCand || cnt < k) return false;
  __syncwarp();
  // the candidates' c again, by the same arithmetic, and their ranks
  auto choice = [&](int e) {
    const float l = row[e];
    if (by_l) return l;
    float c = term(l);
    if (!a.sigmoid) c = __fmul_rn(c, inv);
    if (a.bias) c = __fadd_rn(c, a.bias[e]);
    return lifted && a.table[e] >= 0 ? __fadd_rn(c, lift) : c;
  };
  if (cnt <= 32) {
    const int e = lane < cnt ? cand[lane] : INT_MAX;
    const float c = lane < cnt ? choice(e) + 0.0f : -INFINITY;  // -0 as +0
    int r = 0;  // lanes without a candidate hold -inf and come before none
#pragma unroll
    for (int j = 0; j < 16; ++j) r += __shfl_sync(kAll, c, j) > c ? 1 : 0;
    if (cnt > 16) {
#pragma unroll
      for (int j = 16; j < 32; ++j) r += __shfl_sync(kAll, c, j) > c ? 1 : 0;
    }
    const uint32_t alike = __match_any_sync(kAll, __float_as_uint(c));
    if (__any_sync(kAll, lane < cnt && alike != (1u << lane)))
      for (int j = 0; j < cnt; ++j) {
        const int o = __shfl_sync(kAll, e, j);
        r += ((alike >> j) & 1u) && o < e ? 1 : 0;
      }
    if (lane < cnt) {
      skey[r] = c;
      sid[r] = e;
    }
  } else {
    for (int h = lane; h < cnt; h += 32) skey[h] = choice(cand[h]);
    __syncwarp();
    int r[kCand / 32] = {}, e[kCand / 32];
    float c[kCand / 32];
#pragma unroll
    for (int h = 0; h < kCand / 32; ++h) {
      const int at = 32 * h + lane;
      if (at >= cnt) break;
      e[h] = cand[at];
      c[h] = skey[at];
      for (int j = 0; j < cnt; ++j) r[h] += skey[j] > c[h] || (skey[j] == c[h] && cand[j] < e[h]) ? 1 : 0;
    }
    __syncwarp();
#pragma unroll
    for (int h = 0; h < kCand / 32; ++h)
      if (32 * h + lane < cnt) {
        skey[r[h]] = c[h];
        sid[r[h]] = e[h];
      }
  }
  __syncwarp();
  my_e = lane < k ? sid[lane] : 0;
  bool ok = true;
  if (!by_l && lane < k && lane + 1 < cnt) {
    // alike in all that counts: the lower one first, as they are
    auto alike = [&](int f) {
      return row[my_e] == row[f] && (!a.bias || a.bias[my_e] == a.bias[f]) &&
             (!lifted || (a.table[my_e] >= 0) == (a.table[f] >= 0));
    };
    ok = skey[lane] - skey[lane + 1] > 2.0f * D;
    if (skey[lane] == skey[lane + 1]) {
      ok = alike(sid[lane + 1]);
      if (ok && lane == k - 1) {  // those behind the last place that are alike, then the first that is not
        int j = k + 1;
        while (j < cnt && skey[j] == skey[lane] && alike(sid[j])) ++j;
        ok = j < cnt ? skey[lane] - skey[j] > 2.0f * D : tau == -FLT_MAX || skey[lane] - tau > 2.0f * D;
      }
    }
  }
  if (__all_sync(kAll, ok)) return true;
  // the candidates in 64 bits, if none that is not among them can be better than the k-th
  if (!(tau == -FLT_MAX || skey[k - 1] - tau > 2.0f * D)) return false;
  double total = 1.0;
  const double lm = (double)lmax;
  if (!a.sigmoid) {
    total = 0.0;
#pragma unroll 4
    for (int e = lane; e < E; e += 32) total += exp((double)row[e] - lm);
    total = warp_sum(total);
  }
  const double quotient = 1.0 / total;
  auto exact = [&](int e) {  // c before the lift, as route_exact has it
    const double l = (double)row[e], v = a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - lm) * quotient;
    return a.bias ? v + (double)a.bias[e] : v;
  };
  double top64 = -INFINITY, low64 = -INFINITY;  // low64: of -c at first
  if (lifted) {
    for (int e = lane; e < E; e += 32) {
      float c = term(row[e]);
      if (!a.sigmoid) c = __fmul_rn(c, inv);
      if (a.bias) c = __fadd_rn(c, a.bias[e]);
      if (c > hi - 2.0f * D) top64 = fmax(top64, exact(e));
      if (c < lo + 2.0f * D) low64 = fmax(low64, -exact(e));
    }
    top64 = warp_max(top64);
    low64 = -warp_max(low64);
  }
  __syncwarp();
  for (int j = lane; j < cnt; j += 32) {
    const int e = cand[j];
    const double c = exact(e);
    wide[j] = Cand{lifted && a.table[e] >= 0 ? lift_of(c, a.L, top64, low64) : c, row[e], e};
  }
  __syncwarp();
  for (int j = lane; j < cnt; j += 32) {
    const Cand me = wide[j];
    int r = 0;
    for (int o = 0; o < cnt; ++o) r += before(wide[o].c, wide[o].l, wide[o].e, me.c, me.l, me.e) ? 1 : 0;
    sid[r] = me.e;
  }
  __syncwarp();
  my_e = lane < k ? sid[lane] : 0;
  return true;
}

// One token by one warp; sm: warp_bytes(E) of shared memory.
template <int NPL, bool FULL, bool PLAIN>
__device__ __forceinline__ void route_token(const RouteGroupedArgs& a, int t, char* sm) {
  const int lane = threadIdx.x & 31;
  const float* row = a.logits + (size_t)t * a.E;
  int my_e = 0;
  float w = 0.0f, lmax = 0.0f, sum = 0.0f;
  if (route_fast<NPL, FULL, PLAIN>(a, row, sm, my_e, lmax, sum)) {
    const float l = lane < a.k ? row[my_e] : 0.0f;
    if (lane < a.k) {
      if (a.sigmoid) {
        w = __fdiv_rn(1.0f, 1.0f + expf(-l));
      } else {  // exp(l - lmax) with what the difference's rounding leaves out
        const float d = __fsub_rn(l, lmax), b = __fsub_rn(d, l);
        const float rest = __fsub_rn(__fsub_rn(l, __fsub_rn(d, b)), __fadd_rn(lmax, b)), p = expf(d);
        w = fmaf(p, rest, p);
      }
    }
    if (__any_sync(kAll, lane < a.k && !(w > 0x1p-100f))) {  // scores that fp32 hardly holds, or not
      const double s = lane >= a.k ? 0.0 : a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)lmax);
      const double den = a.renorm ? warp_sum(s) : a.sigmoid ? 1.0 : (double)sum;
      w = den > 0.0 ? (float)((double)a.scale * (s / den)) : 0.0f;
    } else {
      const float den = a.renorm ? warp_sum(w) : a.sigmoid ? 1.0f : sum;
      w = a.scale * __fdiv_rn(w, den);
    }
  } else {
    double s = 0.0;
    __syncwarp();
    route_exact(a, row, reinterpret_cast<double*>(sm), my_e, s);
    const double den = a.renorm ? warp_sum(lane < a.k ? s : 0.0) : 1.0;
    w = den > 0.0 ? (float)((double)a.scale * (s / den)) : 0.0f;
  }
  const int ks = a.k + a.ns;  // output row: the top-k, then the shared experts
  if (lane < a.k) {
    a.ids[(size_t)t * ks + lane] = my_e;
    a.w[(size_t)t * ks + lane] = w;
  }
  if (lane < a.ns) {
    a.ids[(size_t)t * ks + a.k + lane] = a.E + lane;
    a.w[(size_t)t * ks + a.k + lane] = a.shared_w ? a.shared_w[t] : 1.0f;
  }
}

template <int NPL, bool FULL, bool PLAIN>
__global__ void __launch_bounds__(256, PLAIN && NPL <= 16 ? 5 : 1) route_grouped_kernel(const __grid_constant__ RouteGroupedArgs a) {
  extern __shared__ __align__(16) char route_smem[];
  const int warp = threadIdx.x >> 5, t = blockIdx.x * (blockDim.x >> 5) + warp;
  pdl_wait();
  pdl_launch_dependents();
  if (t < a.T) route_token<NPL, FULL, PLAIN>(a, t, route_smem + warp * warp_bytes(a.E));
}

// One decode token: its routing by warp 0, then the sort and the slot lookup
// of its experts by the block, as moe_sort and moe_slot_lookup write them.
template <int NPL, bool FULL>
__global__ void __launch_bounds__(256)
    route_grouped_sort_lookup_kernel(const __grid_constant__ RouteGroupedArgs a, const SortLookupArgs o) {
  extern __shared__ __align__(16) char route_smem[];
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x < 32) route_token<NPL, FULL, false>(a, 0, route_smem);
  sort_lookup_token(a.ids, a.k + a.ns, a.E + a.ns, o);
}

bool is_plain(const RouteGroupedArgs& a) { return !a.bias && !(a.L > 0.0f) && a.top == a.G; }

template <int NPL, bool FULL>
const void* route_kernel_of(const RouteGroupedArgs& a, bool sort) {
  if (sort) return reinterpret_cast<const void*>(route_grouped_sort_lookup_kernel<NPL, FULL>);
  if (is_plain(a))
    return reinterpret_cast<const void*>(route_grouped_kernel<NPL, FULL, true>);
  return reinterpret_cast<const void*>(route_grouped_kernel<NPL, FULL, false>);
}

template <int NPL>
const void* route_kernel_of(const RouteGroupedArgs& a, bool sort) {
  return a.E == 32 * NPL && reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 ? route_kernel_of<NPL, true>(a, sort)
                                                                            : route_kernel_of<NPL, false>(a, sort);
}

const void* route_kernel_of(const RouteGroupedArgs& a, bool sort) {
  return a.E <= 128   ? route_kernel_of<4>(a, sort)
         : a.E <= 256 ? route_kernel_of<8>(a, sort)
         : a.E <= 512 ? route_kernel_of<16>(a, sort)
                      : route_kernel_of<32>(a, sort);
}

}  // namespace

cudaError_t launch_route_grouped(const RouteGroupedArgs& a, int num_sms, cudaStream_t st) {
  // few tokens spread over the SMs; no more than 48 KB of shared memory a block.
  // With a bias, groups or substitution a thread takes 68 registers, of which
  // an SM holds 3 blocks of 8 warps or 7 of 4: 4096 x 256 takes 8.8 / 7.7 us
  // with blocks of 8 / 4 (one wave), 8192 x 256 13.9 / 12.9, 2048 x 256 6.0 /
  // 5.6; the plain kernel (48 registers) 13.3 / 14.1 at 16384 x 512.
  const int most = is_plain(a) ? 8 : 4;
  int warps = a.T / num_sms;
  warps = warps < 1 ? 1 : warps > most ? most : warps;
  while (warps > 1 && warps * warp_bytes(a.E) > 48 * 1024) --warps;
  return launch_pdl(route_kernel_of(a, false), (a.T + warps - 1) / warps, 32 * warps, warps * warp_bytes(a.E), st, a);
}

cudaError_t launch_route_grouped_sort_lookup(const RouteGroupedArgs& a, const SortLookupArgs& o, cudaStream_t st) {
  return launch_pdl(route_kernel_of(a, true), 1, 256, warp_bytes(a.E), st, a, o);
}

}  // namespace moe
