// Product of 8-bit integer rows with a scale per token and per output
// (moe_int_matmul): y[t][n] = add[t][n] + row_w[t] xs[t] ws[n] sum_k xq[t][k] wq[n][k].
//
// The sum is a whole number of at most 2^30 (K <= 65,536), so int32
// accumulation is exact in any order and any split of K gives the same bits;
// the scales are applied once to each sum.
//
// Up to 16 tokens (32 of few weights) the weight bytes bound the call:
// im_rows_kernel streams them through mma.sync, one block per 16 outputs (1 x
// 4096 x 8192 with fp32 sums: 7.5 us, 4.5 TB/s with the launch in it).  Above,
// im_tc_kernel runs on tcgen05 (kind::i8, s32 accumulators in TMEM) fed by
// TMA, with the weight rows as the MMA's 128-row side so that a few dozen
// tokens fill its other side (48 x 5003 x 2048: 7.0 us), and im_pair_kernel
// with two CTAs to a tile where chunks are long (4096 x 8192 x 4096: 90 us, 3.0
// POP/s; 106 us over seconds, when the card's power limit lowers its clock).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "common.cuh"
#include "ffn_common.cuh"
#include "kernels.h"

namespace moe {
namespace {

// Products rounded one by one (never joined with the sum that follows): every
// kernel gives an output the same bits.
__device__ __forceinline__ float im_scaled(int acc, float xs, float ws) {
  return __fmul_rn((float)acc, __fmul_rn(xs, ws));
}

__device__ __forceinline__ float im_token_scale(const IntMatmulArgs& a, int t) {
  return a.row_w ? __fmul_rn(a.xs[t], a.row_w[t]) : a.xs[t];
}

__device__ __forceinline__ void im_store(const IntMatmulArgs& a, int t, int n, float v) {
  const int64_t at = (int64_t)t * a.N + n;
  if (a.add) v += a.add[at];
  if (a.y_f32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<uint16_t*>(a.y)[at] = f32_to_bf16_rne(v);
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
// Tokens the streaming kernel takes, and takes where the weights are few: 24
// tokens x 2048 x 768 run in 3.1 us here and 3.9 on the tensor-core tiles, x
// 4096 x 2048 in 5.3 and 5.9, x 4096 x 8192 in 10.8 and 10.3.
constexpr int kRowsTokens = 16, kRowsMaxTokens = 32;
constexpr int64_t kRowsMaxWeights = 1 << 23;
// 128-input units a warp keeps in flight; the registers hold fewer next to more token tiles
__host__ __device__ constexpr int rows_depth(int nt) { return nt == 1 ? 4 : nt == 2 ? 2 : 1; }

// D (16 x 8, s32) += A (16 x 32, s8, row) . B (32 x 8, s8, column).
__device__ __forceinline__ void mma_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 ld_stream(const int8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// One block: 16 outputs, up to 8 NT tokens, the whole of K, its W warps taking
// units of 128 inputs in turn.  Lane (g, q) loads bytes 16 q and 64 + 16 q of
// the unit's rows g and g + 8 and of token g (whole 128-byte lines per row);
// they are the fragments of four MMAs over inputs that both operands permute
// alike: bytes 0..7 of the lanes' 16 are one MMA's inputs, 8..15 the next one's.
// A ring of rows_depth units in registers keeps 2 KB a unit and warp on the
// way (128 KB an SM at two blocks of eight warps: what 6.5 TB/s needs at HBM
// latency).  Rows past N and tokens past T read the last one's and are not
// stored.  The warps' sums meet in shared memory.
template <int NT, int W>
__global__ void __launch_bounds__(32 * W, 16 / W) im_rows_kernel(const IntMatmulArgs a) {
  constexpr int kDepth = rows_depth(NT);
  __shared__ int s_acc[W][NT][4][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
  const int n0 = blockIdx.x * 16, U = (a.K + 127) / 128;
  const int8_t* wa = a.wq + (int64_t)min(n0 + g, a.N - 1) * a.K + 16 * q;
  const int8_t* wb = a.wq + (int64_t)min(n0 + g + 8, a.N - 1) * a.K + 16 * q;
  const int8_t* xp[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xp[j] = a.xq + (int64_t)min(8 * j + g, a.T - 1) * a.K + 16 * q;
  pdl_wait();
  pdl_launch_dependents();
  int acc[NT][4] = {};
  uint4 w[kDepth][4], x[kDepth][NT][2];
  auto load = [&](int u, uint4 (&wv)[4], uint4 (&xv)[NT][2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = 128 * u + 64 * h;  // this lane's 16 inputs: k + 16 q ..; K is a multiple of 16
      const bool in = u < U && k + 16 * q < a.K;
      wv[2 * h] = in ? ld_stream(wa + k) : make_uint4(0u, 0u, 0u, 0u);
      wv[2 * h + 1] = in ? ld_stream(wb + k) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        if (in) xv[j][h] = *reinterpret_cast<const uint4*>(xp[j] + k);  // else any value: its weights are 0
    }
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) load(warp + i * W, w[i], x[i]);
  for (int u0 = warp; u0 < U; u0 += kDepth * W) {
#pragma unroll
    for (int i = 0; i < kDepth; ++i) {
      if (u0 + i * W >= U) break;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 va = w[i][2 * h], vb = w[i][2 * h + 1];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          mma_s8(acc[j], va.x, vb.x, va.y, vb.y, x[i][j][h].x, x[i][j][h].y);
          mma_s8(acc[j], va.z, vb.z, va.w, vb.w, x[i][j][h].z, x[i][j][h].w);
        }
      }
      load(u0 + (kDepth + i) * W, w[i], x[i]);
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) s_acc[warp][j][i][lane] = acc[j][i];
  __syncthreads();
  // accumulator i of lane (g, q): output g + 8 (i / 2), token 2 q + i % 2
  for (int o = threadIdx.x; o < NT * 128; o += 32 * W) {
    const int n = o & 15, t = o >> 4, j = t >> 3, i = 2 * (n >> 3) + (t & 1), l = 4 * (n & 7) + ((t & 7) >> 1);
    if (n0 + n >= a.N || t >= a.T) continue;
    int sum = 0;
#pragma unroll
    for (int v = 0; v < W; ++v) sum += s_acc[v][j][i][l];
    im_store(a, t, n0 + n, im_scaled(sum, im_token_scale(a, t), a.ws[n0 + n]));
  }
}

// ---------------------------------------------------------------------------
// many tokens
// ---------------------------------------------------------------------------
constexpr int kTcBM = 128;  // outputs of a tile (MMA M)
constexpr int kTcBK = 128;  // inputs of a stage: one 128-byte swizzled row per output and token
constexpr int kTcProdWarp = 0, kTcMmaWarp = 1, kTcEpiWarp0 = 4;
// the stores of a 128 x 256 tile take 8 warps longer than the MMAs of 512 inputs; a split call's CTAs share an SM
__host__ __device__ constexpr int tc_epi_warps(bool split) { return split ? 8 : 16; }
__host__ __device__ constexpr int tc_threads(bool split) { return 32 * (kTcEpiWarp0 + tc_epi_warps(split)); }
constexpr int kTcSplitMaxTokens = 64;  // token tiles whose K may be split
constexpr int kTcSplitCtas = 256;      // CTAs of a split call: clusters of up to 8, two CTAs to an SM
__host__ __device__ constexpr int tc_stages(int nb) { return nb == 256 ? 4 : nb == 128 ? 6 : 8; }
__host__ __device__ constexpr int tc_stage_bytes(int nb) { return (kTcBM + nb) * kTcBK; }
// a split call's CTAs hold half of an SM's shared memory, so that two of them share it
__host__ __device__ constexpr int tc_split_stages(int nb) { return nb == 32 ? 4 : 3; }
__host__ __device__ constexpr int tc_smem_bytes(int nb, int stages, bool split) {
  return stages * tc_stage_bytes(nb) + 1024 + 256 + (split ? kTcBM * nb * 4 : 0);
}

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* tm, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          smem_addr(dst)),
      "l"(tm), "r"(x), "r"(y), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void tmap_prefetch(const CUtensorMap* tm) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}
// Descriptor of a K-major operand of 128-byte swizzled rows, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)1u << 16) | ((uint64_t)(1024u >> 4) << 32) |
         ((uint64_t)1u << 46) | ((uint64_t)2u << 61);
}
// Instruction descriptor, kind::i8: s32 accumulator (bits 4-5 = 2), A and B
// signed (bits 7-9 = 1, bits 10-12 = 1), both K-major, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
__device__ __forceinline__ uint32_t idesc_s8(int M, int N) {
  return (2u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D (TMEM, s32) (+)= A . B^T over 32 inputs, both operands in shared memory.
__device__ __forceinline__ void umma_s8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// 32 TMEM lanes x 32 columns: thread i gets lane (base lane + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Limit of the waits for a CTA's own copies and MMAs before it exits: those
// end within microseconds, so a lowered limit does not cut them short.
__device__ __forceinline__ long long exit_limit(const IntMatmulArgs& a) {
  return a.wait_limit > (1ll << 24) ? a.wait_limit : 1ll << 24;
}

// Bounded wait that also gives up once another role of the CTA has aborted.
// A thread is suspended for 20 us (40,000 cycles) at most, and polls instead
// where the limit is shorter than that.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                        long long limit_cycles) {
  if (mbar_test(bar, parity)) return true;
  const long long t0 = clock64();
  for (;;) {
    if (limit_cycles < 40000 ? mbar_test(bar, parity) : mbar_try_wait(bar, parity, 20000u)) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > limit_cycles) {
      *abort_flag = 1;
      return false;
    }
  }
}

// The same for a warp that goes on together: its lanes may see the barrier and
// the flag in different orders, so they go on only if all of them may, and
// leave together (what follows the wait has warp-wide loads and shuffles).
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                             long long limit_cycles) {
  return __all_sync(0xffffffffu, !*abort_flag && tc_wait(bar, parity, abort_flag, limit_cycles));
}

// 32 tokens (t.., the first `cnt` of them exist) of one output per lane, from
// the accumulators v: y is written 128 (fp32) or 64 (bf16) contiguous bytes
// per token and warp.  xs: the tokens' scales.  With `pairs` (N even, y
// 4-byte aligned) two lanes swap halves, so that one of them writes both
// outputs of the even token and the other both of the odd one.
template <bool FULL>
__device__ __forceinline__ void im_store_chunk(const IntMatmulArgs& a, const uint32_t (&v)[32], const float* xs,
                                               float ws, int n, int t, int cnt, bool pairs) {
  const bool in = n < a.N;
  const int64_t at = (int64_t)t * a.N + n;
#pragma unroll
  for (int i0 = 0; i0 < 32; i0 += 8) {
    if (!FULL && i0 >= cnt) break;
    const float4 x0 = *reinterpret_cast<const float4*>(xs + i0), x1 = *reinterpret_cast<const float4*>(xs + i0 + 4);
    const float x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = im_scaled((int)v[i0 + i], x[i], ws);
    if (a.add) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in && (FULL || i0 + i < cnt)) f[i] += a.add[at + (int64_t)(i0 + i) * a.N];
    }
    if (a.y_f32) {
      float* y = static_cast<float*>(a.y) + at + (int64_t)i0 * a.N;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in && (FULL || i0 + i < cnt)) y[(int64_t)i * a.N] = f[i];
    } else if (pairs) {
      const bool odd = n & 1;
      uint16_t* y = static_cast<uint16_t*>(a.y) + at + (int64_t)(i0 + odd) * a.N - odd;
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        const float got = __shfl_xor_sync(0xffffffffu, odd ? f[i] : f[i + 1], 1);
        const __nv_bfloat162 w = odd ? __floats2bfloat162_rn(got, f[i + 1]) : __floats2bfloat162_rn(f[i], got);
        if (in && (FULL || i0 + i + odd < cnt)) *reinterpret_cast<__nv_bfloat162*>(y + (int64_t)i * a.N) = w;
      }
    } else {
      uint16_t* y = static_cast<uint16_t*>(a.y) + at + (int64_t)i0 * a.N;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (in && (FULL || i0 + i < cnt)) y[(int64_t)i * a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(f[i]));
    }
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t ra;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(ra) : "r"(saddr), "r"(rank));
  return ra;
}
__device__ __forceinline__ void st_cluster(uint32_t raddr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(raddr), "r"(v) : "memory");
}

// Tiles of 128 outputs x NB tokens (the outputs' tiles fastest).  Warp 0
// loads stages by TMA, warp 1 issues the MMAs, the warps from 4 on scale and store.
// Inputs past K and rows past N or T arrive as zeros.
//   SPLIT false: persistent, CTA i takes tiles i, i + grid, ...; accumulators
//     are double-buffered in TMEM, so that a tile's stores run under the next
//     one's MMAs.
//   SPLIT true: one tile per cluster of `split` (a power of two) CTAs, each
//     with its share of K.  Each CTA finishes every split-th token: the others
//     write their s32 sums of it into its shared memory (stores, which nothing
//     waits for one by one, where reading them from there measured 2 us more).
template <int NB, bool SPLIT>
__global__ void __launch_bounds__(tc_threads(SPLIT), SPLIT ? 2 : 1)
    im_tc_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                 const IntMatmulArgs a, const int mtiles, const int ntiles, const int split, const int nst) {
  extern __shared__ uint8_t im_smem[];
  constexpr int kEpi = tc_epi_warps(SPLIT), kStage = tc_stage_bytes(NB), kCols = SPLIT ? NB : 2 * NB;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(im_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + nst * kStage);  // TMA -> MMA
  uint64_t* empty = full + nst;                                       // MMA -> TMA
  uint64_t* accfull = empty + nst;                                    // MMA -> epilogue
  uint64_t* accempty = accfull + 2;                                       // epilogue -> MMA
  uint64_t* drain = accempty + 2;
  int* red = reinterpret_cast<int*>(base + nst * kStage + 256);  // SPLIT: [source CTA][token / split][output]
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ __align__(16) float s_xs[kEpi][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&accfull[c], 1);
      mbar_init(&accempty[c], kEpi);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    s_abort = 0;
    tmap_prefetch(&tm_w);
    tmap_prefetch(&tm_x);
  }
  if (warp == kTcMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&s_tmem)),
                 "r"(kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (SPLIT) cluster_sync();  // every CTA of the cluster runs before its shared memory is written to
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int nkb = (a.K + kTcBK - 1) / kTcBK, tiles = mtiles * ntiles;
  const int rank = SPLIT ? (int)cluster_rank() : 0;
  const int kb0 = SPLIT ? nkb * rank / split : 0, kb1 = SPLIT ? nkb * (rank + 1) / split : nkb;
  const int tile0 = SPLIT ? blockIdx.x / split : blockIdx.x, step = SPLIT ? tiles : gridDim.x;
  const bool pairs = !(a.N & 1) && !(reinterpret_cast<uintptr_t>(a.y) & 3);
  pdl_wait();
  pdl_launch_dependents();

  if (warp == kTcProdWarp) {
    if (lane == 0) {
      asm volatile("fence.proxy.async.global;" ::: "memory");  // rows that earlier kernels wrote, to TMA's reads
      int s = 0;
      uint32_t ph = 0, issued = 0, last_ph = 0;
      for (int t = tile0; t < tiles && !s_abort; t += step) {
        const int m0 = (t % mtiles) * kTcBM, t0 = (t / mtiles) * NB;
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!tc_wait(&empty[s], ph ^ 1u, &s_abort, a.wait_limit)) {
            ok = false;
            break;
          }
          uint8_t* st = base + s * kStage;
          mbar_arrive_expect_tx(&full[s], kStage);
          tma_load_2d(st, &tm_w, kb * kTcBK, m0, &full[s]);
          tma_load_2d(st + kTcBM * kTcBK, &tm_x, kb * kTcBK, t0, &full[s]);
          issued |= 1u << s;
          last_ph = (last_ph & ~(1u << s)) | (ph << s);
          if (++s == nst) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      for (int q = 0; q < nst; ++q)  // every copy issued lands before the CTA can exit
        if ((issued >> q) & 1u) mbar_wait_bounded(&full[q], (last_ph >> q) & 1u, exit_limit(a));
    }
  } else if (warp == kTcMmaWarp) {
    if (lane == 0) {
      int s = 0, c = 0;
      uint32_t ph = 0, pc = 0;
      bool issued_any = false;
      for (int t = tile0; t < tiles && !s_abort; t += step) {
        const int t0 = (t / mtiles) * NB, n = a.T - t0 < NB ? a.T - t0 : NB;
        const uint32_t idesc = idesc_s8(kTcBM, (n + 31) & ~31);
        if (!tc_wait(&accempty[c], pc ^ 1u, &s_abort, a.wait_limit)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(c * NB);
        bool ok = true;
        for (int kb = kb0; kb < kb1; ++kb) {
          const uint64_t ad = sw128_desc(smem_addr(base + s * kStage));
          const uint64_t bd = sw128_desc(smem_addr(base + s * kStage + kTcBM * kTcBK));
          if (!tc_wait(&full[s], ph, &s_abort, a.wait_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kTcBK / 32; ++k) umma_s8(d, ad + 2 * k, bd + 2 * k, idesc, (kb - kb0) | k ? 1u : 0u);
          issued_any = true;
          umma_commit(&empty[s]);
          if (++s == nst) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit(&accfull[c]);
        if (++c == 2) {
          c = 0;
          pc ^= 1u;
        }
      }
      if (issued_any) {  // every MMA issued completes before TMEM is freed
        umma_commit(drain);
        mbar_wait_bounded(drain, 0, exit_limit(a));
      }
    }
  } else if (warp >= kTcEpiWarp0) {
    // warp i reads TMEM lanes 32 (i % 4)..; the warps of a quadrant take 32-token chunks in turn
    const int q = warp & 3, part = (warp - kTcEpiWarp0) >> 2;
    float* xs = s_xs[warp - kTcEpiWarp0];
    int c = 0;
    uint32_t pc = 0;
    for (int t = tile0; t < tiles; t += step) {
      const int n = (t % mtiles) * kTcBM + 32 * q + lane, t0 = (t / mtiles) * NB;
      const float ws = n < a.N ? a.ws[n] : 0.0f;
      if (!tc_wait_warp(&accfull[c], pc, &s_abort, a.wait_limit)) break;
      tc_fence_after();
      for (int col = 32 * part; col < NB && t0 + col < a.T; col += 8 * kEpi) {
        uint32_t v[32];
        if constexpr (SPLIT) {
          tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(c * NB + col), v);
          const uint32_t mine = smem_addr(red) + (uint32_t)((rank * (NB / split)) * kTcBM + 32 * q + lane) * 4;
          const int lg = __ffs(split) - 1;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (t0 + col + i < a.T)
              st_cluster(map_rank(mine + (uint32_t)((col + i) >> lg) * (kTcBM * 4), (uint32_t)(i & (split - 1))), v[i]);
        } else {
          const int cnt = a.T - t0 - col;
          __syncwarp();
          xs[lane] = lane < cnt ? im_token_scale(a, t0 + col + lane) : 0.0f;
          __syncwarp();
          tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(c * NB + col), v);
          if (cnt >= 32)
            im_store_chunk<true>(a, v, xs, ws, n, t0 + col, 32, pairs);
          else
            im_store_chunk<false>(a, v, xs, ws, n, t0 + col, cnt, pairs);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&accempty[c]);
      if (++c == 2) {
        c = 0;
        pc ^= 1u;
      }
    }
  }
  if constexpr (SPLIT) {
    cluster_sync();  // every CTA of the cluster comes here, also after a wait that ran out
    const int m0 = (tile0 % mtiles) * kTcBM, t0 = (tile0 / mtiles) * NB, n = a.T - t0 < NB ? a.T - t0 : NB;
    const bool quads = !(a.N & 3) && !(reinterpret_cast<uintptr_t>(a.y) & 15) &&
                       !(reinterpret_cast<uintptr_t>(a.add) & 15) && m0 + 4 * lane < a.N;
    float ws[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) ws[i] = m0 + 4 * lane + i < a.N ? a.ws[m0 + 4 * lane + i] : 0.0f;
    for (int l = warp; l * split + rank < n; l += kTcEpiWarp0 + kEpi) {
      const int j = l * split + rank;
      const float xs = im_token_scale(a, t0 + j);
      int4 sum = make_int4(0, 0, 0, 0);
      for (int r = 0; r < split; ++r) {
        const int4 v = *reinterpret_cast<const int4*>(red + (r * (NB / split) + l) * kTcBM + 4 * lane);
        sum.x += v.x, sum.y += v.y, sum.z += v.z, sum.w += v.w;
      }
      float4 f = make_float4(im_scaled(sum.x, xs, ws[0]), im_scaled(sum.y, xs, ws[1]), im_scaled(sum.z, xs, ws[2]),
                             im_scaled(sum.w, xs, ws[3]));
      const int64_t at = (int64_t)(t0 + j) * a.N + m0 + 4 * lane;
      if (quads) {
        if (a.add) {
          const float4 d = *reinterpret_cast<const float4*>(a.add + at);
          f.x += d.x, f.y += d.y, f.z += d.z, f.w += d.w;
        }
        if (a.y_f32) {
          *reinterpret_cast<float4*>(static_cast<float*>(a.y) + at) = f;
        } else {
          __nv_bfloat162* y = reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(a.y) + at);
          y[0] = __floats2bfloat162_rn(f.x, f.y);
          y[1] = __floats2bfloat162_rn(f.z, f.w);
        }
      } else {
        const float fv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (m0 + 4 * lane + i < a.N) im_store(a, t0 + j, m0 + 4 * lane + i, fv[i]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s_abort && tid == 0 && a.dev_err) atomicOr(a.dev_err, MOE_DEV_ERR_TIMEOUT);
  if (warp == kTcMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kCols) : "memory");
}

// ---------------------------------------------------------------------------
// two CTAs per tile
// ---------------------------------------------------------------------------
// Tiles of 256 outputs x 256 tokens on pairs of SMs (cta_group::2): each CTA
// brings 128 outputs and 128 tokens per stage and keeps the accumulators of
// its 128 outputs, and one thread of the pair's first CTA issues the MMAs of
// both.  A 128 x 256 tile of one CTA moves 48 KB from L2 per 128 inputs and
// measured 53 bytes a clock and SM there, which bounded it; the pair moves
// 32 KB per CTA for the same MMAs.
constexpr int kPairBM = 256, kPairBN = 256, kPairStages = 6;
constexpr int kPairStage = (kPairBM + kPairBN) / 2 * kTcBK;  // bytes of a CTA's share of a stage
// eight warps store: sixteen took 4 % longer at K 4096 (99 us against 95), where the stores run under the MMAs
constexpr int kPairEpiWarps = 8, kPairThreads = 32 * (kTcEpiWarp0 + kPairEpiWarps);
constexpr int kPairSmem = kPairStages * kPairStage + 1024 + 256;

// A load into this CTA's shared memory that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* tm, int x, int y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_addr(dst)),
      "l"(tm), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void umma_s8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n}\n" ::"r"(
          d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this offset in both CTAs once the MMAs issued so far are complete.
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
// The same for this CTA's barrier alone.
__device__ __forceinline__ void umma_commit_pair_local(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1)
    im_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                   const IntMatmulArgs a, const int mtiles, const int ntiles) {
  extern __shared__ uint8_t im_smem[];
  constexpr int kEpi = kPairEpiWarps;
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(im_smem) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(base + kPairStages * kPairStage);  // both CTAs' TMA -> MMA (CTA 0's)
  uint64_t* empty = full + kPairStages;   // MMA -> TMA (each CTA's)
  uint64_t* accfull = empty + kPairStages;  // MMA -> epilogue (each CTA's)
  uint64_t* accempty = accfull + 2;         // both CTAs' epilogues -> MMA (CTA 0's)
  uint64_t* drain = accempty + 2;           // MMA at exit (CTA 0's)
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ __align__(16) float s_xs[kEpi][32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&accfull[c], 1);
      mbar_init(&accempty[c], 2 * kEpi);
    }
    mbar_init(drain, 1);
    fence_barrier_init();
    s_abort = 0;
    tmap_prefetch(&tm_w);
    tmap_prefetch(&tm_x);
  }
  if (warp == kTcMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the pair's barriers exist before either CTA's copies or arrivals reach them
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  const int nkb = (a.K + kTcBK - 1) / kTcBK, tiles = mtiles * ntiles;
  const int tile0 = blockIdx.x >> 1, step = gridDim.x >> 1;
  const bool pairs = !(a.N & 1) && !(reinterpret_cast<uintptr_t>(a.y) & 3);
  pdl_wait();
  pdl_launch_dependents();

  if (warp == kTcProdWarp) {
    if (lane == 0) {
      asm volatile("fence.proxy.async.global;" ::: "memory");  // rows that earlier kernels wrote, to TMA's reads
      int s = 0;
      uint32_t ph = 0, issued = 0;
      for (int t = tile0; t < tiles && !s_abort; t += step) {
        const int m0 = (t % mtiles) * kPairBM + 128 * (int)rank, t0 = (t / mtiles) * kPairBN + 128 * (int)rank;
        bool ok = true;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!tc_wait(&empty[s], ph ^ 1u, &s_abort, a.wait_limit)) {
            ok = false;
            break;
          }
          uint8_t* st = base + s * kPairStage;
          const uint32_t bar = map_rank(smem_addr(&full[s]), 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStage);
          tma_load_2d_pair(st, &tm_w, kb * kTcBK, m0, bar);
          tma_load_2d_pair(st + 128 * kTcBK, &tm_x, kb * kTcBK, t0, bar);
          issued |= 1u << s;
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
      }
      // every copy issued lands, and is read, before the CTA can exit: its stage's next emptying says so
      for (int q = 0; q < kPairStages; ++q) {
        const uint32_t last = s > q ? ph : ph ^ 1u;  // phase in which stage q was last filled
        if (((issued >> q) & 1u) && !mbar_wait_bounded(&empty[q], last, exit_limit(a))) break;
      }
    }
  } else if (warp == kTcMmaWarp) {
    if (lane == 0 && rank == 0) {
      const uint32_t idesc = idesc_s8(kPairBM, kPairBN);
      int s = 0, c = 0;
      uint32_t ph = 0, pc = 0;
      bool issued_any = false;
      for (int t = tile0; t < tiles && !s_abort; t += step) {
        if (!tc_wait(&accempty[c], pc ^ 1u, &s_abort, a.wait_limit)) break;
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(c * kPairBN);
        bool ok = true;
        for (int kb = 0; kb < nkb; ++kb) {
          const uint64_t ad = sw128_desc(smem_addr(base + s * kPairStage));
          const uint64_t bd = sw128_desc(smem_addr(base + s * kPairStage + 128 * kTcBK));
          if (!tc_wait(&full[s], ph, &s_abort, a.wait_limit)) {
            ok = false;
            break;
          }
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kTcBK / 32; ++k) umma_s8_pair(d, ad + 2 * k, bd + 2 * k, idesc, kb | k ? 1u : 0u);
          issued_any = true;
          umma_commit_pair(&empty[s]);
          if (++s == kPairStages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit_pair(&accfull[c]);
        if (++c == 2) {
          c = 0;
          pc ^= 1u;
        }
      }
      if (issued_any) {  // every MMA issued completes before TMEM is freed
        // its arrival is waited for here only, so it must not reach the other CTA, which may have gone
        umma_commit_pair_local(drain);
        mbar_wait_bounded(drain, 0, exit_limit(a));
      }
    }
  } else if (warp >= kTcEpiWarp0) {
    const int q = warp & 3, part = (warp - kTcEpiWarp0) >> 2;
    float* xs = s_xs[warp - kTcEpiWarp0];
    int c = 0;
    uint32_t pc = 0;
    for (int t = tile0; t < tiles; t += step) {
      const int n = (t % mtiles) * kPairBM + 128 * (int)rank + 32 * q + lane, t0 = (t / mtiles) * kPairBN;
      const float ws = n < a.N ? a.ws[n] : 0.0f;
      if (!tc_wait_warp(&accfull[c], pc, &s_abort, a.wait_limit)) break;
      tc_fence_after();
      for (int col = 32 * part; col < kPairBN && t0 + col < a.T; col += 8 * kEpi) {
        uint32_t v[32];
        const int cnt = a.T - t0 - col;
        __syncwarp();
        xs[lane] = lane < cnt ? im_token_scale(a, t0 + col + lane) : 0.0f;
        __syncwarp();
        tmem_ld32(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(c * kPairBN + col), v);
        if (cnt >= 32)
          im_store_chunk<true>(a, v, xs, ws, n, t0 + col, 32, pairs);
        else
          im_store_chunk<false>(a, v, xs, ws, n, t0 + col, cnt, pairs);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(map_rank(smem_addr(&accempty[c]), 0));
      if (++c == 2) {
        c = 0;
        pc ^= 1u;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other's copies, MMAs or arrivals may reach it
  tc_fence_after();
  if (s_abort && tid == 0 && a.dev_err) atomicOr(a.dev_err, MOE_DEV_ERR_TIMEOUT);
  if (warp == kTcMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
PFN_cuTensorMapEncodeTiled_v12000 tmap_encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Rows of K bytes; a box is `rows` rows x 128 bytes, 128-byte swizzled.
bool encode_rows(CUtensorMap* m, const int8_t* p, int n, int K, int rows) {
  const auto fn = tmap_encoder();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)n}, strides[1] = {(cuuint64_t)K};
  const cuuint32_t box[2] = {(cuuint32_t)kTcBK, (cuuint32_t)rows}, es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB>
cudaError_t launch_tc(const IntMatmulArgs& a, int split, int num_sms, cudaStream_t st) {
  while (split & (split - 1)) split &= split - 1;  // a power of two, which the kernel's owners of tokens rely on
  static int smem_set[2][4] = {};
  const int mtiles = (a.N + kTcBM - 1) / kTcBM, ntiles = (a.T + NB - 1) / NB;
  const int64_t tiles = (int64_t)mtiles * ntiles;
  const int nkb = (a.K + kTcBK - 1) / kTcBK;
  const void* kern = split > 1 ? reinterpret_cast<const void*>(im_tc_kernel<NB, NB <= kTcSplitMaxTokens>)
                               : reinterpret_cast<const void*>(im_tc_kernel<NB, false>);
  cudaError_t e = ensure_smem_attr(kern, smem_set[split > 1]);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, tx;
  if (!encode_rows(&tw, a.wq, a.N, a.K, kTcBM) || !encode_rows(&tx, a.xq, a.T, a.K, NB)) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(split > 1 ? tiles * split : std::min<int64_t>(tiles, num_sms)));
  cfg.blockDim = dim3(tc_threads(split > 1));
  const int nst = split > 1 ? std::min(tc_split_stages(NB), (nkb + split - 1) / split) : tc_stages(NB);
  cfg.dynamicSmemBytes = tc_smem_bytes(NB, nst, split > 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {(unsigned)split, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  void* argv[] = {&tw, &tx, const_cast<IntMatmulArgs*>(&a), const_cast<int*>(&mtiles), const_cast<int*>(&ntiles),
                  &split, const_cast<int*>(&nst)};
  return cudaLaunchKernelExC(&cfg, kern, argv);
}

cudaError_t launch_pair(const IntMatmulArgs& a, int num_sms, cudaStream_t st) {
  static int smem_set[4] = {};
  const void* kern = reinterpret_cast<const void*>(im_pair_kernel);
  cudaError_t e = ensure_smem_attr(kern, smem_set);
  if (e != cudaSuccess) return e;
  CUtensorMap tw, tx;
  if (!encode_rows(&tw, a.wq, a.N, a.K, 128) || !encode_rows(&tx, a.xq, a.T, a.K, 128)) return cudaErrorInvalidValue;
  const int mtiles = (a.N + kPairBM - 1) / kPairBM, ntiles = (a.T + kPairBN - 1) / kPairBN;
  const int64_t pairs = std::min<int64_t>((int64_t)mtiles * ntiles, num_sms / 2);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  void* argv[] = {&tw, &tx, const_cast<IntMatmulArgs*>(&a), const_cast<int*>(&mtiles), const_cast<int*>(&ntiles)};
  return cudaLaunchKernelExC(&cfg, kern, argv);
}

struct TcPlan {
  int nb, split;  // tokens of a tile (0: 256 x 256 on pairs of SMs), CTAs that share a tile's K
};

// The tile and split of a call: the least estimated time, in us,
//   3.6 + rounds x (128-input blocks of a CTA) x block + stores (+ split),
// where a round is one tile per SM (or pair, or two half-size CTAs per SM of a
// split call).  Its constants were fitted to every choice timed at 47 sizes
// (N 1024 to 16384, K 512 to 8192, 17 to 4096 tokens, weights not in L2): the
// choice is within 8 % of the best one there.  Some of what it decides between:
//   64 x 1536 x 2048     split 4 ways 4.4 us, whole 7.8
//   512 x 4096 x 2048    128-token tiles 9.5 us, 64-token tiles (two rounds) 14.5
//   1024 x 4096 x 8192   pairs 27.4 us, 256-token tiles 30.3, 128-token tiles 44.5
TcPlan tc_plan(const IntMatmulArgs& a, int num_sms) {
  static constexpr struct {
    int nb;
    float block, stores;
  } kTile[] = {{32, 0.285f, 0.25f}, {64, 0.30f, 0.4f}, {128, 0.325f, 0.7f}, {256, 0.40f, 2.2f}, {0, 0.36f, 3.0f}};
  const int nkb = (a.K + kTcBK - 1) / kTcBK;
  TcPlan best{64, 1};
  float least = 3e38f;
  for (const auto& c : kTile) {
    const int bm = c.nb ? kTcBM : kPairBM, bn = c.nb ? c.nb : kPairBN, slots = c.nb ? num_sms : num_sms / 2;
    if (bn > 32 && a.T <= bn / 2) break;  // a narrower tile holds every token
    const int64_t tiles = (int64_t)((a.N + bm - 1) / bm) * ((a.T + bn - 1) / bn);
    for (int split = 1; split <= 8; split *= 2) {
      if (split > 1 && (c.nb == 0 || c.nb > kTcSplitMaxTokens || tiles * split > kTcSplitCtas || split > nkb / 2)) break;
      const int64_t rounds = (tiles * split + slots - 1) / slots;
      float t = 3.6f + c.stores + (float)rounds * (float)((nkb + split - 1) / split) * c.block;
      if (split > 1) {
        t += c.nb == 32 ? 0.2f : 0.9f;
        if (rounds > 1) t += 0.5f - 0.25f * (float)rounds * (float)((nkb + split - 1) / split) * c.block;  // on one SM
      }
      if (t < least) {
        least = t;
        best = {c.nb, split};
      }
    }
  }
  return best;
}

template <int NT>
const void* rows_kernel(int W) {
  return W == 8   ? reinterpret_cast<const void*>(im_rows_kernel<NT, 8>)
         : W == 4 ? reinterpret_cast<const void*>(im_rows_kernel<NT, 4>)
                  : reinterpret_cast<const void*>(im_rows_kernel<NT, 2>);
}

}  // namespace

cudaError_t launch_int_matmul(const IntMatmulArgs& a, int num_sms, cudaStream_t st) {
  if (a.T <= kRowsTokens || (a.T <= kRowsMaxTokens && (int64_t)a.N * a.K <= kRowsMaxWeights)) {
    // enough units for each warp to fill its ring
    const int W = a.K >= 4096 ? 8 : a.K >= 2048 ? 4 : 2;
    const void* kern = a.T <= 8    ? rows_kernel<1>(W)
                       : a.T <= 16 ? rows_kernel<2>(W)
                       : a.T <= 24 ? rows_kernel<3>(W)
                                   : rows_kernel<4>(W);
    return launch_pdl(kern, (a.N + 15) / 16, 32 * W, 0, st, a);
  }
  const TcPlan p = tc_plan(a, num_sms);
  if (p.nb == 32) return launch_tc<32>(a, p.split, num_sms, st);
  if (p.nb == 64) return launch_tc<64>(a, p.split, num_sms, st);
  if (p.nb == 128) return launch_tc<128>(a, 1, num_sms, st);
  if (p.nb == 256) return launch_tc<256>(a, 1, num_sms, st);
  return launch_pair(a, num_sms, st);
}

}  // namespace moe
