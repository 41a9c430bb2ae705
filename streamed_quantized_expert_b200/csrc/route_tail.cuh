// What follows the routing of one decode token in the same block (stages 2
// and 3), shared by the kernels that route a token by softmax and by grouped
// scores.
#pragma once

#include "common.cuh"
#include "kernels.h"

namespace moe {

// The sort of one token's n distinct experts ids[0..n) (rank order, n <= 32,
// of Ew in all) and the slot lookup over the whole active list, as
// sort_small_kernel and lookup_kernel write them for T = 1, by the 256 threads
// of a block in which ids have been written.  The active list is the routed
// experts ascending, then the shared ones; pair j of rank r sits at position
// r.  With host_meta (page-locked host memory the device can address), warp 1
// also writes n_active to host_meta[0] and the active list to host_meta[2 ..],
// then, once those writes are visible system-wide, seq to host_meta[1]: the
// host waits for seq there instead of copying the list back and synchronising.
__device__ __forceinline__ void sort_lookup_token(const int32_t* ids, int n, int Ew, const SortLookupArgs& o) {
  __shared__ int s_sel[32];  // the token's experts, rank order
  __shared__ int s_act[32];  // ascending
  const int tid = threadIdx.x;
  __syncthreads();  // the block's own global writes of ids are visible to it
  if (tid < n) s_sel[tid] = ids[tid];
  __syncthreads();
  if (tid < n) {
    const int e = s_sel[tid];
    int r = 0;
    for (int j = 0; j < n; ++j) r += s_sel[j] < e;
    s_act[r] = e;
    o.active[r] = e;
    o.pairs[r] = tid;
  }
  for (int e = tid; e <= Ew; e += 256) {
    int c = 0;
    for (int j = 0; j < n; ++j) c += s_sel[j] < e;
    o.offsets[e] = c;
  }
  __syncthreads();
  if (tid < 32) {  // lookup: one lane per active expert
    const bool in = tid < n;
    const int e = in ? s_act[tid] : -1;
    const int sl = in ? o.table[e] : 0;
    if (in) o.slots[tid] = sl;
    if (in && sl >= o.n_slots && o.dev_err) atomicOr(o.dev_err, MOE_DEV_ERR_SLOT_RANGE);
    const unsigned bal = __ballot_sync(0xffffffffu, in && sl < 0);
    if (in && sl < 0) o.miss[__popc(bal & ((1u << tid) - 1u))] = e;
    if (tid == 0) {
      *o.n_active = n;
      *o.n_miss = __popc(bal);
    }
  } else if (tid < 64 && o.host_meta) {
    const int lane = tid - 32;
    if (lane < n) o.host_meta[2 + lane] = s_act[lane];
    if (lane == 0) o.host_meta[0] = n;
    __threadfence_system();
    __syncwarp();
    if (lane == 0) *reinterpret_cast<volatile int32_t*>(o.host_meta + 1) = o.seq;
  }
}

}  // namespace moe
