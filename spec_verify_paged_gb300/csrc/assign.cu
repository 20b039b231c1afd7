// assign.cu -- pages for sequences that grow and shrink (kv_assign_pages,
// include/svp.h): pages past the target lengths go onto the stack of free
// pages, missing ones are taken from its top, and every new position gets its
// slot (page * 16 + row).
//
// The order is fixed (releases by sequence and page, then takes by sequence
// and page), so where an entry goes follows from prefix sums over the
// sequences, which every CTA works out for itself, 1024 sequences at a time:
//   release r of R    -> stack[free + r]
//   take i            <- stack[free + R - 1 - i]
//   new position t    -> slot entry t
// One cluster does a call.  Its CTAs share out the entries (an entry finds its
// sequence by a binary search in the prefix sums); a cluster barrier separates
// the releases from the takes, which may take what was just released, and the
// reads of the old lengths from the writes of the new ones.
// Bound by that chain: launch, lengths, scans, barriers.
#include <cooperative_groups.h>

#include <cstdint>

#include "ptx.cuh"
#include "svp.h"
#include "svp_internal.h"

namespace svp {

static __device__ unsigned int g_status_assign;

namespace {

namespace cg = cooperative_groups;
using u64 = unsigned long long;

constexpr int kAssignThreads = 1024;

struct AssignShared {
  u64 warp_sum[2][32];
  u64 before[kAssignThreads];    // exclusive prefix of a chunk's entries
  u64 first[kAssignThreads];     // takes: the sequence's first on the stack
  int from[kAssignThreads];      // its first entry (a page or a position)
  unsigned char served[kAssignThreads];
};

__device__ __forceinline__ void raise_assign(unsigned f) {
  atomicOr(&g_status_assign, f);
}

// Exclusive prefix sum over the block; `sum` becomes the block's total.
__device__ __forceinline__ u64 scan(u64 v, u64 *warp_sum, u64 &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();  // warp_sum may still be read from an earlier scan
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  const u64 x = warp_sum[lane];
  u64 y = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const u64 z = __shfl_up_sync(0xffffffffu, y, off);
    if (lane >= off) y += z;
  }
  sum = __shfl_sync(0xffffffffu, y, 31);
  return __shfl_sync(0xffffffffu, y - x, warp) + incl - v;
}

// What sequence b asks for.
struct Ask {
  int old_len, new_len;  // equal where the lengths are not valid
  int have, want;        // pages
  bool bad;
};
__device__ __forceinline__ Ask ask_of(const AssignParams &p, int b) {
  Ask a = {0, 0, 0, 0, false};
  if (b >= p.batch) return a;
  const int L = p.seq_lens[b], N = p.new_lens[b];
  const long long cap = (long long)p.max_blocks * kBlockSize;
  a.old_len = a.new_len = L;
  if (L < 0 || L > cap || N < 0 || N > cap) {
    a.bad = true;
    return a;
  }
  a.new_len = N;
  a.have = (int)(((long long)L + kBlockSize - 1) / kBlockSize);
  a.want = (int)(((long long)N + kBlockSize - 1) / kBlockSize);
  return a;
}

// The sequence (of a chunk) that holds entry i: the last with before <= i.
__device__ __forceinline__ int holder(const u64 *before, u64 i) {
  int lo = 0;
#pragma unroll
  for (int step = kAssignThreads / 2; step > 0; step >>= 1)
    if (before[lo + step] <= i) lo += step;
  return lo;
}

__global__ void __launch_bounds__(kAssignThreads)
    assign_pages_kernel(const AssignParams p) {
  __shared__ AssignShared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  const u64 me = (u64)rank * kAssignThreads + tid;
  const u64 all = (u64)nc * kAssignThreads;
  pdl_wait();
  pdl_launch_dependents();
  const bool leader = rank == 0;
  const int F = *p.free_count;

  // ---- the pages that come back ----
  u64 R = 0, sum;
  for (int b0 = 0; b0 < p.batch; b0 += kAssignThreads) {
    const Ask a = ask_of(p, b0 + tid);
    scan(a.have > a.want ? (u64)(a.have - a.want) : 0, sm.warp_sum[0], sum);
    R += sum;
    if (a.bad && leader) raise_assign(SVP_DEV_BAD_SEQ_LEN);
  }
  if (F < 0 || (long long)F + (long long)R > p.capacity) {
    // no stack of this size, or one that its pages do not fit: do nothing
    // (uniform over the cluster)
    if (leader && tid == 0) raise_assign(SVP_DEV_NO_PAGES);
    for (u64 i = me; i < (u64)p.n_slots; i += all) p.slots[i] = -1;
    if (p.offsets)
      for (u64 i = me; i <= (u64)p.batch; i += all) p.offsets[i] = 0;
    return;
  }
  u64 done = 0;
  if (R > 0) {
    for (int b0 = 0; b0 < p.batch; b0 += kAssignThreads) {
      const Ask a = ask_of(p, b0 + tid);
      const u64 before =
          scan(a.have > a.want ? (u64)(a.have - a.want) : 0, sm.warp_sum[0], sum);
      sm.before[tid] = before;
      sm.from[tid] = a.want;
      __syncthreads();
      for (u64 i = me; i < sum; i += all) {
        const int s = holder(sm.before, i);
        int32_t *const entry = p.block_table + (size_t)(b0 + s) * p.max_blocks +
                               sm.from[s] + (i - sm.before[s]);
        const int page = *entry;
        if (page < 0 || page >= p.num_blocks) raise_assign(SVP_DEV_BAD_BLOCK_ID);
        p.free_pages[(u64)F + done + i] = page;
        *entry = -1;
      }
      done += sum;
      __syncthreads();
    }
    cluster.sync();  // released pages may be taken below
  }
  const u64 top = (u64)F + R;  // pages there are

  // ---- the pages taken, and the slots ----
  // Sequences are served in order: from the first whose pages or slots run
  // out, no sequence that needs any is.
  u64 taken = 0, tokens = 0;     // asked for by the chunks before
  u64 given = 0;                 // pages taken by sequences served
  for (int b0 = 0; b0 < p.batch; b0 += kAssignThreads) {
    const Ask a = ask_of(p, b0 + tid);
    const u64 need = a.want > a.have ? (u64)(a.want - a.have) : 0;
    const u64 rows = a.new_len > a.old_len ? (u64)(a.new_len - a.old_len) : 0;
    u64 all_need, all_rows, all_given;
    const u64 n0 = scan(need, sm.warp_sum[0], all_need);
    const u64 r0 = scan(rows, sm.warp_sum[1], all_rows);
    const bool fits =
        (need == 0 || taken + n0 + need <= top) &&
        (rows == 0 || !p.slots || tokens + r0 + rows <= (u64)p.n_slots);
    const u64 g0 = scan(fits ? need : 0, sm.warp_sum[0], all_given);
    if (leader && p.offsets && b0 + tid < p.batch) {
      const u64 at = tokens + r0;
      p.offsets[b0 + tid] = at > 0x7fffffffull ? 0x7fffffff : (int)at;
    }
    if (leader && !fits) raise_assign(SVP_DEV_NO_PAGES);
    if (all_given > 0) {
      sm.before[tid] = g0;
      sm.from[tid] = a.have;
      __syncthreads();
      for (u64 i = me; i < all_given; i += all) {
        const int s = holder(sm.before, i);
        const int page = p.free_pages[top - 1 - (given + i)];
        if (page < 0 || page >= p.num_blocks) raise_assign(SVP_DEV_BAD_BLOCK_ID);
        p.block_table[(size_t)(b0 + s) * p.max_blocks + sm.from[s] +
                      (i - sm.before[s])] = page;
      }
      __syncthreads();
    }
    if (p.slots && all_rows > 0) {
      sm.before[tid] = r0;
      sm.first[tid] = given + g0;
      sm.from[tid] = a.old_len;
      sm.served[tid] = fits;
      __syncthreads();
      for (u64 i = me; i < all_rows; i += all) {
        if (tokens + i >= (u64)p.n_slots) break;
        const int s = holder(sm.before, i);
        long long slot = -1;
        if (sm.served[s]) {
          const int old = sm.from[s];
          const int pos = old + (int)(i - sm.before[s]);
          const int have = (int)(((long long)old + kBlockSize - 1) / kBlockSize);
          const int k = pos / kBlockSize;
          const int page =
              k < have ? p.block_table[(size_t)(b0 + s) * p.max_blocks + k]
                       : p.free_pages[top - 1 - (sm.first[s] + (k - have))];
          if (page >= 0 && page < p.num_blocks)
            slot = (long long)page * kBlockSize + pos % kBlockSize;
          else
            raise_assign(SVP_DEV_BAD_BLOCK_ID);
        }
        p.slots[tokens + i] = slot;
      }
      __syncthreads();
    }
    taken += all_need;
    tokens += all_rows;
    given += all_given;
  }
  if (p.slots)
    for (u64 i = tokens + me; i < (u64)p.n_slots; i += all) p.slots[i] = -1;
  cluster.sync();  // every CTA has read the lengths and the count

  // ---- the new state ----
  if (!leader) return;
  if (tid == 0) {
    *p.free_count = (int)(top - given);
    if (p.offsets)
      p.offsets[p.batch] = tokens > 0x7fffffffull ? 0x7fffffff : (int)tokens;
  }
  taken = tokens = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kAssignThreads) {
    const Ask a = ask_of(p, b0 + tid);
    const u64 need = a.want > a.have ? (u64)(a.want - a.have) : 0;
    const u64 rows = a.new_len > a.old_len ? (u64)(a.new_len - a.old_len) : 0;
    u64 all_need, all_rows;
    const u64 n0 = scan(need, sm.warp_sum[0], all_need);
    const u64 r0 = scan(rows, sm.warp_sum[1], all_rows);
    const bool fits =
        (need == 0 || taken + n0 + need <= top) &&
        (rows == 0 || !p.slots || tokens + r0 + rows <= (u64)p.n_slots);
    if (fits && !a.bad && b0 + tid < p.batch) p.seq_lens[b0 + tid] = a.new_len;
    taken += all_need;
    tokens += all_rows;
  }
}

}  // namespace

cudaError_t launch_assign_pages(const AssignParams &p, cudaStream_t stream) {
  // one CTA for a decode step's few entries, eight for prompts
  const int nc = p.n_slots > 8 * kAssignThreads ? 8 : 1;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc);
  cfg.blockDim = dim3(kAssignThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, assign_pages_kernel, p);
}

cudaError_t read_status_assign(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_assign, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_assign, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
