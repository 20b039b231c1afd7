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
// Up to 1024 sequences are read and scanned once, by one scan for the three
// sums; more go chunk by chunk.
// Bound by that chain: launch, lengths, scan, table or stack, barriers.  64
// sequences that get 5 rows each, with the append of 8 heads and the release:
// 12 us as calls, 9.6 as graph nodes; 64 prompts of up to 2048 rows (65,568
// slots, 4132 pages) 9.5 us for the assignment and 5 for the release beside an
// append of 75.
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

// The sequence (of a chunk) that holds entry i: the last with before <= i;
// span: a power of two, at least the chunk's sequences.
__device__ __forceinline__ int holder(const u64 *before, u64 i, int span) {
  int lo = 0;
  for (int step = span / 2; step > 0; step >>= 1)
    if (before[lo + step] <= i) lo += step;
  return lo;
}

// No stack of this size, or one that its pages do not fit: nothing changes.
__device__ __forceinline__ void refuse(const AssignParams &p, u64 me, u64 all) {
  if (me == 0) raise_assign(SVP_DEV_NO_PAGES);
  for (u64 i = me; i < (u64)p.n_slots; i += all) p.slots[i] = -1;
  if (p.offsets)
    for (u64 i = me; i <= (u64)p.batch; i += all) p.offsets[i] = 0;
}

__device__ __forceinline__ int saturated(u64 x) {
  return x > 0x7fffffffull ? 0x7fffffff : (int)x;
}

// The slot of a sequence's new position: its page is one it had, or take
// `first` on and counting.
__device__ __forceinline__ long long slot_of(const AssignParams &p, int b, int old_len,
                                             int nth, u64 first, u64 top) {
  const int pos = old_len + nth;
  const int have = (int)(((long long)old_len + kBlockSize - 1) / kBlockSize);
  const int k = pos / kBlockSize;
  const int page = k < have ? p.block_table[(size_t)b * p.max_blocks + k]
                            : p.free_pages[top - 1 - (first + (u64)(k - have))];
  if (page >= 0 && page < p.num_blocks)
    return (long long)page * kBlockSize + pos % kBlockSize;
  raise_assign(SVP_DEV_BAD_BLOCK_ID);
  return -1;
}

// Up to kAssignThreads sequences.
struct AssignOne {
  u64 sums[3][32];
  u64 give[kAssignThreads], need[kAssignThreads], rows[kAssignThreads];
  int old_len[kAssignThreads], want[kAssignThreads];
  u64 given;
  unsigned char served[kAssignThreads];
};

__global__ void __launch_bounds__(kAssignThreads, 1)
    assign_one_kernel(const AssignParams p, int span) {
  __shared__ AssignOne sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const u64 me = (u64)rank * kAssignThreads + tid;
  const u64 all = (u64)nc * kAssignThreads;
  // (nothing may start early after this one: the next kernel's block table
  // and lengths are what it writes)
  pdl_wait();
  const int F = *p.free_count;
  const Ask a = ask_of(p, tid);
  if (a.bad && rank == 0) raise_assign(SVP_DEV_BAD_SEQ_LEN);
  // pages that come back, pages that are missing, new positions
  u64 v[3] = {a.have > a.want ? (u64)(a.have - a.want) : 0,
              a.want > a.have ? (u64)(a.want - a.have) : 0,
              a.new_len > a.old_len ? (u64)(a.new_len - a.old_len) : 0};
  const u64 mine[3] = {v[0], v[1], v[2]};
  u64 sum[3];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1)
#pragma unroll
    for (int x = 0; x < 3; ++x) {
      const u64 y = __shfl_up_sync(0xffffffffu, v[x], off);
      if (lane >= off) v[x] += y;
    }
  if (lane == 31) {
#pragma unroll
    for (int x = 0; x < 3; ++x) sm.sums[x][warp] = v[x];
  }
  __syncthreads();
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    u64 y = sm.sums[x][lane];
    const u64 own = y;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const u64 z = __shfl_up_sync(0xffffffffu, y, off);
      if (lane >= off) y += z;
    }
    sum[x] = __shfl_sync(0xffffffffu, y, 31);
    v[x] += __shfl_sync(0xffffffffu, y - own, warp) - mine[x];
  }
  const u64 R = sum[0], top = (u64)F + R;
  if (F < 0 || (long long)top > p.capacity) {
    refuse(p, me, all);  // (the whole cluster)
    return;
  }
  // Sequences are served in order: from the first whose pages or slots run
  // out, no sequence that needs any is.
  const bool fits = (mine[1] == 0 || v[1] + mine[1] <= top) &&
                    (mine[2] == 0 || !p.slots || v[2] + mine[2] <= (u64)p.n_slots);
  sm.give[tid] = v[0];
  sm.need[tid] = v[1];
  sm.rows[tid] = v[2];
  sm.old_len[tid] = a.old_len;
  sm.want[tid] = a.want;
  sm.served[tid] = fits;
  if (tid == 0) sm.given = sum[1];
  __syncthreads();
  if (!fits && mine[1] > 0) atomicMin(&sm.given, v[1]);
  if (!fits && rank == 0) raise_assign(SVP_DEV_NO_PAGES);
  for (u64 i = me; i < R; i += all) {
    const int s = holder(sm.give, i, span);
    int32_t *const entry = p.block_table + (size_t)s * p.max_blocks + sm.want[s] +
                           (i - sm.give[s]);
    const int page = *entry;
    if (page < 0 || page >= p.num_blocks) raise_assign(SVP_DEV_BAD_BLOCK_ID);
    p.free_pages[(u64)F + i] = page;
    *entry = -1;
  }
  // what was released may be taken, and every CTA has read the lengths
  if (nc > 1) cluster.sync(); else __syncthreads();
  const u64 given = sm.given;  // pages of the sequences served
  for (u64 i = me; i < given; i += all) {
    const int s = holder(sm.need, i, span);
    const int have =
        (int)(((long long)sm.old_len[s] + kBlockSize - 1) / kBlockSize);
    const int page = p.free_pages[top - 1 - i];
    if (page < 0 || page >= p.num_blocks) raise_assign(SVP_DEV_BAD_BLOCK_ID);
    p.block_table[(size_t)s * p.max_blocks + have + (i - sm.need[s])] = page;
  }
  if (p.slots) {
#pragma unroll 4
    for (u64 i = me; i < (u64)p.n_slots; i += all) {
      long long slot = -1;
      if (i < sum[2]) {
        const int s = holder(sm.rows, i, span);
        if (sm.served[s])
          slot = slot_of(p, s, sm.old_len[s], (int)(i - sm.rows[s]), sm.need[s], top);
      }
      p.slots[i] = slot;
    }
  }
  if (rank != 0) return;
  if (tid < p.batch) {
    if (fits && !a.bad) p.seq_lens[tid] = a.new_len;
    if (p.offsets) p.offsets[tid] = saturated(v[2]);
  }
  if (tid == 0) {
    *p.free_count = (int)(top - given);
    if (p.offsets) p.offsets[p.batch] = saturated(sum[2]);
  }
}

__global__ void __launch_bounds__(kAssignThreads, 1)
    assign_pages_kernel(const AssignParams p) {
  __shared__ AssignShared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  const u64 me = (u64)rank * kAssignThreads + tid;
  const u64 all = (u64)nc * kAssignThreads;
  // (nothing may start early after this one: the next kernel's block table
  // and lengths are what it writes)
  pdl_wait();
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
    refuse(p, me, all);  // (the whole cluster)
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
        const int s = holder(sm.before, i, kAssignThreads);
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
    if (leader && p.offsets && b0 + tid < p.batch)
      p.offsets[b0 + tid] = saturated(tokens + r0);
    if (leader && !fits) raise_assign(SVP_DEV_NO_PAGES);
    if (all_given > 0) {
      sm.before[tid] = g0;
      sm.from[tid] = a.have;
      __syncthreads();
      for (u64 i = me; i < all_given; i += all) {
        const int s = holder(sm.before, i, kAssignThreads);
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
        const int s = holder(sm.before, i, kAssignThreads);
        p.slots[tokens + i] =
            sm.served[s] ? slot_of(p, b0 + s, sm.from[s], (int)(i - sm.before[s]),
                                   sm.first[s], top)
                         : -1;
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
    if (p.offsets) p.offsets[p.batch] = saturated(tokens);
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
  // one CTA for a decode step's few entries, eight where there may be many
  const bool many = p.n_slots > 4 * kAssignThreads ||
                    (!p.slots && (long long)p.batch * p.max_blocks > 4 * kAssignThreads);
  const int nc = many ? 8 : 1;
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
  if (p.batch > kAssignThreads) return cudaLaunchKernelEx(&cfg, assign_pages_kernel, p);
  int span = 1;
  while (span < p.batch) span *= 2;
  return cudaLaunchKernelEx(&cfg, assign_one_kernel, p, span);
}

cudaError_t status_word_assign(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_assign);
}

}  // namespace svp
