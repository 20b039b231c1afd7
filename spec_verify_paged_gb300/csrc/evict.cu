// evict.cu -- eviction from the paged cache by accumulated attention weight
// (kv_evict, include/svp.h): per (sequence, kv head) the sinks, the newest
// rows and the best-scored rest are kept, in position order.
//
// Two kernels:
//  * select_kernel: the k-th largest score of a group by a radix search over
//    the scores' bits (11, 11 and 10 bits, most significant first), then one
//    scan that numbers the kept positions.  One cluster of CTAs per group,
//    each with a run of positions; scores are read from memory once and
//    their ordered keys kept in shared memory (beyond 16,384 positions per
//    CTA they are read again each pass).  The histograms are added across
//    the cluster through distributed shared memory.  Bound by one read of
//    the scores and, for short contexts, by the chain of passes.
//  * compact_kernel: moves the kept rows of K, V and the scores.  Kept
//    positions are increasing, so slot i never lies after its source: with
//    all loads of a batch of rows before its stores, and batches in order,
//    the move is safe in place.  Bound by the moved bytes, read and written.
#include <cooperative_groups.h>

#include <cstdint>

#include "attn_common.cuh"

namespace svp {

static __device__ unsigned int g_status_evict;

namespace {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;
constexpr int kSelCache = 16384;    // keys a CTA holds in shared memory
constexpr int kSelRun = 4096;       // positions per CTA the cluster size aims at
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;

struct SelShared {
  unsigned hist[2][kBins];
  unsigned long long warp_sum[kSelThreads / 32];
  unsigned long long total;       // this CTA's kept-for-sure and tied counts
  unsigned bin, above;
};

// Ascending unsigned order of the scores; NaN as -inf, -0 as +0.
__device__ __forceinline__ unsigned score_key(float x) {
  x = (x != x) ? -INFINITY : x + 0.f;
  const unsigned u = __float_as_uint(x);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive prefix sum over the block; `sum` becomes the block's total.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T *warp_sum, T &sum) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const T y = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += y;
  }
  __syncthreads();  // warp_sum may still be read from an earlier scan
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  T before = 0;
  sum = 0;
#pragma unroll
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const T x = warp_sum[w];
    if (w < warp) before += x;
    sum += x;
  }
  return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads)
    select_kernel(const EvictParams p, int cache_cap) {
  extern __shared__ unsigned keys[];
  __shared__ SelShared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x;
  const int group = blockIdx.x / nc;
  const int b = group / p.num_kv_heads, g = group % p.num_kv_heads;
  pdl_wait();
  pdl_launch_dependents();
  int32_t *const kept = p.kept + (size_t)group * p.budget;
  const int L = p.seq_lens[b];
  const bool bad = L < 0 || L > (long long)p.max_blocks * kBlockSize;
  if (bad || L <= p.budget) {  // nothing to choose (uniform over the cluster)
    if (bad && tid == 0 && rank == 0)
      atomicOr(&g_status_evict, (unsigned)SVP_DEV_BAD_SEQ_LEN);
    for (int i = rank * kSelThreads + tid; i < p.budget; i += nc * kSelThreads)
      kept[i] = !bad && i < L ? i : -1;
    return;
  }
  // this CTA's positions [lo, hi), thread's run of `run` of them: odd, so
  // that a warp's runs start in different banks
  const int per = (L + nc - 1) / nc;
  const int lo = min(rank * per, L), hi = min(lo + per, L);
  const int run = ((per + kSelThreads - 1) / kSelThreads) | 1;
  const bool cached = per <= cache_cap;
  const int mid0 = p.n_sink, mid1 = L - p.n_recent;  // the candidates
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  auto load_key = [&](int j) {
    const int phys = __ldg(table + j / kBlockSize);
    if (phys < 0 || phys >= p.num_blocks) {
      atomicOr(&g_status_evict, (unsigned)SVP_DEV_BAD_BLOCK_ID);
      return score_key(-INFINITY);
    }
    return score_key(p.scores[((size_t)phys * p.num_kv_heads + g) * kBlockSize +
                              j % kBlockSize]);
  };
  auto key_of = [&](int j) { return cached ? keys[j - lo] : load_key(j); };

  // ---- the k-th largest candidate ----
  const unsigned k = (unsigned)(p.budget - p.n_sink - p.n_recent);
  unsigned need = k;       // candidates still to take among those that match
  unsigned prefix = 0;     // the threshold's bits found so far
  for (int i = tid; i < 2 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
  __syncthreads();
  if (cached) {
#pragma unroll 4
    for (int j = lo + tid; j < hi; j += kSelThreads) {
      const unsigned key = load_key(j);
      keys[j - lo] = key;
      if (j >= mid0 && j < mid1) atomicAdd(&sm.hist[0][key >> 21], 1u);
    }
  }
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    unsigned *const hist = sm.hist[pass & 1];
    if (pass > 0 || !cached) {
      for (int j = max(lo, mid0) + tid; j < min(hi, mid1); j += kSelThreads) {
        const unsigned key = key_of(j);
        if (pass == 0 || (key >> (shift + bits)) == (prefix >> (shift + bits)))
          atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
      }
    }
    if (nc > 1) cluster.sync(); else __syncthreads();
    // bins from the largest down, four per thread, summed over the cluster
    unsigned c[4], mine = 0;
    const int top = (1 << bits) - 1 - 4 * tid;  // this thread: top .. top - 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 0;
      if (top - i >= 0)
        for (int r = 0; r < nc; ++r)
          c[i] += nc > 1 ? cluster.map_shared_rank(hist, r)[top - i] : hist[top - i];
      mine += c[i];
    }
    unsigned all;
    unsigned above = block_scan<unsigned>(
        mine, reinterpret_cast<unsigned *>(sm.warp_sum), all);
    if (above < need && above + mine >= need) {  // exactly one thread
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + c[i] >= need) {
          sm.bin = (unsigned)(top - i);
          sm.above = above;
          above = need;  // found
        } else {
          above += c[i];
        }
      }
    }
    if (need == 0 && tid == 0) {  // nothing to take: above every key
      sm.bin = (1u << bits) - 1u;
      sm.above = 0;
    }
    __syncthreads();
    prefix |= sm.bin << shift;
    need -= sm.above;
    // the other histogram is free (its readers passed the barrier above)
    // and is counted into after the next clearing
    unsigned *const next = sm.hist[(pass & 1) ^ 1];
    if (pass == 1)
      for (int i = tid; i < kBins; i += kSelThreads) next[i] = 0;
    __syncthreads();
  }
  // kept: keys above `prefix`, and the first `need` of those equal to it

  // ---- number the kept positions ----
  const int j_begin = min(lo + tid * run, hi), j_end = min(j_begin + run, hi);
  unsigned sure = 0, tied = 0;
  for (int j = j_begin; j < j_end; ++j) {
    const unsigned key = key_of(j);
    const bool forced = j < mid0 || j >= mid1;
    sure += forced || (k > 0 && key > prefix);
    tied += !forced && key == prefix;
  }
  unsigned long long sum;
  const unsigned long long mine = ((unsigned long long)sure << 32) | tied;
  unsigned long long before = block_scan<unsigned long long>(mine, sm.warp_sum, sum);
  if (nc > 1) {
    if (tid == 0) sm.total = sum;
    cluster.sync();
    for (int r = 0; r < rank; ++r)
      before += *cluster.map_shared_rank(&sm.total, r);
  }
  unsigned n_sure = (unsigned)(before >> 32), n_tied = (unsigned)before;
  for (int j = j_begin; j < j_end; ++j) {
    const unsigned key = key_of(j);
    const bool forced = j < mid0 || j >= mid1;
    const bool is_tied = !forced && key == prefix;
    if (forced || (k > 0 && key > prefix) || (is_tied && n_tied < need))
      kept[n_sure + min(n_tied, need)] = j;
    n_sure += forced || (k > 0 && key > prefix);
    n_tied += is_tied;
  }
  if (nc > 1) cluster.sync();  // no CTA leaves while its totals may be read
}

// ---- the move ----
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;

// Rows of `units` vectors of type V.  Side 0: K, 1: V (blockIdx.y), in
// `splits` parts; side 2: the scores, as rows of one 4-byte unit.
template <typename V>
__device__ __forceinline__ void move_rows(const EvictParams &p, char *data,
                                          int units, int b, int g, int part,
                                          int parts, long long *src_row,
                                          long long *dst_row) {
  const int tid = threadIdx.x;
  const int group = b * p.num_kv_heads + g;
  const int32_t *const kept = p.kept + (size_t)group * p.budget;
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  const int32_t *const dtable = p.dst_table + (size_t)b * p.dst_blocks;
  // a sequence is compacted in place iff its first destination page is its
  // first source page; its parts then take columns instead of rows, so that
  // no part writes what another has still to read
  const bool in_place = dtable[0] == table[0];
  int r0 = 0, r1 = p.budget, u0 = 0, u1 = units;
  if (in_place) {
    u0 = units * part / parts;
    u1 = units * (part + 1) / parts;
  } else {
    r0 = (int)((long long)p.budget * part / parts);
    r1 = (int)((long long)p.budget * (part + 1) / parts);
  }
  const int nu = u1 - u0;
  if (nu <= 0) return;
  for (int base = r0; base < r1; base += kMoveThreads) {
    const int n = min(kMoveThreads, r1 - base);
    // addresses of up to 256 rows, one row per thread
    __syncthreads();  // the previous rows' addresses have been used
    if (tid < n) {
      long long s = -1, d = -1;
      const int slot = base + tid, from = kept[slot];
      if (from >= 0) {
        const int ps = table[from / kBlockSize], pd = dtable[slot / kBlockSize];
        if (ps >= 0 && ps < p.num_blocks && pd >= 0 && pd < p.num_blocks) {
          s = ((long long)ps * p.num_kv_heads + g) * kBlockSize + from % kBlockSize;
          d = ((long long)pd * p.num_kv_heads + g) * kBlockSize + slot % kBlockSize;
          if (s == d) s = -1;  // already there
        } else {
          atomicOr(&g_status_evict, (unsigned)SVP_DEV_BAD_BLOCK_ID);
        }
      }
      src_row[tid] = s;
      dst_row[tid] = d;
    }
    const int some = __syncthreads_or(tid < n && src_row[tid] >= 0);
    if (!some) continue;
    const int total = n * nu;
    for (int i0 = 0; i0 < total; i0 += kMoveThreads * kMoveUnroll) {
      V v[kMoveUnroll];
      long long to[kMoveUnroll];
#pragma unroll
      for (int x = 0; x < kMoveUnroll; ++x) {
        const int i = i0 + x * kMoveThreads + tid;
        to[x] = -1;
        if (i < total) {
          const int r = i / nu, u = u0 + i % nu;
          if (src_row[r] >= 0) {
            v[x] = reinterpret_cast<const V *>(data)[src_row[r] * units + u];
            to[x] = dst_row[r] * units + u;
          }
        }
      }
      if (in_place) __syncthreads();  // the batch is read before it is written
#pragma unroll
      for (int x = 0; x < kMoveUnroll; ++x)
        if (to[x] >= 0) reinterpret_cast<V *>(data)[to[x]] = v[x];
    }
  }
}

template <typename V>
__global__ void __launch_bounds__(kMoveThreads)
    compact_kernel(const EvictParams p, int parts) {
  __shared__ long long src_row[kMoveThreads], dst_row[kMoveThreads];
  pdl_wait();  // the selection
  pdl_launch_dependents();
  const int part = blockIdx.x % parts, group = blockIdx.x / parts;
  const int b = group / p.num_kv_heads, g = group % p.num_kv_heads;
  const int side = blockIdx.y;
  if (side < 2) {
    move_rows<V>(p, static_cast<char *>(side ? p.v_cache : p.k_cache),
                 p.row_bytes / (int)sizeof(V), b, g, part, parts, src_row,
                 dst_row);
    return;
  }
  if (part != 0) return;
  move_rows<uint32_t>(p, reinterpret_cast<char *>(p.scores), 1, b, g, 0, 1,
                      src_row, dst_row);
  if (g == 0 && threadIdx.x == 0) {
    const int L = p.seq_lens[b];
    const bool bad = L < 0 || L > (long long)p.max_blocks * kBlockSize;
    p.new_lens[b] = bad ? -1 : min(L, p.budget);
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams &p, int sms, cudaStream_t stream) {
  const long long groups = (long long)p.batch * p.num_kv_heads;
  const long long max_len = (long long)p.max_blocks * kBlockSize;
  // a CTA chooses among about 4096 positions: eight keys per thread
  int nc = 1;
  while (nc < kMaxCluster && max_len > (long long)nc * kSelRun) nc *= 2;
  if (groups * nc > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const long long per = (max_len + nc - 1) / nc;
  const int cap = (int)(per < kSelCache ? per : kSelCache);
  const size_t smem = (size_t)cap * sizeof(unsigned);
  cudaError_t e = cudaSuccess;
  if (smem > 24 * 1024) {  // beyond 48 KB with the static part
    e = cudaFuncSetAttribute(select_kernel,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSelCache * (int)sizeof(unsigned));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(groups * nc));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, select_kernel, p, cap);
  if (e != cudaSuccess) return e;

  // parts of a group's K or V: enough CTAs to fill the SMs, none with fewer
  // than 128 rows
  long long parts = ((long long)sms * 8 + 2 * groups - 1) / (2 * groups);
  const long long most = (p.budget + 127) / 128;
  if (parts > most) parts = most;
  if (parts > 16) parts = 16;
  if (groups * parts > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)(groups * parts), 3);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  // the widest vector that divides a row: 16 bytes, or 8 / 4 for the 72- and
  // 36-byte rows of a 4-bit cache
  if (p.row_bytes % 16 == 0)
    return cudaLaunchKernelEx(&cfg, compact_kernel<uint4>, p, (int)parts);
  if (p.row_bytes % 8 == 0)
    return cudaLaunchKernelEx(&cfg, compact_kernel<uint2>, p, (int)parts);
  return cudaLaunchKernelEx(&cfg, compact_kernel<uint32_t>, p, (int)parts);
}

cudaError_t read_status_evict(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_evict, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_evict, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
