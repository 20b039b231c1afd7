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
//    the cluster through distributed shared memory.  Bound by latency, not
//    by the scores' bytes: a load of page id and scores, three rounds of
//    histogram, cluster barrier and scan, and the numbering (131,072
//    positions on eight CTAs: 12-16, 10, 10, 5 and 14 thousand cycles, 27 us;
//    the 17 MB of scores of 32 such groups are 2.5 us).  Sixteen CTAs per
//    cluster were slower (four sequences of 131,072: 1.3 times the whole call:
//    such clusters find room on few GPCs at a time), and so were four keys to
//    a read in the later passes on short contexts, and eight warps for groups
//    of one CTA (32 x 32 heads of up to 4096: 1.18 times the whole call).
//  * compact_kernel: moves the kept rows of K, V and the scores, a cluster to
//    a group and side.  Bound by the moved bytes, read and written; scattered
//    72-byte rows read 2.3 times their bytes (partial sectors and bursts).
// Measured (both kernels, call times): 32 sequences of 32 heads, 2200 to 4096
// positions, 2048 kept, bf16 rows of 256 bytes: 352 us to other pages, 0.92 of
// the bytes' time at the copy rate, and 356 in place; one sequence of 8 heads,
// 1024 of 1087: 9.1 us; 4096 of 4200: 24 and 21; 16,384 of 131,072 4-bit rows,
// one sequence 45 and 48, four 89 and 94.
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
  alignas(16) unsigned hist[2][kBins];
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
  // every warp scans the warps' sums
  constexpr int NW = kSelThreads / 32;
  static_assert(NW == 16, "four steps");
  const T x = lane < NW ? warp_sum[lane] : T(0);
  T y = x;
#pragma unroll
  for (int off = 1; off < NW; off <<= 1) {
    const T z = __shfl_up_sync(kFull, y, off);
    if (lane >= off) y += z;
  }
  sum = __shfl_sync(kFull, y, NW - 1);
  return __shfl_sync(kFull, y - x, warp) + incl - v;
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
    for (unsigned i = rank * kSelThreads + tid; i < (unsigned)p.budget;
         i += nc * kSelThreads)
      kept[i] = !bad && (int)i < L ? (int)i : -1;
    return;
  }
  // this CTA's positions [lo, hi): whole pages
  const int per = ((L + nc - 1) / nc + kBlockSize - 1) / kBlockSize * kBlockSize;
  const int lo = min(rank * per, L), hi = min(lo + per, L);
  const bool cached = per <= cache_cap;
  const int mid0 = p.n_sink, mid1 = L - p.n_recent;  // the candidates
  const int c0 = max(lo, mid0), c1 = min(hi, mid1);  // this CTA's
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  // where position j's page keeps this head's scores, or null
  auto page_scores = [&](int j) -> const float * {
    const int phys = __ldg(table + j / kBlockSize);
    if (phys < 0 || phys >= p.num_blocks) {
      atomicOr(&g_status_evict, (unsigned)SVP_DEV_BAD_BLOCK_ID);
      return nullptr;
    }
    return p.scores + ((size_t)phys * p.num_kv_heads + g) * kBlockSize;
  };
  auto key_of = [&](int j) {
    if (cached) return keys[j - lo];
    const float *at = page_scores(j);
    return score_key(at ? at[j % kBlockSize] : -INFINITY);
  };

  // ---- the k-th largest candidate ----
  const unsigned k = (unsigned)(p.budget - p.n_sink - p.n_recent);
  unsigned need = k;       // candidates still to take among those that match
  unsigned prefix = 0;     // the threshold's bits found so far
  for (int i = tid; i < 2 * kBins / 4; i += kSelThreads)
    reinterpret_cast<uint4 *>(&sm.hist[0][0])[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
  if (cached) {
    // four positions of a page at a time, all loads of up to 16 in flight.  lo
    // is a page's start, or L where the sequence ends before this CTA's run (a
    // short sequence in a wide table): rounded up, so that no thread of such a
    // CTA takes the last, partial four of another's
    constexpr int U = 4;
    for (int q0 = (lo + 3) / 4 + tid; q0 * 4 < hi; q0 += U * kSelThreads) {
      const float *at[U];
      float4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (q0 + u * kSelThreads) * 4;
        at[u] = j < hi ? page_scores(j) : nullptr;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (q0 + u * kSelThreads) * 4;
        v[u] = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (at[u]) v[u] = *reinterpret_cast<const float4 *>(at[u] + j % kBlockSize);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = (q0 + u * kSelThreads) * 4;
        if (j >= hi) continue;
        const unsigned key[4] = {score_key(v[u].x), score_key(v[u].y),
                                 score_key(v[u].z), score_key(v[u].w)};
        *reinterpret_cast<uint4 *>(keys + (j - lo)) =
            make_uint4(key[0], key[1], key[2], key[3]);
        const bool inside = j >= c0 && j + 4 <= c1;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (inside || (j + e >= c0 && j + e < c1))
            atomicAdd(&sm.hist[0][key[e] >> 21], 1u);
      }
    }
  }
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bits = pass == 2 ? 10 : 11;
    unsigned *const hist = sm.hist[pass & 1];
    // (shift + bits is 32 in the first pass: everything matches)
    const int above_bits = pass == 0 ? 31 : shift + bits;
    const unsigned match = pass == 0 ? 0u : prefix >> above_bits;
    auto tally = [&](unsigned key) {
      if (pass == 0 || (key >> above_bits) == match)
        atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1u);
    };
    if (pass > 0 || !cached) {
      for (int j = c0 + tid; j < c1; j += kSelThreads) tally(key_of(j));
    }
    if (nc > 1) cluster.sync(); else __syncthreads();
    // bins from the largest down, four per thread, summed over the cluster
    // (one 16-byte read of every CTA, all in flight)
    const int quad = (1 << bits) / 4 - 1 - tid;  // this thread's four bins
    uint4 q4 = make_uint4(0, 0, 0, 0);
    if (quad >= 0 && nc == 1) {
      q4 = reinterpret_cast<const uint4 *>(hist)[quad];
    } else if (quad >= 0) {
      uint4 part[kMaxCluster];
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        part[r] = make_uint4(0, 0, 0, 0);
        if (r < nc)
          part[r] = reinterpret_cast<const uint4 *>(
              cluster.map_shared_rank(hist, r))[quad];
      }
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        q4.x += part[r].x;
        q4.y += part[r].y;
        q4.z += part[r].z;
        q4.w += part[r].w;
      }
    }
    const unsigned c[4] = {q4.w, q4.z, q4.y, q4.x};
    const unsigned mine = c[0] + c[1] + c[2] + c[3];
    unsigned all;
    unsigned above = block_scan<unsigned>(
        mine, reinterpret_cast<unsigned *>(sm.warp_sum), all);
    if (above < need && above + mine >= need) {  // exactly one thread
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (above < need && above + c[i] >= need) {
          sm.bin = (unsigned)(4 * quad + 3 - i);
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
    // the first histogram is free (its readers passed the barrier above) and
    // serves the last pass
    if (pass == 1)
      reinterpret_cast<uint4 *>(sm.hist[0])[tid] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    prefix |= sm.bin << shift;
    need -= sm.above;
  }
  // kept: keys above `prefix`, and the first `need` of those equal to it

  // ---- number the kept positions ----
  // a warp numbers a run of them, 32 at a time: once to count, and once more,
  // with the counts before it known, to write
  constexpr int NW = kSelThreads / 32;
  const int lane = tid & 31, warp = tid >> 5;
  const int w_run = (per + 32 * NW - 1) / (32 * NW) * 32;
  const int w0 = min(lo + warp * w_run, hi), w1 = min(w0 + w_run, hi);
  auto look = [&](int j, bool &for_sure, bool &is_tied) {
    for_sure = is_tied = false;
    if (j < w1) {
      const unsigned key = key_of(j);
      const bool forced = j < mid0 || j >= mid1;
      for_sure = forced || key > prefix;  // (k = 0: no key is above)
      is_tied = !forced && key == prefix;
    }
  };
  unsigned sure = 0, tied = 0;
#pragma unroll 4
  for (int j = w0; j < w1; j += 32) {
    bool a, t;
    look(j + lane, a, t);
    sure += __popc(__ballot_sync(kFull, a));
    tied += __popc(__ballot_sync(kFull, t));
  }
  unsigned long long sum;
  unsigned long long before = block_scan<unsigned long long>(
      lane == 0 ? ((unsigned long long)sure << 32) | tied : 0, sm.warp_sum, sum);
  before = __shfl_sync(kFull, before, 0);
  if (nc > 1) {
    if (tid == 0) sm.total = sum;
    cluster.sync();
    for (int r = 0; r < rank; ++r)
      before += *cluster.map_shared_rank(&sm.total, r);
  }
  unsigned n_sure = (unsigned)(before >> 32), n_tied = (unsigned)before;
  const unsigned lower = (1u << lane) - 1u;
#pragma unroll 4
  for (int j = w0; j < w1; j += 32) {
    bool a, t;
    look(j + lane, a, t);
    const unsigned all_a = __ballot_sync(kFull, a);
    const unsigned all_t = __ballot_sync(kFull, t);
    const unsigned ties = n_tied + __popc(all_t & lower);
    if (a || (t && ties < need))
      kept[n_sure + __popc(all_a & lower) + min(ties, need)] = j + lane;
    n_sure += __popc(all_a);
    n_tied += __popc(all_t);
  }
  if (nc > 1) cluster.sync();  // no CTA leaves while its totals may be read
}

// ---- the move ----
constexpr int kMoveWarps = 8;
constexpr int kMoveRows = 128;  // rows whose addresses a warp works out at once

// Vectors a lane has in flight, of rows of NU vectors, and the rows they make
// for a warp: about 16 vectors (with 8, evictions in place took 4-12% longer).
template <int NU>
__host__ __device__ constexpr int move_vectors() {
  return NU == 9 ? 18 : NU * (kMoveRows / 32) < 16 ? NU * (kMoveRows / 32) : 16;
}
template <int NU>
__host__ __device__ constexpr int move_step() {
  return move_vectors<NU>() * 32 / NU;
}

// The kept rows of one (sequence, head) on one side, by a cluster: rows of NU
// vectors of type V.  A step is R consecutive slots for each of the cluster's
// warps; a warp works out the addresses of 128 of its rows at once, then takes
// them step by step, all of a step's vectors (up to 18 per lane) in flight.
// In place, every warp's reads of a step come before any warp's writes of it
// (one barrier): slot i's source is row i or a later one, so no step writes
// what a later step reads.  Pages of the call's own need no barrier.
template <typename V, int NU>
__device__ __forceinline__ void move_rows(const EvictParams &p, V *data, int b,
                                          int g, bool in_place, int nc, int rank,
                                          long long *from, long long *to) {
  constexpr int RPL = kMoveRows / 32;
  constexpr int U = move_vectors<NU>(), R = move_step<NU>();
  static_assert(U * 32 % NU == 0 && kMoveRows % R == 0, "whole rows and steps");
  const int lane = threadIdx.x & 31;
  const int me = rank * kMoveWarps + (threadIdx.x >> 5);
  const unsigned stride = nc * kMoveWarps * R;  // slots of a step
  const unsigned budget = p.budget;
  const int32_t *const kept =
      p.kept + (size_t)(b * p.num_kv_heads + g) * p.budget;
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  const int32_t *const dtable = p.dst_table + (size_t)b * p.dst_blocks;
  for (unsigned base = 0; base < budget; base += stride * (kMoveRows / R)) {
    // this warp's row i: step i / R, row i % R of its R
    auto slot_of = [&](int i) {
      return base + (unsigned)(i / R) * stride + me * R + i % R;
    };
    int pos[RPL], ps[RPL], pd[RPL];
#pragma unroll
    for (int x = 0; x < RPL; ++x) {
      const unsigned slot = slot_of(x * 32 + lane);
      pos[x] = slot < budget ? kept[slot] : -1;
    }
#pragma unroll
    for (int x = 0; x < RPL; ++x) {
      ps[x] = pd[x] = -1;
      if (pos[x] >= 0) {
        ps[x] = table[pos[x] / kBlockSize];
        pd[x] = dtable[slot_of(x * 32 + lane) / kBlockSize];
      }
    }
    __syncwarp();  // the addresses before have been used
#pragma unroll
    for (int x = 0; x < RPL; ++x) {
      long long s = -1, d = -1;
      if (pos[x] >= 0) {
        if (ps[x] >= 0 && ps[x] < p.num_blocks && pd[x] >= 0 &&
            pd[x] < p.num_blocks) {
          s = ((long long)ps[x] * p.num_kv_heads + g) * kBlockSize +
              pos[x] % kBlockSize;
          d = ((long long)pd[x] * p.num_kv_heads + g) * kBlockSize +
              slot_of(x * 32 + lane) % kBlockSize;
          if (s == d) s = -1;  // already there
        } else {
          atomicOr(&g_status_evict, (unsigned)SVP_DEV_BAD_BLOCK_ID);
        }
      }
      from[x * 32 + lane] = s < 0 ? -1 : s * NU;
      to[x * 32 + lane] = d * NU;
    }
    __syncwarp();
#pragma unroll 1
    for (int k = 0; k < kMoveRows / R; ++k) {
      if (base + k * stride >= budget) break;  // the same for all
      V v[U];
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int i = x * 32 + lane;
        const long long at = from[k * R + i / NU];
        if (at >= 0) v[x] = data[at + i % NU];
      }
      if (in_place) {
        if (nc > 1) cg::this_cluster().sync(); else __syncthreads();
      }
#pragma unroll
      for (int x = 0; x < U; ++x) {
        const int i = x * 32 + lane;
        if (from[k * R + i / NU] >= 0) data[to[k * R + i / NU] + i % NU] = v[x];
      }
    }
  }
}

// A cluster per group and side: side 0 K, 1 V, 2 the scores.  In place means:
// the first destination page is the first source page.
template <typename V, int UNITS>
__global__ void __launch_bounds__(32 * kMoveWarps)
    compact_kernel(const EvictParams p) {
  __shared__ long long from[kMoveWarps][kMoveRows], to[kMoveWarps][kMoveRows];
  const int nc = (int)cg::this_cluster().num_blocks();
  const int rank = (int)cg::this_cluster().block_rank();
  pdl_wait();  // the selection
  pdl_launch_dependents();
  const int w = threadIdx.x >> 5;
  const int side = blockIdx.y;
  const int group = blockIdx.x / nc;
  const int b = group / p.num_kv_heads, g = group % p.num_kv_heads;
  if (side == 2 && g == 0 && rank == 0 && threadIdx.x == 0) {
    const int L = p.seq_lens[b];
    const bool bad = L < 0 || L > (long long)p.max_blocks * kBlockSize;
    p.new_lens[b] = bad ? -1 : min(L, p.budget);
  }
  const bool in_place = p.dst_table[(size_t)b * p.dst_blocks] ==
                        p.block_table[(size_t)b * p.max_blocks];
  if (side == 2)
    move_rows<float, 1>(p, p.scores, b, g, in_place, nc, rank, from[w], to[w]);
  else
    move_rows<V, UNITS>(p, static_cast<V *>(side ? p.v_cache : p.k_cache), b, g,
                        in_place, nc, rank, from[w], to[w]);
}

template <typename V, int UNITS>
cudaError_t launch_compact(const EvictParams &p, int sms, cudaLaunchConfig_t cfg) {
  const long long groups = (long long)p.batch * p.num_kv_heads;
  // enough CTAs for 32 warps on every SM, but no more than one step's rows
  int nc = 1;
  while (nc < kMaxCluster && 2 * groups * nc < 4LL * sms &&
         nc * kMoveWarps * move_step<UNITS>() < p.budget)
    nc *= 2;
  if (groups * nc > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)(groups * nc), 3);
  cfg.blockDim = dim3(32 * kMoveWarps);
  cfg.dynamicSmemBytes = 0;
  cfg.attrs[1].val.clusterDim.x = (unsigned)nc;
  cfg.numAttrs = nc > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, compact_kernel<V, UNITS>, p);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams &p, int sms, cudaStream_t stream) {
  const long long groups = (long long)p.batch * p.num_kv_heads;
  const long long max_len = (long long)p.max_blocks * kBlockSize;
  // a CTA chooses among about 4096 positions: eight keys per thread
  int nc = 1;
  while (nc < kMaxCluster && max_len > (long long)nc * kSelRun) nc *= 2;
  if (groups * nc > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const long long per =
      ((max_len + nc - 1) / nc + kBlockSize - 1) / kBlockSize * kBlockSize;
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

  // vectors of 16 bytes, or 8 / 4 for the 72- and 36-byte rows of a 4-bit
  // cache
  switch (p.row_bytes) {
    case 36: return launch_compact<uint32_t, 9>(p, sms, cfg);
    case 72: return launch_compact<uint2, 9>(p, sms, cfg);
    case 64: return launch_compact<uint4, 4>(p, sms, cfg);
    case 128: return launch_compact<uint4, 8>(p, sms, cfg);
    case 256: return launch_compact<uint4, 16>(p, sms, cfg);
    default: return launch_compact<uint4, 32>(p, sms, cfg);  // 512
  }
}

cudaError_t status_word_evict(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_evict);
}

}  // namespace svp
