// logprobs.cu -- log probabilities of given tokens, their ranks, the rows'
// entropies and most likely alternatives (token_logprobs, include/svp.h).
//
// With z = x / T over the allowed tokens of a row, m = max x and
// S = sum exp((x - m) / T):
//   log p(t)  = (x_t - m) / T - ln S
//   entropy   = ln S - (1 / S) sum ((x - m) / T) exp((x - m) / T)
// so one maximum and one pass of exponentials give everything but the order.
//
// A cluster of 1 to 8 CTAs takes a row; every thread keeps its part of the row
// in registers, so the logits are read once.  The alternatives: the k-th
// largest of the threads' own largest values bounds the k-th largest of all
// from below, and few elements reach that bound; they are gathered and ranked
// by counting.  Where many do (equal logits), the k-th largest is found bit by
// bit instead.  Equal logits are ordered by token, so no result depends on
// the order of atomics.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"

namespace svp {

static __device__ unsigned int g_status_logprobs;

namespace {

namespace cg = cooperative_groups;

constexpr int kLpThreads = 512;
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kLpCluster = 8;
constexpr int kLpFound = 512;  // candidates ranked by counting

struct Found {
  unsigned key;
  int token;
};
struct LpShared {
  Found found[kLpFound];
  Found best[kMaxTop];     // this CTA's alternatives, in order
  Found all[kLpCluster * kMaxTop];
  float warp_f[kLpWarps][2];
  unsigned warp_u[2][kLpWarps];
  float top;               // this CTA's largest logit
  float sum, sum_z;        // relative to the row's
  unsigned ahead, n_found, n_best;
};

// Ascending order of logits; NaN above everything, -0 as +0.  0: no logit
// (not allowed, or -inf).
__device__ __forceinline__ unsigned logit_key(float x) {
  if (x != x) return 0xffffffffu;
  if (x == -INFINITY) return 0u;
  const unsigned u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float key_logit(unsigned k) {
  if (k == 0xffffffffu) return NAN;
  return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ unsigned lp_sum(unsigned v, LpShared &sm, int round) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = __reduce_add_sync(kFull, v);
  unsigned *const row = sm.warp_u[round & 1];
  if (lane == 0) row[warp] = v;
  __syncthreads();
  return __reduce_add_sync(kFull, lane < kLpWarps ? row[lane] : 0u);
}

template <int DT, int NV>  // NV: 16-byte vectors of a thread
__global__ void __launch_bounds__(kLpThreads)
    token_logprobs_kernel(const LogprobParams p) {
  constexpr int VEC = DT == SVP_F32 ? 4 : 8;
  constexpr int SIZE = 16 / VEC;
  __shared__ LpShared sm;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t row = blockIdx.x / (unsigned)nc;
  pdl_wait();
  pdl_launch_dependents();
  const int token = p.tokens[row];
  if (token < 0 || token >= p.vocab) {  // padding, or no token: nothing is read
    if (rank == 0) {
      if (tid == 0) {
        if (token >= 0) atomicOr(&g_status_logprobs, (unsigned)SVP_DEV_BAD_TOKEN);
        p.logprobs[row] = 0.f;
        if (p.entropy) p.entropy[row] = 0.f;
        if (p.ranks) p.ranks[row] = -1;
      }
      for (int i = tid; i < p.n_top; i += kLpThreads) {
        p.top_logprobs[row * p.n_top + i] = -INFINITY;
        p.top_tokens[row * p.n_top + i] = -1;
      }
    }
    return;  // the whole cluster
  }

  // ---- the row into registers ----
  // Rows start anywhere: vectors are aligned ones that cover the row, the
  // first and the last may hold less than VEC of its elements.
  const char *const base = static_cast<const char *>(p.logits) +
                           row * (size_t)p.vocab * SIZE;
  const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / SIZE;
  const char *const aligned = base - shift * SIZE;
  const int n_vec = (shift + p.vocab + VEC - 1) / VEC;
  const uint32_t *const allowed =
      p.allowed ? p.allowed + row * (size_t)p.words : nullptr;
  uint4 raw[NV];
  uint32_t bits[NV];  // which elements take part
  auto vec_of = [&](int i) { return (i * nc + rank) * kLpThreads + tid; };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = vec_of(i);
    raw[i] = make_uint4(0, 0, 0, 0);
    bits[i] = 0u;
    if (v < n_vec) {
      const int t0 = v * VEC - shift;  // token of the vector's first element
      if (t0 >= 0 && t0 + VEC <= p.vocab) {
        raw[i] = __ldg(reinterpret_cast<const uint4 *>(aligned) + v);
        bits[i] = (1u << VEC) - 1u;
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          if (t0 + e < 0 || t0 + e >= p.vocab) continue;
          bits[i] |= 1u << e;
          if constexpr (DT == SVP_F32)
            w[e] = __ldg(reinterpret_cast<const uint32_t *>(base) + t0 + e);
          else
            w[e / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t *>(base) +
                                        t0 + e) << (16 * (e % 2));
        }
        raw[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  if (allowed) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (bits[i] == 0u) continue;
      // VEC bits from bit t0 on (from bit 0 where the row's first vector
      // starts before it), out of one or two words
      const int t0 = vec_of(i) * VEC - shift;
      const int from = t0 < 0 ? 0 : t0;
      const int w = from >> 5;
      const uint32_t w0 = __ldg(allowed + w);
      const uint32_t w1 = w + 1 < p.words ? __ldg(allowed + w + 1) : 0u;
      const uint32_t m = __funnelshift_r(w0, w1, from & 31);
      bits[i] &= m << (from - t0);
    }
  }
  auto value = [&](int i, int e) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    if constexpr (DT == SVP_F32) return __uint_as_float(w[e]);
    else
      return __uint_as_float(e % 2 ? w[e / 2] & 0xffff0000u : w[e / 2] << 16);
  };
  // the order key of element e of vector i: 0 where it takes no part
  auto key = [&](int i, int e) {
    return (bits[i] >> e) & 1u ? logit_key(value(i, e)) : 0u;
  };

  // ---- the largest logit ----
  unsigned mine = 0;  // this thread's largest key
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) mine = max(mine, key(i, e));
  {
    const unsigned m = __reduce_max_sync(kFull, mine);
    if (lane == 0) sm.warp_u[0][warp] = m;
    __syncthreads();
    const unsigned x =
        __reduce_max_sync(kFull, lane < kLpWarps ? sm.warp_u[0][lane] : 0u);
    if (tid == 0) sm.top = __uint_as_float(x);  // the key's bits
  }
  if (nc > 1) cluster.sync(); else __syncthreads();
  unsigned top_key = 0;
  for (int r = 0; r < nc; ++r)
    top_key = max(top_key, __float_as_uint(nc > 1 ? *cluster.map_shared_rank(&sm.top, r)
                                                  : sm.top));
  const float top = top_key ? key_logit(top_key) : 0.f;

  // ---- sums, and how many are ahead of the token ----
  const bool in_mask = !allowed || ((allowed[token >> 5] >> (token & 31)) & 1u);
  float xt;
  if constexpr (DT == SVP_F32) xt = reinterpret_cast<const float *>(base)[token];
  else
    xt = __uint_as_float((uint32_t)reinterpret_cast<const uint16_t *>(base)[token] << 16);
  const unsigned kt = in_mask ? logit_key(xt) : 0u;
  float s = 0.f, sz = 0.f;
  unsigned ahead = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int t0 = vec_of(i) * VEC - shift;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const unsigned k = key(i, e);
      if (k == 0u) continue;
      const float d = (value(i, e) - top) * p.sc;  // in units of log 2
      const float w = ex2(d);
      s += w;
      sz = fmaf(w, d > -200.f ? d : 0.f, sz);
      ahead += k > kt || (k == kt && t0 + e < token) ? 1u : 0u;
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    s += __shfl_xor_sync(kFull, s, off);
    sz += __shfl_xor_sync(kFull, sz, off);
  }
  if (lane == 0) {
    sm.warp_f[warp][0] = s;
    sm.warp_f[warp][1] = sz;
  }
  const unsigned n_ahead = lp_sum(ahead, sm, 1);  // its barrier serves both
  if (tid == 0) {
    float a = 0.f, c = 0.f;
    for (int w = 0; w < kLpWarps; ++w) {
      a += sm.warp_f[w][0];
      c += sm.warp_f[w][1];
    }
    sm.sum = a;
    sm.sum_z = c;
    sm.ahead = n_ahead;
    sm.n_found = 0;
  }
  __syncthreads();

  // ---- this CTA's alternatives ----
  if (p.n_top > 0) {
    const unsigned k = (unsigned)p.n_top;
    // the largest bound that k threads reach: with fewer threads that hold
    // anything, every element
    unsigned edge = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const unsigned at = edge | (1u << bit);
      if ((unsigned)__syncthreads_count(mine >= at) >= k) edge = at;
    }
    if (edge == 0) edge = 1;
    unsigned reach = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) reach += key(i, e) >= edge ? 1u : 0u;
    unsigned n = lp_sum(reach, sm, 0);
    int last = 0x7fffffff;  // the last token that counts among those at the edge
    if (n > kLpFound) {
      // the k-th largest of all, then the token up to which its equals count
      edge = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const unsigned at = edge | (1u << bit);
        unsigned c = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) c += key(i, e) >= at ? 1u : 0u;
        if (lp_sum(c, sm, bit) >= k) edge = at;
      }
      last = 0;
      for (int bit = 30; bit >= 0; --bit) {
        // do fewer than k come before token `at`?
        const int at = last | (1 << bit);
        unsigned c = 0;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const unsigned x = key(i, e);
            c += x > edge || (x == edge && vec_of(i) * VEC - shift + e < at) ? 1u : 0u;
          }
        if (lp_sum(c, sm, bit + 1) < k) last = at;  // (+ 1: in turn with the above)
      }
      n = k;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const unsigned x = key(i, e);
        const int t = vec_of(i) * VEC - shift + e;
        if (x > edge || (x == edge && t <= last)) {
          const unsigned at = atomicAdd(&sm.n_found, 1u);
          sm.found[at].key = x;
          sm.found[at].token = t;
        }
      }
    __syncthreads();
    const unsigned keep = min(n, k);
    for (unsigned c = tid; c < n; c += kLpThreads) {
      const Found f = sm.found[c];
      unsigned r = 0;
      for (unsigned o = 0; o < n; ++o) {
        const Found h = sm.found[o];
        r += h.key > f.key || (h.key == f.key && h.token < f.token) ? 1u : 0u;
      }
      if (r < keep) sm.best[r] = f;
    }
    if (tid == 0) sm.n_best = keep;
  }
  if (nc > 1) cluster.sync(); else __syncthreads();

  // ---- the row's results ----
  if (rank == 0) {
    float total = 0.f, total_z = 0.f;
    unsigned n_before = 0;
    for (int r = 0; r < nc; ++r) {
      const LpShared *o = nc > 1 ? cluster.map_shared_rank(&sm, r) : &sm;
      total += o->sum;
      total_z += o->sum_z;
      n_before += o->ahead;
    }
    const float ln = logf(total);
    if (tid == 0) {
      // a row that allows nothing has no probabilities: -inf, entropy 0
      p.logprobs[row] = total != total ? NAN
                        : kt == 0u     ? -INFINITY
                                       : (xt - top) * p.inv_t - ln;
      if (p.entropy)
        p.entropy[row] = top_key == 0u ? 0.f : ln - total_z / total * kLn2;
      if (p.ranks) p.ranks[row] = kt == 0u ? -1 : (int)n_before;
    }
    if (p.n_top > 0) {
      unsigned n = 0, from[kLpCluster + 1];
#pragma unroll
      for (int r = 0; r < kLpCluster; ++r) {
        from[r] = n;
        if (r < nc) n += nc > 1 ? cluster.map_shared_rank(&sm, r)->n_best : sm.n_best;
      }
      from[kLpCluster] = n;
#pragma unroll
      for (int r = 0; r < kLpCluster; ++r) {
        const unsigned c = from[r + 1] - from[r];
        if (r < nc)
          for (unsigned i = tid; i < c; i += kLpThreads)
            sm.all[from[r] + i] =
                nc > 1 ? cluster.map_shared_rank(&sm, r)->best[i] : sm.best[i];
      }
      __syncthreads();
      for (unsigned c = tid; c < n; c += kLpThreads) {
        const Found f = sm.all[c];
        unsigned r = 0;
        for (unsigned o = 0; o < n; ++o) {
          const Found h = sm.all[o];
          r += h.key > f.key || (h.key == f.key && h.token < f.token) ? 1u : 0u;
        }
        if (r < (unsigned)p.n_top) {
          p.top_logprobs[row * p.n_top + r] = (key_logit(f.key) - top) * p.inv_t - ln;
          p.top_tokens[row * p.n_top + r] = f.token;
        }
      }
      for (unsigned i = n + tid; i < (unsigned)p.n_top; i += kLpThreads) {
        p.top_logprobs[row * p.n_top + i] = -INFINITY;
        p.top_tokens[row * p.n_top + i] = -1;
      }
    }
  }
  if (nc > 1) cluster.sync();  // results may still be read
}

template <int DT, int NV>
cudaError_t logprobs_t(const LogprobParams &p, int nc, cudaStream_t stream) {
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.rows * nc));
  cfg.blockDim = dim3(kLpThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<DT, NV>, p);
}

template <int DT>
cudaError_t logprobs_dt(const LogprobParams &p, int sms, cudaStream_t stream) {
  constexpr int VEC = DT == SVP_F32 ? 4 : 8;
  // vectors of a row, one more where it starts off a 16-byte boundary
  const int vecs = (p.vocab + 2 * VEC - 2) / VEC;
  const int per_cta = (vecs + kLpThreads - 1) / kLpThreads;  // of a thread, nc = 1
  // few rows: more CTAs to a row; long rows: as many as keep a thread's part
  // in 8 vectors
  int nc = 1;
  while (nc < kLpCluster && per_cta > nc &&
         (per_cta > 8 * nc || (long long)p.rows * nc < 2LL * sms))
    nc *= 2;
  const int nv = (per_cta + nc - 1) / nc;
  if (nv <= 1) return logprobs_t<DT, 1>(p, nc, stream);
  if (nv <= 2) return logprobs_t<DT, 2>(p, nc, stream);
  if (nv <= 4) return logprobs_t<DT, 4>(p, nc, stream);
  if (nv <= 8) return logprobs_t<DT, 8>(p, nc, stream);
  if (nv <= 20) return logprobs_t<DT, 20>(p, nc, stream);
  return cudaErrorInvalidConfiguration;  // more than kMaxVocab
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams &p, int dtype, int sms,
                                  cudaStream_t stream) {
  return dtype == SVP_F32 ? logprobs_dt<SVP_F32>(p, sms, stream)
                          : logprobs_dt<SVP_BF16>(p, sms, stream);
}

cudaError_t read_status_logprobs(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_logprobs, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_logprobs, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
