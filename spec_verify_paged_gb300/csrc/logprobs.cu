// logprobs.cu -- log probabilities of given tokens, their ranks, the rows'
// entropies and most likely alternatives (token_logprobs, include/svp.h).
//
// With z = x / T over the allowed tokens of a row, r any logit near the largest
// and S = sum exp((x - r) / T):
//   log p(t)  = (x_t - r) / T - ln S
//   entropy   = ln S - (1 / S) sum ((x - r) / T) exp((x - r) / T)
// A thread moves its r only when a logit exceeds it by a factor 2^8 of
// probability, so one pass of exponentials gives everything but the order.
//
// A cluster of 1 to 8 CTAs takes a row; a thread's vectors lie a CTA's width
// apart.  What bounds it for long rows is instructions, about twelve an element
// (nineteen with a mask and alternatives), and what a CTA does once: so a row
// takes as few CTAs as fill the GPU, two fp32 values are multiplied and added at
// once, what can be done on pairs of bf16 is (the maximum, the count of the
// tokens ahead), and few vectors are looked at again, out of L2, for the
// alternatives.  Tried on 512
// masked rows of 131,072 bf16: the row in registers, with everything unrolled,
// 148 us (waiting for instructions); in shared memory, four CTAs a row, 98.  The
// CTAs' sums meet in the first one's shared memory at the end, by one cluster
// barrier.
//
// The alternatives: the k-th largest of the threads' own largest values bounds
// the k-th largest of all from below, and few elements reach that bound; they
// are gathered and ranked by counting.  Where more than 256 do (equal or evenly
// spread logits), the k-th largest is found bit by bit instead, and then the last
// of its equals by its token's bits: 64 more passes over the CTA's share, out of
// L2 at best (512 rows of 131,072 equal bf16 logits, 20 alternatives, 4.1 ms, fp32
// 5.8; 80 rows of 32,000 0.23).  Equal logits are ordered by token, so no result
// depends on the order of atomics.
//
// Measured: 512 rows of 131,072 bf16: 36 us, 44 with 20 alternatives, 52 with
// those and a mask (0.54, 0.45 and 0.40 of the copy rate; issue active 61 %);
// fp32 54 and 70 (0.73, 0.57).  80 rows of 32,000 fp32, 5 alternatives: 9 us with
// 40 % of them padding, 10.7 with none.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"

namespace svp {

static __device__ unsigned int g_status_logprobs;

namespace {

namespace cg = cooperative_groups;

constexpr int kLpCluster = 8;
constexpr int kLpFound = 256;  // candidates ranked by counting
constexpr int kLpSlack = 8;    // threads more than k that may reach the bound
constexpr int kLpBins = 256;   // over the two octaves below the largest logit

// The two halves of a cluster barrier: what comes before the arrival is visible
// after the wait.
__device__ __forceinline__ void lp_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void lp_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

struct Found {
  unsigned key;
  int token;
};
// Sums of weights w = 2^d and of w d, d = (x - r) / T + e in units of log 2.
struct LpSums {
  float r, e, s, sz;
};
struct LpPart {            // one CTA's share of the row's results
  LpSums sums;
  unsigned ahead, n_best, key;
};
template <int W>
struct LpShared {
  alignas(16) Found found[kLpFound + 1];
  // in the first CTA: the others' best too, n_top of each, keys of 0 where a CTA
  // has fewer
  alignas(16) Found best[kLpCluster * kMaxTop + 1];
  LpPart part[kLpCluster];          // in the first CTA
  LpSums warp_f[W];
  unsigned warp_u[2][W];
  alignas(16) unsigned hist[kLpBins];           // of the threads' largest keys
  unsigned n_found, n_high;
  unsigned short high[32 * W];      // threads that reach the bound
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
constexpr unsigned kLowestKey = 0x00800000u;  // of the lowest finite logit

template <int W>
__device__ __forceinline__ unsigned lp_sum(unsigned v, LpShared<W> &sm, int round) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  v = __reduce_add_sync(kFull, v);
  unsigned *const row = sm.warp_u[round & 1];
  if (lane == 0) row[warp] = v;
  __syncthreads();
  return __reduce_add_sync(kFull, lane < W ? row[lane] : 0u);
}

__device__ __forceinline__ float max_nan_f(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) {
  return __uint_as_float(w & 0xffff0000u);
}

// The bytes of y that the four digits of `sel` name; a digit of 8 and more
// spreads the sign of the byte it names (less 8).
__device__ __forceinline__ uint32_t spread(uint32_t y, uint32_t sel) {
  uint32_t r;
  asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(y), "r"(sel));
  return r;
}

// Two fp32 values at once.
__device__ __forceinline__ uint64_t two(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void parts(uint64_t x, float &lo, float &hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A 16-byte vector of logits.
template <int DT>
struct Vec {
  static constexpr int N = DT == SVP_F32 ? 4 : 8;
  static constexpr uint32_t kNone = DT == SVP_F32 ? 0xff800000u : 0xff80ff80u;
  static constexpr uint32_t kLowest = DT == SVP_F32 ? 0xff7fffffu : 0xff7f0000u;
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(kNone, kNone, kNone, kNone);
  }
  static __device__ __forceinline__ float value(const uint4 &v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == SVP_F32) return __uint_as_float(w[e]);
    else return e % 2 ? hi_f(w[e / 2]) : lo_f(w[e / 2]);
  }
  // the largest element, NaN if there is one
  static __device__ __forceinline__ float top(const uint4 &v) {
    if constexpr (DT == SVP_F32) {
      return max_nan_f(max_nan_f(__uint_as_float(v.x), __uint_as_float(v.y)),
                       max_nan_f(__uint_as_float(v.z), __uint_as_float(v.w)));
    } else {
      const uint32_t m = max_nan_2(max_nan_2(v.x, v.y), max_nan_2(v.z, v.w));
      return max_nan_f(lo_f(m), hi_f(m));
    }
  }
  // elements 2 i and 2 i + 1, nothing as a finite value far below every logit
  // that counts
  static __device__ __forceinline__ uint64_t pair(const uint4 &v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == SVP_F32)
      return two(fmaxf(__uint_as_float(w[2 * i]), -1e30f),
                 fmaxf(__uint_as_float(w[2 * i + 1]), -1e30f));
    uint32_t c;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(c) : "r"(w[i]), "r"(0xf14af14au));  // -1e30
    return two(lo_f(c), hi_f(c));
  }
  // v where bit e of `bits` is set, -inf elsewhere.  Four bits become the sign
  // bits of four bytes, which the byte permutation spreads.
  static __device__ __forceinline__ uint4 masked(const uint4 &v, uint32_t bits) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == SVP_F32) {
      const uint32_t y = (bits & 15u) * 0x10204080u;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = spread(y, 0x8888 + 0x1111 * e);
        w[e] = (w[e] & m) | (kNone & ~m);
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t y = ((bits >> (4 * h)) & 15u) * 0x10204080u;
        const uint32_t m0 = spread(y, 0x9988);
        const uint32_t m1 = spread(y, 0xbbaa);
        w[2 * h] = (w[2 * h] & m0) | (kNone & ~m0);
        w[2 * h + 1] = (w[2 * h + 1] & m1) | (kNone & ~m1);
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Two parts' sums, relative to the larger reference.
__device__ __forceinline__ LpSums join(const LpSums &a, const LpSums &b, float sc) {
  const LpSums &o = a.r >= b.r ? a : b;
  const float da = fmaxf((a.r - o.r) * sc - a.e + o.e, -1e4f);
  const float db = fmaxf((b.r - o.r) * sc - b.e + o.e, -1e4f);
  const float fa = ex2(da), fb = ex2(db);
  return {o.r, o.e, fmaf(a.s, fa, b.s * fb),
          fmaf(a.sz, fa, a.s * (da * fa)) + fmaf(b.sz, fb, b.s * (db * fb))};
}

// The next value above x (x below +inf), as the type has it.
template <int DT>
__device__ __forceinline__ float next_up(float x) {
  constexpr uint32_t ulp = DT == SVP_F32 ? 1u : 0x10000u;
  if (x == 0.f) return __uint_as_float(ulp);
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float((u >> 31) ? u - ulp : u + ulp);
}

template <int DT, int T>
__global__ void __launch_bounds__(T)
    token_logprobs_kernel(const LogprobParams p) {
  using V = Vec<DT>;
  constexpr int VEC = V::N, SIZE = 16 / VEC, W = T / 32;
  __shared__ LpShared<W> sm;
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
      for (int i = tid; i < p.n_top; i += T) {
        p.top_logprobs[row * p.n_top + i] = -INFINITY;
        p.top_tokens[row * p.n_top + i] = -1;
      }
    }
    return;  // the whole cluster
  }
  if (nc > 1) lp_arrive();  // the first CTA's shared memory is there

  // ---- the row ----
  // Rows start anywhere.  The whole aligned vectors are dealt out; what is left
  // before and after them is one extra vector of the first CTA's thread 0 and
  // its second warp's first.
  const char *const base = static_cast<const char *>(p.logits) +
                           row * (size_t)p.vocab * SIZE;
  const int shift = (int)(reinterpret_cast<uintptr_t>(base) & 15u) / SIZE;
  const int f0 = shift ? 1 : 0, f1 = max((shift + p.vocab) / VEC, f0);
  const int part = (f1 - f0 + nc - 1) / nc;
  const int v0 = min(f0 + rank * part, f1);  // this CTA's
  const int n_vec = min(part, f1 - v0);
  const uint4 *const aligned = reinterpret_cast<const uint4 *>(base - shift * SIZE) + v0;
  const int t00 = v0 * VEC - shift;          // the first one's first token
  const uint32_t *const allowed =
      p.allowed ? p.allowed + row * (size_t)p.words : nullptr;
  auto element = [&](int t) {  // logit of token t
    if constexpr (DT == SVP_F32) return reinterpret_cast<const float *>(base)[t];
    else
      return __uint_as_float(
          (uint32_t)reinterpret_cast<const uint16_t *>(base)[t] << 16);
  };
  auto may = [&](int t) {
    return !allowed || ((allowed[t >> 5] >> (t & 31)) & 1u);
  };
  const float xt = element(token);
  const unsigned kt = may(token) ? logit_key(xt) : 0u;
  uint4 extra = V::none();
  const bool has_extra = rank == 0 && warp < 2;  // (the warp)
  const int extra0 = warp == 0 ? 0 : f1 * VEC - shift;  // its tokens
  const int extra1 = warp == 0 ? min(f0 * VEC - shift, p.vocab) : p.vocab;
  if (has_extra && lane == 0) {
    uint32_t w[4] = {V::kNone, V::kNone, V::kNone, V::kNone};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      if (extra0 + e >= extra1 || !may(extra0 + e)) continue;
      const uint32_t u = __float_as_uint(element(extra0 + e));
      if constexpr (DT == SVP_F32) w[e] = u;
      else
        w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | u : (w[e / 2] & 0xffff0000u) | (u >> 16);
    }
    extra = make_uint4(w[0], w[1], w[2], w[3]);
  }

  // the bits of vector i: VEC of them, out of one word or two
  auto bits_of = [&](int i) {
    const int t0 = t00 + i * VEC;
    if (shift == 0) {  // they lie in one byte
      const uint32_t y = *(reinterpret_cast<const unsigned char *>(allowed) + t0 / 8);
      return VEC == 8 ? y : y >> (t0 & 4);
    }
    const uint32_t w0 = allowed[t0 >> 5];
    const uint32_t w1 = (t0 & 31) + VEC > 32 ? allowed[(t0 >> 5) + 1] : 0u;
    return __funnelshift_r(w0, w1, t0 & 31);
  };
  // vector i as it counts: with -inf for what is not allowed
  auto fetch = [&](int i) {
    const uint4 v = aligned[i];
    return allowed ? V::masked(v, bits_of(i)) : v;
  };

  // f(key, token) of every logit of this thread, for rare rows
  auto each = [&](auto f) {
#pragma unroll 1
    for (int i = tid; i < n_vec; i += T) {
      const uint4 v = fetch(i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(logit_key(V::value(v, e)), t00 + i * VEC + e);
    }
    if (has_extra) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) f(logit_key(V::value(extra, e)), extra0 + e);
    }
  };

  if (tid == 0) sm.n_found = sm.n_high = 0;
  for (int i = tid; i < kLpBins; i += T) sm.hist[i] = 0u;

  // ---- sums, the largest logit, and how many are ahead of the token ----
  // Tokens before it are ahead with a logit that is not smaller, those after
  // it with a larger one: not below one of two bounds.  The vector that holds
  // the token counts as after; thread 0 of the cluster adds the equals in it.
  const bool ranked = p.ranks && kt != 0u;
  const bool plain_rank = ranked && xt < INFINITY;
  const float up = next_up<DT>(xt);
  unsigned ahead = 0;
  uint32_t n2 = 0u;  // counts of two halves: exact in bf16 up to 256
  float big = -INFINITY;
  float r = __uint_as_float(V::kLowest);  // the reference, and
  float margin = fminf(8.f / p.sc, 1e30f);  // how far a logit may exceed it
  // The distance to it in units of log 2 is x sc - c, c = r sc: one
  // instruction, exact but for c's rounding, which is kept (LpSums::e).  Where c
  // would not be fine enough (huge logits, extreme temperatures), (x - r) sc.
  const bool mild = p.sc > 1e-20f && p.sc < 1e8f;
  bool fine = false;
  uint64_t minus_c = 0, sums = two(0.f, 0.f), sums_z = two(0.f, 0.f);
  const uint64_t sc2 = two(p.sc, p.sc);
  auto take = [&](const uint4 &v, int t0) {
    const float top = V::top(v);
    big = max_nan_f(big, top);
    if (top > r + margin) {
      const bool was_fine = fine;
      float c0, c1;
      parts(minus_c, c0, c1);
      const float e0 = was_fine ? fmaf(r, p.sc, c0) : 0.f;
      fine = mild && fabsf(top * p.sc) < 0x1p20f;
      const float c = -(top * p.sc);
      minus_c = two(c, c);
      const float e1 = fine ? fmaf(top, p.sc, c) : 0.f;
      const float d = fmaxf((r - top) * p.sc - e0 + e1, -1e4f), f = ex2(d);
      sums_z = fma2(sums, two(d, d), sums_z);
      sums_z = fma2(sums_z, two(f, f), 0ull);
      sums = fma2(sums, two(f, f), 0ull);
      r = top;
    }
    if (top == -INFINITY) return;
    if (fine) {
#pragma unroll
      for (int i = 0; i < VEC / 2; ++i) {
        const uint64_t d = fma2(V::pair(v, i), sc2, minus_c);
        float d0, d1;
        parts(d, d0, d1);
        const uint64_t w = two(ex2(d0), ex2(d1));
        sums = add2(sums, w);
        sums_z = fma2(w, d, sums_z);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 2) {
        const uint64_t d = two(fmaxf((V::value(v, i) - r) * p.sc, -1e4f),
                               fmaxf((V::value(v, i + 1) - r) * p.sc, -1e4f));
        float d0, d1;
        parts(d, d0, d1);
        const uint64_t w = two(ex2(d0), ex2(d1));
        sums = add2(sums, w);
        sums_z = fma2(w, d, sums_z);
      }
    }
    if (!plain_rank) return;
    const float at = t0 + VEC <= token ? xt : up;
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (DT == SVP_F32) {
#pragma unroll
      for (int e = 0; e < 4; ++e) ahead += !(__uint_as_float(w[e]) < at) ? 1u : 0u;
    } else {
      const uint32_t u = __float_as_uint(at);
      const uint32_t at2 = (u & 0xffff0000u) | (u >> 16);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t r;
        asm("set.geu.bf16x2.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w[e]), "r"(at2));
        asm("add.rn.bf16x2 %0, %0, %1;" : "+r"(n2) : "r"(r));
      }
    }
  };
  auto pour = [&] {  // the halves' counts, before they pass 256
    if constexpr (DT != SVP_F32) {
      ahead += (unsigned)(lo_f(n2) + hi_f(n2));
      n2 = 0u;
    }
  };
  constexpr int U = 4;  // vectors on their way at a time
#pragma unroll 1
  for (int i0 = tid; i0 < n_vec; i0 += 32 * T) {  // at most 128 in a half
#pragma unroll 1
    for (int i = i0; i < min(n_vec, i0 + 32 * T); i += U * T) {
      uint4 v[U];
      uint32_t bits[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        v[u] = i + u * T < n_vec ? aligned[i + u * T] : V::none();
      if (allowed) {
#pragma unroll
        for (int u = 0; u < U; ++u) bits[u] = i + u * T < n_vec ? bits_of(i + u * T) : 0u;
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = V::masked(v[u], bits[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) take(v[u], t00 + (i + u * T) * VEC);
    }
    pour();
  }
  if (has_extra) {
    take(extra, warp == 0 ? -shift : extra0);
    pour();
  }
  LpSums a;
  {
    float c0, c1, x0, x1;
    parts(minus_c, c0, c1);
    a.r = r;
    a.e = fine ? fmaf(r, p.sc, c0) : 0.f;
    parts(sums, x0, x1);
    a.s = x0 + x1;
    parts(sums_z, x0, x1);
    a.sz = x0 + x1;
  }
  const unsigned mine = logit_key(big);  // this thread's largest key
  if (plain_rank && rank == 0 && tid == 0) {
    const int from = (token + shift) / VEC * VEC - shift;
    for (int t = max(from, 0); t < token; ++t)
      if (may(t) && element(t) == xt) ++ahead;
  }
  if (ranked && !plain_rank)  // +inf or NaN: by key
    each([&](unsigned x, int t) {
      ahead += x > kt || (x == kt && t < token) ? 1u : 0u;
    });
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const LpSums o = {__shfl_xor_sync(kFull, a.r, off), __shfl_xor_sync(kFull, a.e, off),
                      __shfl_xor_sync(kFull, a.s, off), __shfl_xor_sync(kFull, a.sz, off)};
    a = join(a, o, p.sc);
  }
  const unsigned wm = __reduce_max_sync(kFull, mine);
  if (lane == 0) {
    sm.warp_f[warp] = a;
    sm.warp_u[0][warp] = wm;
  }
  const unsigned n_ahead = lp_sum(ahead, sm, 1);  // its barrier serves all
  const unsigned top_key =
      __reduce_max_sync(kFull, lane < W ? sm.warp_u[0][lane] : 0u);

  // ---- this CTA's alternatives ----
  unsigned keep = 0;
  if (p.n_top > 0 && top_key > 0u) {
    const unsigned k = (unsigned)p.n_top;
    // A bound that at least k threads reach, and few more: the lower end of the
    // part of the two octaves below the largest that holds the k-th.
    unsigned edge = kLowestKey;
    const unsigned low = top_key - (2u << 23);
    unsigned in_range = 0;
    if (top_key > kLowestKey + (2u << 23)) {
      if (mine > low)
        atomicAdd(&sm.hist[(top_key - mine) >> 16], 1u);  // from the largest down
      __syncthreads();
      constexpr int PER = kLpBins / 32;
      unsigned c[PER], before = 0;
#pragma unroll
      for (int i = 0; i < PER; i += 4) {
        const uint4 y = *reinterpret_cast<const uint4 *>(sm.hist + lane * PER + i);
        c[i] = y.x;
        c[i + 1] = y.y;
        c[i + 2] = y.z;
        c[i + 3] = y.w;
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) before += c[i];
      const unsigned own = before;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const unsigned y = __shfl_up_sync(kFull, before, off);
        if (lane >= off) before += y;
      }
      in_range = __shfl_sync(kFull, before, 31);
      before -= own;
      unsigned at = 0xffffffffu;  // the first bin by whose end there are k
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        before += c[i];
        if (before >= k) at = min(at, (unsigned)(lane * PER + i));
      }
      at = __reduce_min_sync(kFull, at);
      if (in_range >= k) edge = top_key - (at << 16) - 0xffffu;
    }
    if (in_range < k) {
      // bit by bit, from the lowest logit on (with fewer threads that hold any,
      // every element)
      unsigned hi = top_key == 0xffffffffu ? top_key : top_key + 1u;
      while (hi > edge + 1u) {
        const unsigned mid = edge + (hi - edge) / 2u;
        const unsigned c = (unsigned)__syncthreads_count(mine >= mid);
        if (c >= k) {
          edge = mid;
          if (c <= k + kLpSlack) break;
        } else {
          hi = mid;
        }
      }
    }
    auto add = [&](unsigned x, int t) {
      const unsigned at = atomicAdd(&sm.n_found, 1u);
      if (at < kLpFound) {
        sm.found[at].key = x;
        sm.found[at].token = t;
      }
    };
    auto some = [&](const uint4 &v, int t0) {
      if (logit_key(V::top(v)) < edge) return;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const unsigned x = logit_key(V::value(v, e));
        if (x >= edge) add(x, t0 + e);
      }
    };
    // the vectors of the threads that reach it, as many at once as a warp takes
    if (mine >= edge) sm.high[atomicAdd(&sm.n_high, 1u)] = (unsigned short)tid;
    __syncthreads();
    const int n_high = (int)sm.n_high;
    int lanes = 1;  // for a thread's vectors
    while (lanes < 32 && lanes * T < n_vec) lanes *= 2;
    const int per = 32 / lanes;
    for (int x = warp * per + lane / lanes; x < n_high; x += W * per)
      for (int i = sm.high[x] + lane % lanes * T; i < n_vec; i += lanes * T)
        some(fetch(i), t00 + i * VEC);
    if (has_extra && mine >= edge) some(extra, extra0);
    __syncthreads();
    unsigned n = sm.n_found;
    if (n > kLpFound) {
      // the k-th largest of all, then the token up to which its equals count
      edge = 0;
      for (int bit = 31; bit >= 0; --bit) {
        const unsigned at = edge | (1u << bit);
        unsigned c = 0;
        each([&](unsigned x, int) { c += x >= at ? 1u : 0u; });
        if (lp_sum(c, sm, bit) >= k) edge = at;
      }
      int last = 0;
      for (int bit = 30; bit >= 0; --bit) {
        // do fewer than k come before token `at`?
        const int at = last | (1 << bit);
        unsigned c = 0;
        each([&](unsigned x, int t) {
          c += x > edge || (x == edge && t < at) ? 1u : 0u;
        });
        if (lp_sum(c, sm, bit + 1) < k) last = at;  // (+ 1: in turn with the above)
      }
      if (tid == 0) sm.n_found = 0;
      __syncthreads();
      each([&](unsigned x, int t) {
        if (x > edge || (x == edge && t <= last)) add(x, t);
      });
      __syncthreads();
      n = k;
    }
    keep = min(n, k);
    if (tid == 0) sm.found[n].key = 0u;  // (n <= kLpFound)
    __syncthreads();
    if (nc > 1) lp_wait();
    Found *const best =
        (nc > 1 ? cluster.map_shared_rank(sm.best, 0) : sm.best) + rank * p.n_top;
    for (unsigned r = keep + tid; r < k; r += T) best[r] = Found{0u, 0};
    for (unsigned c = tid; c < n; c += T) {
      const Found f = sm.found[c];
      unsigned r = 0;
#pragma unroll 4
      for (unsigned o = 0; o < n; o += 2) {  // (one more is there: nothing)
        const uint4 h = *reinterpret_cast<const uint4 *>(sm.found + o);
        r += h.x > f.key || (h.x == f.key && (int)h.y < f.token) ? 1u : 0u;
        r += h.z > f.key || (h.z == f.key && (int)h.w < f.token) ? 1u : 0u;
      }
      if (r < keep) best[r] = f;
    }
  } else {
    if (nc > 1) lp_wait();
    Found *const best =
        (nc > 1 ? cluster.map_shared_rank(sm.best, 0) : sm.best) + rank * p.n_top;
    for (int r = tid; r < p.n_top; r += T) best[r] = Found{0u, 0};
  }
  // (the counting takes them in pairs)
  if (rank == 0 && tid == 0) sm.best[nc * p.n_top] = Found{0u, 0};
  if (tid == 0) {
    LpPart part;
    part.key = top_key;
    part.sums = sm.warp_f[0];
    for (int w = 1; w < W; ++w) part.sums = join(part.sums, sm.warp_f[w], p.sc);
    if (top_key > logit_key(3.402823466e38f)) part.sums.s = NAN;  // +inf or NaN
    part.ahead = n_ahead;
    part.n_best = keep;
    LpPart *const to =
        nc > 1 ? cluster.map_shared_rank(&sm.part[rank], 0) : &sm.part[0];
    *to = part;
  }
  // the others' results are in the first CTA, which alone goes on
  if (nc > 1) {
    lp_arrive();
    if (rank != 0) return;
    lp_wait();
  } else {
    __syncthreads();
  }

  // ---- the row's results ----
  unsigned row_key = 0, n_before = 0;
  LpSums all = sm.part[0].sums;
  for (int r = 0; r < nc; ++r) {
    row_key = max(row_key, sm.part[r].key);
    n_before += sm.part[r].ahead;
    if (r > 0) all = join(all, sm.part[r].sums, p.sc);
  }
  const float ln = logf(all.s);
  auto log_p = [&](float x) {
    return fmaf(x - all.r, p.inv_t, all.e * kLn2) - ln;
  };
  if (tid == 0) {
    // a row that allows nothing has no probabilities: -inf, entropy 0
    p.logprobs[row] = all.s != all.s ? NAN : kt == 0u ? -INFINITY : log_p(xt);
    if (p.entropy)
      p.entropy[row] = row_key == 0u ? 0.f : ln - all.sz / all.s * kLn2;
    if (p.ranks) p.ranks[row] = kt == 0u ? -1 : (int)n_before;
  }
  if (p.n_top > 0) {
    const int n_all = nc * p.n_top;
    unsigned n = 0;
    for (int r = 0; r < nc; ++r) n += sm.part[r].n_best;
    for (int x = tid; x < n_all; x += T) {
      const Found f = sm.best[x];
      if (f.key == 0u) continue;
      unsigned r = 0;  // how many are before it
#pragma unroll 4
      for (int o = 0; o < n_all; o += 2) {
        const uint4 h = *reinterpret_cast<const uint4 *>(sm.best + o);
        r += h.x > f.key || (h.x == f.key && (int)h.y < f.token) ? 1u : 0u;
        r += h.z > f.key || (h.z == f.key && (int)h.w < f.token) ? 1u : 0u;
      }
      if (r < (unsigned)p.n_top) {
        p.top_logprobs[row * p.n_top + r] = log_p(key_logit(f.key));
        p.top_tokens[row * p.n_top + r] = f.token;
      }
    }
    for (unsigned i = n + tid; i < (unsigned)p.n_top; i += T) {
      p.top_logprobs[row * p.n_top + i] = -INFINITY;
      p.top_tokens[row * p.n_top + i] = -1;
    }
  }
}

template <int DT, int T>
cudaError_t logprobs_t(const LogprobParams &p, int sms, cudaStream_t stream) {
  const int vecs = p.vocab / Vec<DT>::N;
  // more CTAs to a row while there are few of them and a thread has a vector:
  // 80 rows of 32,000 fp32 take 11.0 us with four, 14.1 with eight; 512 of 131,072
  // bf16 44 with one, 47 with two, 61 with four
  int nc = 1;
  while (nc < kLpCluster && (long long)p.rows * nc < 2LL * sms && vecs > T * nc) nc *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = nc;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.rows * (unsigned)nc);
  cfg.blockDim = dim3(T);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<DT, T>, p);
}

template <int DT>
cudaError_t logprobs_dt(const LogprobParams &p, int sms, cudaStream_t stream) {
  // Short rows: what a CTA does once counts, so fewer threads, of which an SM
  // holds more CTAs (2048 rows of 1000 fp32 13.7 us where 256 threads take 22.4;
  // 1561 of 4785 bf16 18.0, 23.6; but 600 of 32,000 fp32 25.3, 19.6).
  return p.vocab / Vec<DT>::N <= 1024 ? logprobs_t<DT, 128>(p, sms, stream)
                                      : logprobs_t<DT, 256>(p, sms, stream);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobParams &p, int dtype, int sms,
                                  cudaStream_t stream) {
  return dtype == SVP_F32 ? logprobs_dt<SVP_F32>(p, sms, stream)
                          : logprobs_dt<SVP_BF16>(p, sms, stream);
}

cudaError_t status_word_logprobs(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_logprobs);
}

}  // namespace svp
