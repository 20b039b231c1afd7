// attention_fp4.cu -- paged decode / speculative-verify attention over a
// 4-bit cache (E2M1 codes, one E4M3 scale per 16 elements; fp4.cuh).
//
// What it computes: as attention.cu, with K = code * scale * k_scale and
// V = code * scale * v_scale.  k_scale is folded into the score scale,
// v_scale multiplies the outputs, code * scale is exact in fp16.
//
// What bounds it: latency.  A cached element is 9/16 byte, so at the copy
// rate an SM has to turn 80 elements a nanosecond into products: a page of K
// and V (2304 bytes, D = 128) may take 99 cycles.  Its conversion, products
// and softmax are about 250 warp instructions for up to 8 rows, 63 issue
// cycles of the SM's four schedulers, but take 111 with the three warps a
// scheduler that registers leave (without the copies; issue active 50%, and
// 1.6 of the stalls an instruction are fixed latencies).  Hence as few
// instructions an element as there are: even a single query row goes through
// mma.sync (keys as M, query rows as N = 8), so the conversion (one cvt and
// one fp16 multiply per two elements) is done once per element for all rows,
// and the codes go from shared memory to the matrix instruction through
// registers only.
//
//  * S^T = K Q^T, one 16-key page per m16 tile: lane (g, t) takes
//    consecutive codes (whole scale blocks) of two keys.  Q is fp16 with a
//    power-of-two scale per row (fp4.cuh).
//  * Softmax on the accumulators in the log2 domain.  The running maximum is
//    lazy: a row's reference moves only when a score exceeds it by 2^8, so
//    the usual page costs one vote instead of shuffled maxima.  P is fp16 at
//    2^6 times its softmax weight relative to the reference (at most 2^14),
//    which keeps weights down to 2^-20 normal: rounding P costs each weight
//    half an fp16 step, 2^-11, as bf16 P costs 2^-8; the row sums are fp32
//    and of the weights before that rounding.
//  * O^T = V^T P^T: P's fp16 pairs become the B operand by movmatrix.  Lane
//    (g, t) reads D/8 consecutive codes of four keys; the nibbles of two
//    keys are interleaved before the conversion, so one cvt yields the pair
//    of keys that the A operand wants for one dimension.
//  * Every warp is on its own: it takes one slice of the flattened page list
//    (the stream-K order of attn_common.cuh, with a warp where that has a
//    CTA), copies its pages itself (1-D bulk copies -- a head's page is one
//    run of 9 D bytes -- four pages to a stage, two or three stages), keeps a
//    segment's whole state in registers and writes the segment's result from
//    there.  No barrier joins the warps, so a warp that ends a segment
//    (normalise, write, next Q) costs the others nothing.
//  * Short sequences (kWholePages) are taken whole, a group by one warp or by
//    a team of neighbours whose results meet in shared memory: no prefix of
//    the lengths to build, no partials in memory and no second launch (250
//    tokens of four heads: 7.4 us a call).
//  * A group of pages cut by slice borders leaves one normalised partial per
//    slice; merge_fp4_kernel joins them by log-sum-exp in slice order.
//  * Rows whose memory holds no valid data take no part: masked keys score
//    -inf whatever their bytes, and their V scale is replaced by 0.
//
// Measured (call times, D = 128; of the cache's bytes at the copy rate): 32
// sequences of 32 heads, up to 4096 tokens, one row each: 78.5 us, 0.64 (a
// bf16 cache: 242 us); four sequences of 131,072 tokens, 8 rows: 123 us, 0.73
// (326); 16 sequences of 8 heads, up to 8192 tokens, 20 rows: 60 us, 0.24
// (68) -- there an SM's eight warps issue 0.34 instructions a cycle and
// scheduler, waiting on the fixed latencies of conversion, MMA and
// exponential chains (1.9 stalls an instruction) and on code (0.7).
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_attn4;

namespace {

constexpr int kStagePages = kTilePagesFp4;    // 4
constexpr int kNoPage = 0x7fffff00;           // j0 of a page that is not there
constexpr float kRefOffset = 6.f;             // P = 2^6 at the reference
constexpr float kRefSlack = 14.f;             // largest log2 P before a move
constexpr float kNoRef = -3e38f;              // below any finite score

// Warps of a CTA (one per SM) for NT n8 tiles of query rows: what the
// registers allow (O alone takes 32 per tile), 168 per thread for twelve
// warps, 255 for eight (twelve warps for two tiles spill: 56 us against 46
// for 16 rows on 98 MB of cache).
template <int NT>
__host__ __device__ constexpr int warps4() {
  return NT == 1 ? 12 : 8;
}
// Stages of a warp's ring: 9 D bytes x 8 each, as many as fit.
template <int NT>
__host__ __device__ constexpr int stages4() {
  return NT == 2 ? 3 : 2;
}
// Three tiles leave no registers for the Q fragments: they wait in shared
// memory, read back by the lane that wrote them, and the pages go one by one
// (in pairs, with spills: 63 us against 59 for 20 rows on 98 MB).
template <int NT>
__host__ __device__ constexpr bool q_in_smem() {
  return NT == 3;
}
constexpr int kChecked = 256;
constexpr int kSegRing4 = 8;  // decoded segments: read .. issued + 1

// A run of pages of one group within a slice.
struct Seg4 {
  int b, g, rg, L;
  int page0, n_pages, n_a, b_start;
  int f, l;    // slices that hold the group's first and last page
  int next;    // flat item after the run
  int valid;
  // pages that end by t_min (the unit's first position; with a tree: before
  // its nodes) and, under a window, lie in that of t_max (its last position)
  // need no per-key test
  int t_min, t_max;
};

template <int D, int STAGES>
struct Warp4 {
  static constexpr int PAGE = 9 * D;  // bytes of one head's 16 rows
  alignas(128) unsigned char kv[STAGES][kStagePages][2][PAGE];
};
// what the issuing side leaves for the reading side
template <int STAGES>
struct Info4 {
  uint64_t full[STAGES];
  int j0[STAGES][kStagePages];
  int meta[STAGES];  // pages; + kChecked: their keys need the visibility test
  Seg4 seg[kSegRing4];
};
template <int D, int NT, int W, int STAGES>
struct Smem4 {
  Warp4<D, STAGES> warp[W];
  uint2 q[q_in_smem<NT>() ? W * NT * (D / 16) * 32 : 1];
  Info4<STAGES> info[W];
  int prefix[1];  // [batch + 1] item prefix, then [batch] lengths: dynamic
};

__device__ __forceinline__ void raise4(unsigned f) {
  atomicOr(&g_status_attn4, f);
}

// Shared-memory reads by 32-bit address: volatile keeps them behind the
// barrier waits (and nothing else in order), and the address arithmetic
// stays 32-bit.
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ void sts32(uint32_t a, int v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void bulk_to(uint32_t dst, const void *src,
                                        uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ bool mbar_try_at(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// Waits (bounded) for the phase; the same answer in every lane.
__device__ __forceinline__ bool mbar_wait_at(uint32_t bar, uint32_t parity) {
  if (__all_sync(kFull, mbar_try_at(bar, parity))) return true;
  const uint64_t start = globaltimer();
  bool ok = false;
  while (!(ok = mbar_try_at(bar, parity)) && globaltimer() - start <= SVP_WAIT_NS) {
  }
  return __all_sync(kFull, ok);
}

// Dims of k-step ks, lane t: four from q_dim on.  A lane's steps cover D/4
// consecutive dims: one or two scale blocks.
template <int D>
__device__ __forceinline__ constexpr int q_dim(int ks, int t) {
  return (D / 4) * t + 4 * ks;
}

// One page's scores: S += K Q^T for 16 keys.  kp: the page's address plus
// this lane's offset k_lane<D>(); qb(ks, nt) gives the Q fragment of a
// k-step.  With one tile the even and the odd k-steps form two chains.
template <int D>
__device__ __forceinline__ uint32_t k_lane(int g, int t) {
  return fp4_key(g, 0) * fp4_row_bytes(D) + (D / 8) * t;
}
template <int D, int NT, typename QB>
__device__ __forceinline__ void page_scores(uint32_t kp, int t,
                                            float (&s)[NT][4], QB qb) {
  constexpr int ROW = fp4_row_bytes(D), C = D / 64;  // scale blocks per lane
  uint2 w[2][C];
  uint32_t sc[2][C];  // fp16 pairs of the block scales
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t row = kp + 2 * h * ROW;  // keys fp4_key(g, h)
#pragma unroll
    for (int c = 0; c < C; ++c)
      w[h][c] = D == 128 ? lds64(row + 8 * c)
                         : make_uint2(lds32(row), lds32(row + 4));
    // the scales lie D/2 bytes from the row's start, C bytes per lane
    const uint32_t at = row + D / 2 - (D / 8 - C) * t;
    if constexpr (C == 2) {
      const uint32_t both = e4m3x2_f16x2(lds_u16(at));
      sc[h][0] = __byte_perm(both, 0, 0x1010);
      sc[h][C - 1] = __byte_perm(both, 0, 0x3232);
    } else {
      sc[h][0] = e4m3x2_f16x2(lds_u8(at) * 0x101u);
    }
  }
  float odd[4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int hw = 0; hw < 2; ++hw) {
      uint32_t k0[4], k1[4];
      e2m1x8_h2(hw ? w[0][c].y : w[0][c].x, k0);
      e2m1x8_h2(hw ? w[1][c].y : w[1][c].x, k1);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t a[4] = {hmul2(k0[2 * i], sc[0][c]),
                               hmul2(k1[2 * i], sc[1][c]),
                               hmul2(k0[2 * i + 1], sc[0][c]),
                               hmul2(k1[2 * i + 1], sc[1][c])};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 b = qb(4 * c + 2 * hw + i, nt);
          float (&to)[4] = NT == 1 && i ? odd : s[nt];
          if (c == 0 && hw == 0 && (NT == 1 || i == 0))
            mma_f16_first(to, a, b.x, b.y);
          else
            mma_f16(to, a, b.x, b.y);
        }
      }
    }
  if constexpr (NT == 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[0][e] += odd[e];
  }
}

// One page's O^T += V^T P^T.  vp: the page's address plus this lane's offset
// v_lane<D>(); sp: the same for its scale byte.  keep: bit s set iff key
// 4t + s holds valid data (its scale counts as 0 otherwise).
template <int D>
__device__ __forceinline__ uint32_t v_lane(int g, int t) {
  return 4 * t * fp4_row_bytes(D) + (D / 16) * g;
}
template <int D>
__device__ __forceinline__ uint32_t v_lane_scale(int g, int t) {
  return 4 * t * fp4_row_bytes(D) + D / 2 + (D / 8) * g / kFp4Group;
}
template <int D, int NT>
__device__ __forceinline__ void page_values(uint32_t vp, uint32_t sp,
                                            unsigned keep,
                                            const uint32_t (&pb)[NT][2],
                                            float (&o)[D / 16][NT][4]) {
  constexpr int ROW = fp4_row_bytes(D), C = D / 64;
  uint32_t w[4][C], sc[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if constexpr (D == 128) {
      const uint2 x = lds64(vp + s * ROW);
      w[s][0] = x.x;
      w[s][C - 1] = x.y;
    } else {
      w[s][0] = lds32(vp + s * ROW);
    }
    sc[s] = lds_u8(sp + s * ROW);
  }
  if (keep != 0xfu) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
      if (!((keep >> s) & 1u)) sc[s] = 0u;
  }
  const uint32_t s01 = e4m3x2_f16x2(__byte_perm(sc[0], sc[1], 0x0040));
  const uint32_t s23 = e4m3x2_f16x2(__byte_perm(sc[2], sc[3], 0x0040));
#pragma unroll
  for (int wi = 0; wi < C; ++wi) {
    // nibbles of two keys side by side: even dims, odd dims
    constexpr uint32_t M = 0x0f0f0f0fu;
    uint32_t e01[4], d01[4], e23[4], d23[4];
    e2m1x8_h2((w[0][wi] & M) | ((w[1][wi] << 4) & ~M), e01);
    e2m1x8_h2(((w[0][wi] >> 4) & M) | (w[1][wi] & ~M), d01);
    e2m1x8_h2((w[2][wi] & M) | ((w[3][wi] << 4) & ~M), e23);
    e2m1x8_h2(((w[2][wi] >> 4) & M) | (w[3][wi] & ~M), d23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a[4] = {hmul2(e01[i], s01), hmul2(d01[i], s01),
                             hmul2(e23[i], s23), hmul2(d23[i], s23)};
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        mma_f16(o[4 * wi + i][nt], a, pb[nt][0], pb[nt][1]);
    }
  }
}

// The first run of pages at or after flat item `pos` (as decode_segment of
// attn_common.cuh, for slices instead of CTAs).
__device__ __forceinline__ Seg4 next_segment(const AttnParams &p,
                                             const int *prefix,
                                             const int *seqlen, int per_seq,
                                             int pos, int end, int total,
                                             int n_slices, int rb) {
  Seg4 s;
  s.valid = 0;
  if (pos >= end) return s;
  int lo = 0, hi = p.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= pos) lo = mid; else hi = mid;
  }
  const int per = (prefix[lo + 1] - prefix[lo]) / per_seq;
  const int nt = per - p.seg_items;
  const int gi = (pos - prefix[lo]) / per;
  const int off = pos - prefix[lo] - gi * per;
  const int first = prefix[lo] + gi * per + p.seg_items;
  const int t0 = off < p.seg_items ? 0 : off - p.seg_items;
  int np;
  s.b = lo;
  s.L = seqlen[lo];
  visible_pages(s.L, p.q_len, p.n_sink, p.window, s.n_a, s.b_start, np);
  s.page0 = t0 * p.ppi;
  s.g = gi / p.n_rg;
  s.rg = gi - s.g * p.n_rg;
  const int items = min(end - (first + t0), nt - t0);
  s.n_pages = min(items * p.ppi, np - s.page0);
  s.next = first + t0 + items;
  s.f = div_u64((unsigned long long)(first + 1) * (unsigned)n_slices - 1u,
                (unsigned)total);
  s.l = div_u64((unsigned long long)(first + nt) * (unsigned)n_slices - 1u,
                (unsigned)total);
  s.valid = s.n_pages > 0;
  const int base = s.L - p.q_len;
  s.t_min = p.tree_mask ? base - 1 : base + s.rg * rb / p.group;
  s.t_max = base + (min(s.rg * rb + rb, p.rows) - 1) / p.group;
  return s;
}

// Part `part` of group `slice` (AttnParams::whole, ::parts), in pairs of pages.
__device__ __forceinline__ Seg4 whole_segment(const AttnParams &p, int per_seq,
                                              int slice, int part, int rb,
                                              int lane) {
  Seg4 s = {};
  s.b = slice / per_seq;
  const int gi = slice - s.b * per_seq;
  s.g = gi / p.n_rg;
  s.rg = gi - s.g * p.n_rg;
  s.L = p.seq_lens[s.b];
  if (s.L < p.q_len || s.L > (long long)p.max_blocks * kBlockSize) {
    if (lane == 0 && gi == 0) raise4(SVP_DEV_BAD_SEQ_LEN);
    return s;
  }
  int np;
  visible_pages(s.L, p.q_len, p.n_sink, p.window, s.n_a, s.b_start, np);
  const int pairs = (np + 1) / 2;
  s.page0 = 2 * (pairs * part / p.parts);
  s.n_pages = min(2 * (pairs * (part + 1) / p.parts), np) - s.page0;
  s.f = s.l = slice;
  s.valid = s.n_pages > 0;
  const int base = s.L - p.q_len;
  s.t_min = p.tree_mask ? base - 1 : base + s.rg * rb / p.group;
  s.t_max = base + (min(s.rg * rb + rb, p.rows) - 1) / p.group;
  return s;
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * warps4<NT>(), 1)
    paged_attention_fp4_kernel(const AttnParams p) {
  constexpr int W = warps4<NT>(), RB = 8 * NT, KS = D / 16;
  constexpr int PJ = NT == 3 ? 1 : 2;  // pages scored together
  static_assert(warps4<2>() == warps4<3>(), "a launch's rest may plan for either");
  constexpr int kStages4 = stages4<NT>();
  static_assert(kStages4 + 2 <= kSegRing4, "a stage holds at most one segment");
  constexpr int PAGE = 9 * D;
  extern __shared__ unsigned char smem_raw[];
  using S = Smem4<D, NT, W, kStages4>;
  S &sm = *reinterpret_cast<S *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int per_seq = p.num_kv_heads * p.n_rg;
  Info4<kStages4> &inf = sm.info[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages4; ++s) mbar_init(&inf.full[s], 1);
    fence_mbar_init();
  }
  __syncwarp();
  // launched early: see AttnParams::early
  if (!p.early) pdl_wait();
  pdl_launch_dependents();  // the merge may be scheduled
  // slice s goes to warp s / gridDim.x of CTA s % gridDim.x: a small call
  // spreads over the SMs (parts of a group: to neighbouring warps)
  const int part = p.whole ? warp % p.parts : 0;
  const int team = p.whole ? warp / p.parts : warp;
  const int slice = team * gridDim.x + blockIdx.x;
  int *const seqlen = sm.prefix + p.batch + 1;
  int total = 0, n_slices = p.batch * per_seq, end = 0;
  if (p.whole) {
    if ((team + 1) * p.parts > W) return;  // warps of no whole team
  } else {
    if (warp == 0)
      build_prefix(p, sm.prefix, seqlen, per_seq, lane, &g_status_attn4);
    __syncthreads();  // the only one: the warps are on their own from here
    total = sm.prefix[p.batch];
    n_slices = (int)min((long long)gridDim.x * W,
                        max(1LL, (long long)total / p.min_pages));
  }
  if (slice >= n_slices) return;
  if (!p.whole) end = slice_begin(slice + 1, total, n_slices);

  // ---- the issuing side: up to kStages4 stages ahead of the reading side.
  // Segment `seg_i` is being issued, the one after it is decoded already and
  // its first block-table entries are on their way. ----
  bool waited = !p.early;  // the grid-dependency wait is behind us
  int issued = 0, seg_i = 0, k = 0;
  // of the segment being issued: its pages, the flat page number from which
  // sinks are skipped and by how much, its first page, head, limits
  int n_pages = 0, page0 = 0, n_a = 0, skip = 0, kvh = 0, t_min = 0, t_max = 0;
  auto decode = [&](int i, int pos) {  // segment i of this slice, into the ring
    const Seg4 s = !p.whole ? next_segment(p, sm.prefix, seqlen, per_seq, pos, end,
                                           total, n_slices, RB)
                   : i == 0 ? whole_segment(p, per_seq, slice, part, RB, lane)
                            : Seg4{};
    if (lane == 0) inf.seg[i % kSegRing4] = s;
    __syncwarp();
  };
  auto entry = [&](int i, int page) {  // block-table entry of a page of segment i
    const Seg4 &s = inf.seg[i % kSegRing4];
    if (!s.valid || page >= s.n_pages) return -1;
    const int pidx = s.page0 + page;
    const int lb = pidx < s.n_a ? pidx : s.b_start + (pidx - s.n_a);
    return __ldg(p.block_table + (size_t)s.b * p.max_blocks + lb);
  };
  auto take_up = [&]() {  // the state of segment seg_i
    const Seg4 &s = inf.seg[seg_i % kSegRing4];
    n_pages = s.valid ? s.n_pages : 0;
    page0 = s.page0;
    n_a = s.n_a;
    skip = s.b_start - n_a;
    kvh = s.g;
    t_min = s.t_min;
    t_max = s.t_max;
    k = 0;
  };
  // a block-table entry as the number of its head's page, -1 for a bad one
  auto head_page = [&](int ph, int page) {
    if (page >= n_pages) return -1;
    if (ph >= 0 && ph < p.num_blocks) return ph * p.num_kv_heads + kvh;
    raise4(SVP_DEV_BAD_BLOCK_ID);
    return -1;
  };
  decode(0, p.whole ? 0 : slice_begin(slice, total, n_slices));
  take_up();
  // entries of pages k .. k + 31 (as head pages), of the 32 after them, and
  // of the following segment's first 32
  int phys = entry(0, lane), phys2 = entry(0, 32 + lane);
  decode(1, n_pages ? inf.seg[0].next : end);
  int phys_a = entry(1, lane);
  phys = head_page(phys, lane);
  const uint32_t bars = smem_u32(&inf.full[0]), metas = smem_u32(&inf.meta[0]);
  const uint32_t j0s = smem_u32(&inf.j0[0][0]);
  const uint32_t kv0 = smem_u32(&sm.warp[warp].kv[0][0][0][0]);
  // lane 2 x + side issues page x's copy of that side
  const unsigned char *const cache =
      static_cast<const unsigned char *>(lane & 1 ? p.v_cache : p.k_cache);
  auto issue = [&]() {
    if (k >= n_pages) return;  // nothing left (uniform)
    const int st = issued % kStages4;
    const int n = min(kStagePages, n_pages - k);
    const int last = page0 + k + ((n + 1) & ~1) - 1;  // of the last pair
    if (!waited) {
      const int pl = page0 + k + n - 1;
      if (((pl < n_a ? pl : pl + skip) + 1) * kBlockSize >
          inf.seg[seg_i % kSegRing4].L - p.q_len) {
        pdl_wait();  // a page may hold some of the appended positions
        waited = true;
      }
    }
    const int x = lane >> 1;
    const int hp = __shfl_sync(kFull, phys, (k + x) & 31);
    const bool good = lane < 2 * n && hp >= 0;
    const unsigned copies = __ballot_sync(kFull, good);
    const int pidx = page0 + k + x;
    int j0 = (pidx < n_a ? pidx : pidx + skip) * kBlockSize;
    if (!good) j0 = kNoPage;
    bool test = __popc(copies) != 2 * n;
    if (p.window == 0) {
      test = test || last * kBlockSize + kBlockSize - 1 > t_min;
    } else {
      const int j1 = j0 + kBlockSize - 1;
      const bool clear =
          j1 <= t_min && (j1 < p.n_sink || j0 > t_max - p.window);
      test = __any_sync(kFull, !clear && x < ((n + 1) & ~1));
    }
    if ((lane & 1) == 0 && lane < 2 * kStagePages)
      sts32(j0s + (st * kStagePages + x) * 4, j0);
    if (lane == 0) {
      sts32(metas + st * 4, n + (test ? kChecked : 0));
#ifdef SVP_TEST_STALL_AFTER
      // test builds only: later stages never arrive, so the waits run out
      if (issued < SVP_TEST_STALL_AFTER)
#endif
        mbar_expect(bars + st * 8, __popc(copies) * PAGE);
    }
    __syncwarp();
#ifdef SVP_TEST_STALL_AFTER
    if (issued < SVP_TEST_STALL_AFTER)
#endif
    if (good)
      bulk_to(kv0 + (st * kStagePages * 2 + lane) * PAGE,
              cache + (size_t)(unsigned)hp * PAGE, PAGE, bars + st * 8);
    ++issued;
    k += n;
    if (k >= n_pages) {
      ++seg_i;
      take_up();
      phys = head_page(phys_a, lane);
      phys2 = entry(seg_i, 32 + lane);
      decode(seg_i + 1, n_pages ? inf.seg[seg_i % kSegRing4].next : end);
      phys_a = entry(seg_i + 1, lane);
    } else if ((k & 31) == 0) {
      phys = head_page(phys2, k + lane);
      phys2 = entry(seg_i, k + 32 + lane);
    }
  };
  for (int s = 0; s < kStages4; ++s) issue();

  // ---- the reading side ----
  const uint32_t k_off = k_lane<D>(g, t), v_off = v_lane<D>(g, t);
  const uint32_t v_off_s = v_lane_scale<D>(g, t);
  int c = 0;  // stages read
  bool gave_up = false;
  // a part's result, where its pages were: rows, their LSEs, whether it gave up
  float *const part_s = reinterpret_cast<float *>(&sm.warp[warp].kv[0][0][0][0]);
  static_assert((RB * D + RB + 1) * 4 <= sizeof(Warp4<D, kStages4>), "a part's result");
  for (int us = 0;; ++us) {
    __syncwarp();
    const Seg4 ui = inf.seg[us % kSegRing4];
    if (!ui.valid) break;
    const int L = ui.L, t0 = L - p.q_len;
    const int row0 = ui.rg * RB;

    // ---- Q fragments: row n = g of each n8 tile, fp16, scaled by row ----
    uint2 qf[NT][KS];
    float qs[NT][2];  // score scale of rows 2t, 2t + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int gr = row0 + nt * 8 + g;
      const bool valid = gr < p.rows;
      const int grc = valid ? gr : row0;
      const int i = grc / p.group;
      const int h = ui.g * p.group + grc % p.group;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          static_cast<const uint16_t *>(p.q) +
          (((size_t)ui.b * p.q_len + i) * p.num_q_heads + h) * D);
      uint32_t top = 0;
#pragma unroll
      for (int x = 0; x < KS / 2; ++x) {  // q_dim: D/4 consecutive dims
        uint4 v = __ldg(src + (KS / 2) * t + x);
        if (!valid) v = make_uint4(0, 0, 0, 0);
        qf[nt][2 * x] = make_uint2(v.x, v.y);
        qf[nt][2 * x + 1] = make_uint2(v.z, v.w);
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 v = qf[nt][ks];
        top = max(top, max(max(v.x & 0x7fffu, (v.x >> 16) & 0x7fffu),
                           max(v.y & 0x7fffu, (v.y >> 16) & 0x7fffu)));
      }
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      const int e = q_exponent(__uint_as_float(top << 16));
      const float f = pow2i(14 - e);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 v = qf[nt][ks];
        qf[nt][ks] = make_uint2(pack_h2(__uint_as_float(v.x << 16) * f,
                                        __uint_as_float(v.x & 0xffff0000u) * f),
                                pack_h2(__uint_as_float(v.y << 16) * f,
                                        __uint_as_float(v.y & 0xffff0000u) * f));
      }
      const float sc = p.qscale * pow2i(e - 14);
      qs[nt][0] = __shfl_sync(kFull, sc, 8 * t);
      qs[nt][1] = __shfl_sync(kFull, sc, 8 * t + 4);
    }
    const uint32_t qa = smem_u32(&sm.q[0]) + (warp * NT * KS * 32 + lane) * 8;
    if constexpr (q_in_smem<NT>()) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          sm.q[((warp * NT + nt) * KS + ks) * 32 + lane] = qf[nt][ks];
      __syncwarp();
    }
    auto qb = [&](int ks, int nt) {
      return q_in_smem<NT>() ? lds64(qa + (nt * KS + ks) * 256) : qf[nt][ks];
    };

    float o[D / 16][NT][4];
    float ref[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      ref[nt][0] = ref[nt][1] = kNoRef;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
        o[i][nt][0] = o[i][nt][1] = o[i][nt][2] = o[i][nt][3] = 0.f;
    }

    // The pages of a segment go two by two.  A pair's scores are computed in
    // the same straight run of code as the previous pair's P V: the two share
    // no data, so the one's chains of conversions and MMAs fill the other's
    // waits (long contexts: 122 us against 126).
    auto ready = [&](int cc) {
      if (mbar_wait_at(bars + (cc % kStages4) * 8, (cc / kStages4) & 1)) return true;
      // give up: flag it, wait (bounded) for the copies still in flight
      if (lane == 0) {
        raise4(SVP_DEV_TIMEOUT);
        int armed = issued;
#ifdef SVP_TEST_STALL_AFTER
        armed = min(armed, SVP_TEST_STALL_AFTER);
#endif
        for (int q = c; q < armed; ++q)
          (void)mbar_wait_drain(&inf.full[q % kStages4], (q / kStages4) & 1);
      }
      return false;
    };
    if (!ready(c)) {
      gave_up = true;
      break;
    }
    int s = c % kStages4, p0 = 0, left = ui.n_pages;
    int meta = (int)lds32(metas + s * 4);  // warp-uniform
    uint32_t pair = kv0 + s * (kStagePages * 2 * PAGE);
    float x[PJ][NT][4];
#pragma unroll
    for (int j = 0; j < PJ; ++j)
      page_scores<D, NT>(pair + j * 2 * PAGE + k_off, t, x[j], qb);
    while (true) {
      const bool checked = meta >= kChecked;
      const int pages = meta & (kChecked - 1);
      // ---- softmax with a lazy reference ----
      float y[PJ][NT][4];
      float far = -INFINITY;
#pragma unroll
      for (int j = 0; j < PJ; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[j][nt][e] = fmaf(x[j][nt][e], qs[nt][e & 1], -ref[nt][e & 1]);
            far = fmaxf(far, y[j][nt][e]);
          }
      unsigned keep[PJ];
#pragma unroll
      for (int j = 0; j < PJ; ++j) keep[j] = 0xfu;
      if (checked || __any_sync(kFull, far > kRefSlack)) {
        // masked keys score -inf; a row whose scores reach beyond the
        // slack gets a new reference
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            uint32_t bits = ~0u;
            int i = 0;
            if (checked) {
              i = min(row0 + nt * 8 + 2 * t + r, p.rows - 1) / p.group;
              bits = row_tree_bits(p, ui.b, i);
            }
            float mx = -INFINITY;
#pragma unroll
            for (int j = 0; j < PJ; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float z = x[j][nt][2 * h + r] * qs[nt][r];
                if (checked &&
                    !key_visible((int)lds32(j0s + (s * kStagePages + p0 + j) * 4) + fp4_key(g, h), t0 + i,
                                 bits, t0, p.n_sink, p.window))
                  z = -INFINITY;
                x[j][nt][2 * h + r] = z;
                mx = fmaxf(mx, z);
              }
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kFull, mx, 16));
            const float to = fmaxf(ref[nt][r], mx - kRefOffset);
            const float alpha = ex2(ref[nt][r] - to);
            ref[nt][r] = to;
            l[nt][r] *= alpha;
#pragma unroll
            for (int d2 = 0; d2 < D / 16; ++d2) {
              o[d2][nt][r] *= alpha;
              o[d2][nt][2 + r] *= alpha;
            }
#pragma unroll
            for (int j = 0; j < PJ; ++j)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                y[j][nt][2 * h + r] = x[j][nt][2 * h + r] - to;
          }
        if (checked) {
#pragma unroll
          for (int j = 0; j < PJ; ++j)
#pragma unroll
            for (int sx = 0; sx < 4; ++sx) {
              const int key = (int)lds32(j0s + (s * kStagePages + p0 + j) * 4) + 4 * t + sx;
              if (!(key < L && (p.window == 0 || key < p.n_sink ||
                                key > t0 - p.window)))
                keep[j] &= ~(1u << sx);
            }
        }
      }
#pragma unroll
      for (int j = 0; j < PJ; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[j][nt][e] = ex2(y[j][nt][e]);
            l[nt][e & 1] += y[j][nt][e];
          }
        }
      uint32_t pb[PJ][NT][2];
#pragma unroll
      for (int j = 0; j < PJ; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[j][nt][0] = transpose8(pack_h2(y[j][nt][0], y[j][nt][1]));
          pb[j][nt][1] = transpose8(pack_h2(y[j][nt][2], y[j][nt][3]));
        }
      // the next pair: of this stage, of the next one, or none (this one's
      // scores are then computed again and dropped)
      const bool stage_end = p0 + PJ >= pages;
      const bool more = !stage_end || left > kStagePages;
      uint32_t next = pair;
      int meta_n = meta;
      if (!stage_end) {
        next = pair + PJ * 2 * PAGE;
      } else if (more) {
        if (!ready(c + 1)) {
          gave_up = true;
          break;
        }
        const int sn = (c + 1) % kStages4;
        next = kv0 + sn * (kStagePages * 2 * PAGE);
        meta_n = (int)lds32(metas + sn * 4);
      }
#pragma unroll
      for (int j = 0; j < PJ; ++j) {
        const uint32_t vp = pair + (j * 2 + 1) * PAGE;
        page_scores<D, NT>(next + j * 2 * PAGE + k_off, t, x[j], qb);
        page_values<D, NT>(vp + v_off, vp + v_off_s, keep[j], pb[j], o);
      }
      pair = next;
      meta = meta_n;
      p0 += PJ;
      if (stage_end) {
        p0 = 0;
        left -= kStagePages;
        s = (c + 1) % kStages4;
        __syncwarp();
        issue();  // into the stage just read
        ++c;
        if (!more) break;
      }
    }

    if (gave_up) break;
    // ---- the segment's result, from registers ----
    if (p.early) pdl_wait();  // outputs are written from here on
    const bool single = p.whole ? p.parts == 1 : ui.f == ui.l;
    if (!p.whole && slice == ui.f && lane == 0)
      p.split[(ui.b * p.num_kv_heads + ui.g) * p.n_rg + ui.rg] =
          make_int2(ui.f, ui.l);
    const size_t slot = (size_t)2 * slice + (slice == ui.f ? 1 : 0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float sum = l[nt][r];
        sum += __shfl_xor_sync(kFull, sum, 4);
        sum += __shfl_xor_sync(kFull, sum, 8);
        sum += __shfl_xor_sync(kFull, sum, 16);
        const int lr = nt * 8 + 2 * t + r, gr = row0 + lr;
        if (gr >= p.rows) continue;
        const float inv = sum == 0.f ? 0.f : p.v_scale / sum;
        const float lse2 = sum == 0.f ? -INFINITY : ref[nt][r] + log2f(sum);
        if (single) {
          const int i = gr / p.group;
          const int h = ui.g * p.group + gr % p.group;
          const size_t row = ((size_t)ui.b * p.q_len + i) * p.num_q_heads + h;
          if (g == 0) p.lse[row] = lse2 * kLn2;
          uint4 *dst = reinterpret_cast<uint4 *>(
              static_cast<uint16_t *>(p.out) + row * D + (D / 8) * g);
#pragma unroll
          for (int i4 = 0; i4 < D / 64; ++i4) {
            uint32_t w[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(
                  o[4 * i4 + x][nt][r] * inv, o[4 * i4 + x][nt][2 + r] * inv);
              w[x] = *reinterpret_cast<const uint32_t *>(&v);
            }
            dst[i4] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        } else {
          float *const to = p.whole ? part_s : p.part_o + slot * RB * D;
          // (+inf, not NaN, of a row that is NaN: maxima keep it and the
          // weight it gives is NaN again)
          if (g == 0)
            (p.whole ? part_s + RB * D : p.part_lse + slot * RB)[lr] =
                lse2 == lse2 ? lse2 : INFINITY;
          float4 *dst = reinterpret_cast<float4 *>(to + lr * D + (D / 8) * g);
#pragma unroll
          for (int i4 = 0; i4 < D / 32; ++i4)
            dst[i4] = make_float4(o[2 * i4][nt][r] * inv, o[2 * i4][nt][2 + r] * inv,
                                  o[2 * i4 + 1][nt][r] * inv,
                                  o[2 * i4 + 1][nt][2 + r] * inv);
        }
      }
  }

  // ---- the parts of a whole group meet: every warp of the team comes here
  // (their limits run out on their own), then takes some of the rows ----
  if (!p.whole || p.parts == 1) return;
  const Seg4 u0 = inf.seg[0];
  __syncwarp();
  if (lane == 0) part_s[RB * D + RB] = gave_up ? 1.f : 0.f;
  if (!u0.valid && lane < RB) part_s[RB * D + lane] = -INFINITY;
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * p.parts) : "memory");
  if (u0.L < p.q_len || u0.L > (long long)p.max_blocks * kBlockSize) return;
  if (p.early) pdl_wait();
  constexpr int STRIDE = sizeof(Warp4<D, kStages4>) / 4;  // to the next part
  const float *const first = part_s - part * STRIDE;
  for (int x = 0; x < p.parts; ++x)
    if (first[x * STRIDE + RB * D + RB] != 0.f) return;
  for (int lr = part; lr < RB; lr += p.parts) {
    const int gr = u0.rg * RB + lr;
    if (gr >= p.rows) break;
    float m = -INFINITY;
    for (int x = 0; x < p.parts; ++x) m = fmaxf(m, first[x * STRIDE + RB * D + lr]);
    float sum = 0.f, a[D / 32] = {};
    for (int x = 0; x < p.parts; ++x) {
      const float lx = first[x * STRIDE + RB * D + lr];
      if (lx == -INFINITY) continue;  // (its rows may not be written)
      const float w = ex2(lx - m);
      sum += w;
#pragma unroll
      for (int d = 0; d < D / 32; ++d)
        a[d] = fmaf(w, first[x * STRIDE + lr * D + (D / 32) * lane + d], a[d]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i = gr / p.group, h = u0.g * p.group + gr % p.group;
    const size_t row = ((size_t)u0.b * p.q_len + i) * p.num_q_heads + h;
    uint32_t w[D / 64];
#pragma unroll
    for (int d = 0; d < D / 64; ++d) {
      const __nv_bfloat162 v =
          __floats2bfloat162_rn(a[2 * d] * inv, a[2 * d + 1] * inv);
      w[d] = *reinterpret_cast<const uint32_t *>(&v);
    }
    uint32_t *const dst = reinterpret_cast<uint32_t *>(
        static_cast<uint16_t *>(p.out) + row * D) + (D / 64) * lane;
    if constexpr (D == 128)
      *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[D / 64 - 1]);
    else
      dst[0] = w[0];
    if (lane == 0) p.lse[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
  }
}

// Joins the partials of the groups that slice borders cut: one CTA per group
// and query row, its warps taking the group's slices in turn, eight loads in
// flight each; the warps' states meet in shared memory in a fixed order.
constexpr int kMergeWarps4 = 4;
template <int D>
__global__ void __launch_bounds__(32 * kMergeWarps4)
    merge_fp4_kernel(const AttnParams p) {
  constexpr int LPS = D / 4;       // lanes of a slice's row
  constexpr int SPW = 32 / LPS;    // slices a warp takes at once
  constexpr int STEP = kMergeWarps4 * SPW;
  constexpr int UNROLL = 4;
  __shared__ float sm_m[STEP], sm_w[STEP];
  __shared__ float4 sm_o[STEP][LPS];
  pdl_launch_dependents();
  pdl_wait();  // launched early: the attention grid must have finished
  const int group = blockIdx.x / p.merge_rows, lr = blockIdx.x % p.merge_rows;
  const int rg = group % p.n_rg, g = (group / p.n_rg) % p.num_kv_heads;
  const int b = group / (p.n_rg * p.num_kv_heads);
  const int gr = rg * p.rb + lr;
  const int L = p.seq_lens[b];
  const int2 fl = p.split[group];
  // nobody records a group of a sequence whose length is out of range, nor
  // one whose slices gave up (a timeout): an unwritten record names anything,
  // so it is followed only within the slots there are
  if (gr >= p.rows || L < p.q_len || L > (long long)p.max_blocks * kBlockSize ||
      fl.x < 0 || fl.y <= fl.x || fl.y >= p.slices)
    return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int me = warp * SPW + lane / LPS, d4 = lane % LPS;
  const int ns = fl.y - fl.x + 1;
  float m = -INFINITY, w_sum = 0.f;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = me; s0 < ns; s0 += STEP * UNROLL) {
    float ls[UNROLL];
    float4 v[UNROLL];
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const int s = s0 + u * STEP;
      ls[u] = -INFINITY;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s < ns) {
        const size_t row =
            ((size_t)2 * (fl.x + s) + (s == 0 ? 1 : 0)) * p.rb + lr;
        ls[u] = p.part_lse[row];
        v[u] = reinterpret_cast<const float4 *>(p.part_o)[row * LPS + d4];
      }
    }
    float mn = m;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) mn = fmaxf(mn, ls[u]);
    if (mn == -INFINITY) continue;
    const float sc = ex2(m - mn);
    w_sum *= sc;
    a.x *= sc; a.y *= sc; a.z *= sc; a.w *= sc;
#pragma unroll
    for (int u = 0; u < UNROLL; ++u) {
      const float w = ex2(ls[u] - mn);
      w_sum += w;
      a.x = fmaf(w, v[u].x, a.x);
      a.y = fmaf(w, v[u].y, a.y);
      a.z = fmaf(w, v[u].z, a.z);
      a.w = fmaf(w, v[u].w, a.w);
    }
    m = mn;
  }
  sm_o[me][d4] = a;
  if (d4 == 0) {
    sm_m[me] = m;
    sm_w[me] = w_sum;
  }
  __syncthreads();
  if (threadIdx.x >= LPS) return;
  float M = -INFINITY;
#pragma unroll
  for (int x = 0; x < STEP; ++x) M = fmaxf(M, sm_m[x]);
  float total = 0.f;
  a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int x = 0; x < STEP; ++x) {
    const float w = sm_m[x] == -INFINITY ? 0.f : ex2(sm_m[x] - M);
    const float4 v = sm_o[x][d4];
    total = fmaf(w, sm_w[x], total);
    a.x = fmaf(w, v.x, a.x);
    a.y = fmaf(w, v.y, a.y);
    a.z = fmaf(w, v.z, a.z);
    a.w = fmaf(w, v.w, a.w);
  }
  const float inv = total == 0.f ? 0.f : 1.f / total;
  const int i = gr / p.group, h = g * p.group + gr % p.group;
  const size_t row = ((size_t)b * p.q_len + i) * p.num_q_heads + h;
  const __nv_bfloat162 lo = __floats2bfloat162_rn(a.x * inv, a.y * inv);
  const __nv_bfloat162 hi = __floats2bfloat162_rn(a.z * inv, a.w * inv);
  reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + row * D)[d4] =
      make_uint2(*reinterpret_cast<const uint32_t *>(&lo),
                 *reinterpret_cast<const uint32_t *>(&hi));
  if (d4 == 0)
    p.lse[row] = total == 0.f ? -INFINITY : (M + log2f(total)) * kLn2;
}

// ---- host side ----

template <int D, int NT>
size_t smem4(int batch) {
  return sizeof(Smem4<D, NT, warps4<NT>(), stages4<NT>()>) + sizeof(int) * 2 * (size_t)batch + 128;
}

template <int D, int NT>
cudaError_t launch4(AttnParams p, int grid, cudaStream_t st) {
  p.slices = grid * warps4<NT>();
  static_assert(sizeof(Smem4<D, NT, warps4<NT>(), stages4<NT>()>) +
                        sizeof(int) * 2 * kBatchFp4 + 128 <=
                    232448,
                "a CTA's shared memory");
  auto kern = paged_attention_fp4_kernel<D, NT>;
  cudaError_t e = allow_smem((const void *)kern, smem4<D, NT>(p.batch));
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, (unsigned)grid, 32u * warps4<NT>(), smem4<D, NT>(p.batch),
                 st, p);
  if (e != cudaSuccess || p.whole) return e;
  const long long blocks =
      (long long)p.batch * p.num_kv_heads * p.n_rg * p.merge_rows;
  return launch_pdl(merge_fp4_kernel<D>, (unsigned)blocks, 32u * kMergeWarps4, 0,
                    st, p);
}

}  // namespace

// Query rows of a unit: one or two n8 tiles, three for 17 to 24 rows; more
// rows are dealt to several units, each reading the pages again (from L2:
// neighbouring units run close together).  Three tiles convert the cache
// once where two units convert it twice, but a warp goes through its pages
// more slowly and the longer code takes longer to fetch, so it needs work:
// 20 rows, 8 heads, 2048 to 8192 positions: batch 1 31 us against 23, 6 41.5
// against 39 (20 pages a warp), 16 60 against 72, 64 165 against 229.
constexpr int kMinPages3 = 20;
int attention_fp4_rows(int rows, long long pages, int sms) {
  if (rows <= 8) return 8;
  return rows > 16 && rows <= 24 && pages >= (long long)kMinPages3 * warps4<3>() * sms
             ? 24 : 16;
}

int attention_fp4_warps(int rb) { return rb <= 8 ? warps4<1>() : warps4<2>(); }

cudaError_t launch_attention_fp4(const AttnParams &p, int grid,
                                 cudaStream_t stream) {
  const bool d64 = p.head_dim == 64;
  switch (p.rb) {
    case 8: return d64 ? launch4<64, 1>(p, grid, stream) : launch4<128, 1>(p, grid, stream);
    case 24: return d64 ? launch4<64, 3>(p, grid, stream) : launch4<128, 3>(p, grid, stream);
    default: return d64 ? launch4<64, 2>(p, grid, stream) : launch4<128, 2>(p, grid, stream);
  }
}

cudaError_t read_status_attention_fp4(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_attn4, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_attn4, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
