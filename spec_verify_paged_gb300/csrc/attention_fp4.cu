// attention_fp4.cu -- paged decode / speculative-verify attention over a
// 4-bit cache (E2M1 codes, one E4M3 scale per 16 elements; fp4.cuh).
//
// What it computes: as attention.cu, with K = code * scale * k_scale and
// V = code * scale * v_scale.  k_scale is folded into the score scale,
// v_scale multiplies the outputs, code * scale is exact in fp16.
//
// What bounds it: a cached element is 9/16 byte, so at the copy rate an SM
// has to turn 80 elements a nanosecond into products.  On the CUDA cores
// that is an FMA per element and query row on top of the conversion; here
// even a single query row goes through mma.sync (keys as M, query rows as
// N = 8): the conversion (one cvt and one fp16 multiply per two elements)
// is done once per element for all rows, and the codes go from shared
// memory to the matrix instruction through registers only.
//
//  * S^T = K Q^T, one 16-key page per m16 tile: lane (g, t) takes 16
//    consecutive codes (one scale block) of keys g and g + 8 for four
//    k-steps.  Q is fp16 with a power-of-two scale per row (fp4.cuh).
//  * Softmax on the accumulators in the log2 domain.  The running maximum is
//    lazy: a row's reference moves only when a score exceeds it by 2^8, so
//    the usual page costs one vote instead of shuffled maxima.  P is fp16 at
//    2^6 times its softmax weight relative to the reference (at most 2^14),
//    which keeps weights down to 2^-20 normal; the row sums are fp32.
//  * O^T = V^T P^T: P's fp16 pairs become the B operand by movmatrix.  Lane
//    (g, t) reads D/8 consecutive codes of four keys; the nibbles of two
//    keys are interleaved before the conversion, so one cvt yields the pair
//    of keys that the A operand wants for one dimension.
//  * One producer warp, 1-D bulk copies (a head's page is one run of 9 D
//    bytes), stages of two pages, mbarrier ring, stream-K slices and the
//    split merge of attn_common.cuh.
//  * Rows whose memory holds no valid data take no part: masked keys score
//    -inf whatever their bytes, and their V scale is replaced by 0.
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <map>
#include <mutex>
#include <tuple>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_attn4;

namespace {

constexpr int kStagePages = 2;
constexpr int kNoPage = 0x7fffff00;           // j0 of a page that is not there
constexpr float kRefOffset = 6.f;             // P = 2^6 at the reference
constexpr float kRefSlack = 14.f;             // largest log2 P before a move
constexpr float kNoRef = -3e38f;              // below any finite score

// The CTA's shape for NT n8 tiles of query rows per warp.  Up to two tiles:
// four consumer warps and the producer warp, several CTAs per SM.  From
// three on a consumer holds 32 accumulators per tile: one CTA per SM, two
// warpgroups of consumers and one whose first warp produces; 384 threads
// launched with 168 registers each are split 224 / 56 (2 x 128 x 224 + 128 x
// 56 = 384 x 168).
template <int NT>
struct Shape4 {
  static constexpr bool kWide = NT > 2;
  static constexpr int W = kWide ? 8 : 4;  // consumer warps
  static constexpr int THREADS = kWide ? 384 : 160;
  static constexpr int CTAS = NT == 1 ? 3 : kWide ? 1 : 2;  // per SM
  static constexpr int STAGES = kWide ? 16 : 8;
};

// MT warps share a stage.
template <int D, int NT, int MT>
struct Smem4 {
  static constexpr int kWarps4 = Shape4<NT>::W, kStages4 = Shape4<NT>::STAGES;
  static constexpr int PAGE = 9 * D;  // bytes of one head's 16 rows
  static constexpr int RW = 8 * NT;
  static constexpr int RB = RW * MT;
  static constexpr bool kQSmem = NT > 2;
  alignas(128) unsigned char kv[kStages4][kStagePages][2][PAGE];
  union {
    uint2 q[kWarps4][kQSmem ? NT * (D / 16) : 1][32];  // Q operand fragments
    float o[kWarps4][RW][D + 4];                       // states, segment end
  } u;
  float red_m[kWarps4][RW];
  float red_l[kWarps4][RW];
  float wf[kWarps4][RB];
  UnitInfo unit[kUnitRing];
  int j0[kStages4][kStagePages];
  int checked[kStages4];  // the stage's keys need the visibility test
  uint64_t full[kStages4], empty[kStages4];
  uint64_t ufull[kUnitRing], uempty[kUnitRing];
  uint64_t epi;
#ifdef SVP_TEST_STALL_AFTER
  uint64_t stall;  // test builds: a barrier nothing arrives on
#endif
  int abort_flag;
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
  float odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
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
          mma_f16(NT == 1 && i ? odd : s[nt], a, b.x, b.y);
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

template <int D, int NT, int MT>
__global__ void __launch_bounds__(Shape4<NT>::THREADS, Shape4<NT>::CTAS)
    paged_attention_fp4_kernel(const AttnParams p) {
  using S = Smem4<D, NT, MT>;
  constexpr int RW = S::RW, RB = S::RB;
  constexpr int kWarps4 = S::kWarps4, kStages4 = S::kStages4;
  constexpr int NSTREAM = kWarps4 / MT;
  constexpr int KS = D / 16;
  constexpr int PJ = NT <= 3 ? kStagePages : 1;  // pages scored together
  // as in attention.cu: a stage always belongs to the same stream
  static_assert(kStages4 % NSTREAM == 0, "ring depth: a multiple of the streams");
  extern __shared__ unsigned char smem_raw[];
  S &sm = *reinterpret_cast<S *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const int groups_per_seq = p.num_kv_heads * p.n_rg;

  if (tid == 0) {
    for (int s = 0; s < kStages4; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], MT);
    }
    for (int u = 0; u < kUnitRing; ++u) {
      mbar_init(&sm.ufull[u], 1);
      mbar_init(&sm.uempty[u], 1);
    }
    mbar_init(&sm.epi, kWarps4);
#ifdef SVP_TEST_STALL_AFTER
    mbar_init(&sm.stall, 1);
#endif
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  // launched early: see AttnParams::early
  if (!p.early) pdl_wait();
  if (tid == 0) {
    p.desc[blockIdx.x].valid = 0;  // until a split group starts
    pdl_launch_dependents();       // the merge may be scheduled
  }

  if (Shape4<NT>::kWide && warp >= kWarps4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
  }
  if (warp > kWarps4) {
    // the producer's idle neighbours
  } else if (warp == kWarps4) {
    // ======================= producer warp =======================
    int *const seqlen = sm.prefix + p.batch + 1;
    const int total = build_prefix(p, sm.prefix, seqlen, groups_per_seq, lane,
                                   &g_status_attn4);
    const int n_ctas = working_ctas(total, p.min_pages);
    const int range_begin = slice_begin(blockIdx.x, total, n_ctas);
    const int range_end = blockIdx.x < n_ctas
                              ? slice_begin(blockIdx.x + 1, total, n_ctas)
                              : total;
    int c = 0;   // stages issued so far
    int us = 0;  // segments published so far
    bool waited = !p.early;
    bool ok = true;
    int pos = range_begin;
    while (true) {
      const int slot = us % kUnitRing;
      if (lane == 0)
        ok = mbar_wait(&sm.uempty[slot], ((us / kUnitRing) & 1) ^ 1);
      ok = __shfl_sync(kFull, ok, 0) && !sm.abort_flag;
      if (!ok) break;
      const UnitInfo seg =
          pos < range_end
              ? decode_segment(p, sm.prefix, seqlen, groups_per_seq, pos,
                               us == 0, range_end, total, n_ctas)
              : UnitInfo{};
      if (!seg.valid) {
        if (lane == 0) {
          sm.unit[slot].valid = 0;
          mbar_arrive(&sm.ufull[slot]);
        }
        break;
      }
      const int n_pages = seg.n_pages;
      // positions of the unit's first and last row: pages that end by the
      // first (with a tree: before its nodes) and lie in the last one's
      // window need no per-key test
      const int base = seg.seq_len - p.q_len;
      const int t_min =
          p.tree_mask ? base - 1 : base + (seg.rg * RB) / p.group;
      const int t_max =
          base + (min(seg.rg * RB + RB, p.rows) - 1) / p.group;
      if (lane == 0) {
        sm.unit[slot] = seg;
        mbar_arrive(&sm.ufull[slot]);
      }
      // 32 block-table entries at a time (16 stages), the next 32 loaded
      // while these go out
      auto entry = [&](int k) {
        return k < n_pages
                   ? __ldg(p.block_table + (size_t)seg.b * p.max_blocks +
                           logical_block(seg, seg.page0 + k))
                   : -1;
      };
      int phys = entry(lane);
      for (int k0 = 0; k0 < n_pages && ok; k0 += 32) {
        const int next = entry(k0 + 32 + lane);
        const int n_here = min(32, n_pages - k0);
        // stages go out in batches, as in attention.cu: lane i arms stage
        // c + i, lane 4 i + r issues copy r of its four
        constexpr int MAXB = 8 < kStages4 ? 8 : kStages4;
        for (int kk = 0; kk < n_here;) {
#ifdef SVP_TEST_STALL_AFTER
          if (c >= SVP_TEST_STALL_AFTER) {
            if (lane == 0) ok = mbar_wait(&sm.stall, 0);
            ok = __shfl_sync(kFull, ok, 0);
            if (!ok) break;
          }
#endif
          const int left = min((n_here - kk + 1) / kStagePages, MAXB);
          if (!waited) {
            const int lb = logical_block(
                seg, seg.page0 + min(k0 + kk + left * kStagePages, n_pages) - 1);
            if ((lb + 1) * kBlockSize > seg.seq_len - p.q_len) {
              pdl_wait();  // it may hold some of the appended positions
              waited = true;
            }
          }
          bool ready = false;
          if (lane == 0)
            ready = mbar_wait(&sm.empty[c % kStages4], ((c / kStages4) & 1) ^ 1);
          ok = __shfl_sync(kFull, ready, 0);
          if (!ok) break;
          if (lane > 0 && lane < left)
            ready = mbar_ready(&sm.empty[(c + lane) % kStages4],
                               (((c + lane) / kStages4) & 1) ^ 1);
          const unsigned run = __ballot_sync(kFull, lane < left && ready);
          const int n = __ffs(~run) - 1;  // stages c .. c + n - 1 are free
          int ph[kStagePages];
#pragma unroll
          for (int x = 0; x < kStagePages; ++x)
            ph[x] = __shfl_sync(kFull, phys, min(kk + kStagePages * lane + x, 31));
          const int ci = lane >> 2, part = lane & 3;  // this lane's copy
          const int ph_c = __shfl_sync(
              kFull, phys, min(kk + kStagePages * ci + (part >> 1), 31));
          if (lane < n) {
            const int s = (c + lane) % kStages4;
            uint32_t bytes = 0;
            bool all_vis = true;
#pragma unroll
            for (int x = 0; x < kStagePages; ++x) {
              const int k = k0 + kk + kStagePages * lane + x;
              int j0 = kNoPage;
              if (k < n_pages) {
                if (ph[x] >= 0 && ph[x] < p.num_blocks) {
                  j0 = logical_block(seg, seg.page0 + k) * kBlockSize;
                  bytes += 2 * S::PAGE;
                } else {
                  raise4(SVP_DEV_BAD_BLOCK_ID);
                }
              }
              sm.j0[s][x] = j0;
              const int j1 = j0 + kBlockSize - 1;
              all_vis = all_vis && j1 <= t_min &&
                        (p.window == 0 || j1 < p.n_sink ||
                         j0 > t_max - p.window);
            }
            sm.checked[s] = !all_vis;
            if (bytes)
              mbar_arrive_expect_tx(&sm.full[s], bytes);
            else
              mbar_arrive(&sm.full[s]);
          }
          __syncwarp();
          if (ci < n && k0 + kk + kStagePages * ci + (part >> 1) < n_pages &&
              ph_c >= 0 && ph_c < p.num_blocks) {
            const int s = (c + ci) % kStages4;
            const size_t off =
                ((size_t)ph_c * p.num_kv_heads + seg.g) * (size_t)S::PAGE;
            bulk_g2s(sm.kv[s][part >> 1][part & 1],
                     static_cast<const unsigned char *>(part & 1 ? p.v_cache
                                                                 : p.k_cache) +
                         off,
                     S::PAGE, &sm.full[s]);
          }
          c += n;
          kk += n * kStagePages;
        }
        phys = next;
      }
      if (!ok) break;
      pos = seg.item0 + (n_pages + p.ppi - 1) / p.ppi;
      ++us;
    }
    if (!ok) {
      if (lane == 0) {
        raise4(SVP_DEV_TIMEOUT);
        sm.abort_flag = 1;
        for (int k = max(0, c - kStages4); k < c; ++k)
          (void)mbar_wait_drain(&sm.full[k % kStages4], (k / kStages4) & 1);
      }
    }
  } else {
    // ======================= consumer warps =======================
    if (Shape4<NT>::kWide)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
    const int g = lane >> 2, t = lane & 3;
    const int stream = warp / MT, mt = warp % MT;
    int c = 0, us = 0;
    uint32_t epi_phase = 0;
    while (true) {
      const int slot = us % kUnitRing;
      const bool ok =
          __all_sync(kFull, mbar_wait(&sm.ufull[slot], (us / kUnitRing) & 1));
      if (!ok) {
        if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
        break;
      }
      const UnitInfo ui = sm.unit[slot];
      if (!ui.valid || sm.abort_flag) break;
      const int b = ui.b, kvh = ui.g, rg = ui.rg, L = ui.seq_len;
      const int t0 = L - p.q_len;
      const int row0 = rg * RB + mt * RW;  // this warp's first row
      bool aborted = false;

      // ---- Q fragments: row n = g of each n8 tile, fp16, scaled by row ----
      uint2 qf[S::kQSmem ? 1 : NT][S::kQSmem ? 1 : KS];
      float qs[NT][2];  // score scale of rows 2t, 2t + 1
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int gr = row0 + nt * 8 + g;
        const bool valid = gr < p.rows;
        const int grc = valid ? gr : rg * RB;
        const int i = grc / p.group;
        const int h = kvh * p.group + grc % p.group;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            static_cast<const uint16_t *>(p.q) +
            (((size_t)b * p.q_len + i) * p.num_q_heads + h) * D);
        uint32_t w[KS][2];
        uint32_t top = 0;
#pragma unroll
        for (int x = 0; x < KS / 2; ++x) {  // q_dim: D/4 consecutive dims
          uint4 v = __ldg(src + (KS / 2) * t + x);
          if (!valid) v = make_uint4(0, 0, 0, 0);
          w[2 * x][0] = v.x;
          w[2 * x][1] = v.y;
          w[2 * x + 1][0] = v.z;
          w[2 * x + 1][1] = v.w;
        }
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            top = max(top, max(w[ks][x] & 0x7fffu, (w[ks][x] >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int e = q_exponent(__uint_as_float(top << 16));
        const float f = pow2i(14 - e);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t hh[2];
#pragma unroll
          for (int x = 0; x < 2; ++x)
            hh[x] = pack_h2(__uint_as_float(w[ks][x] << 16) * f,
                            __uint_as_float(w[ks][x] & 0xffff0000u) * f);
          if constexpr (S::kQSmem)
            sm.u.q[warp][nt * KS + ks][lane] = make_uint2(hh[0], hh[1]);
          else
            qf[nt][ks] = make_uint2(hh[0], hh[1]);
        }
        const float sc = p.qscale * pow2i(e - 14);
        qs[nt][0] = __shfl_sync(kFull, sc, 8 * t);
        qs[nt][1] = __shfl_sync(kFull, sc, 8 * t + 4);
      }
      const uint32_t q_addr = smem_u32(&sm.u.q[warp][0][lane]);
      auto qb = [&](int ks, int nt) -> uint2 {
        if constexpr (S::kQSmem)
          return lds64(q_addr + (nt * KS + ks) * (32 * (int)sizeof(uint2)));
        else
          return qf[nt][ks];
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
      const uint32_t kv0 = smem_u32(&sm.kv[0][0][0][0]);
      const uint32_t k_off = k_lane<D>(g, t), v_off = v_lane<D>(g, t);
      const uint32_t v_off_s = v_lane_scale<D>(g, t);
      const int n_stages = (ui.n_pages + kStagePages - 1) / kStagePages;
      const int first = ((stream - c) % NSTREAM + NSTREAM) % NSTREAM;
      for (int k = first; k < n_stages; k += NSTREAM) {
        const int cc = c + k;
        const int s = cc % kStages4;
        const bool got =
            __all_sync(kFull, mbar_wait(&sm.full[s], (cc / kStages4) & 1));
        if (!got) {
          if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
          aborted = true;
          break;
        }
        const uint32_t st = kv0 + s * (kStagePages * 2 * S::PAGE);
        const bool checked = sm.checked[s] != 0;  // warp-uniform
#pragma unroll
        for (int p0 = 0; p0 < kStagePages; p0 += PJ) {
          float x[PJ][NT][4], y[PJ][NT][4];
#pragma unroll
          for (int j = 0; j < PJ; ++j)
            page_scores<D, NT>(st + (p0 + j) * 2 * S::PAGE + k_off, t, x[j], qb);
          // ---- softmax with a lazy reference ----
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
                  bits = row_tree_bits(p, b, i);
                }
                float mx = -INFINITY;
#pragma unroll
                for (int j = 0; j < PJ; ++j)
#pragma unroll
                  for (int h = 0; h < 2; ++h) {
                    float z = x[j][nt][2 * h + r] * qs[nt][r];
                    if (checked &&
                        !key_visible(sm.j0[s][p0 + j] + fp4_key(g, h), t0 + i,
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
                  const int key = sm.j0[s][p0 + j] + 4 * t + sx;
                  if (!(key < L && (p.window == 0 || key < p.n_sink ||
                                    key > t0 - p.window)))
                    keep[j] &= ~(1u << sx);
                }
            }
          }
#pragma unroll
          for (int j = 0; j < PJ; ++j) {
            uint32_t pb[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                y[j][nt][e] = ex2(y[j][nt][e]);
                l[nt][e & 1] += y[j][nt][e];
              }
              pb[nt][0] = transpose8(pack_h2(y[j][nt][0], y[j][nt][1]));
              pb[nt][1] = transpose8(pack_h2(y[j][nt][2], y[j][nt][3]));
            }
            const uint32_t vp = st + ((p0 + j) * 2 + 1) * S::PAGE;
            page_values<D, NT>(vp + v_off, vp + v_off_s, keep[j], pb, o);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[s]);
      }
      c += n_stages;

      // ---- this warp's states to shared memory ----
      __syncwarp();  // its last reads of the Q fragments
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float sum = l[nt][r];
          sum += __shfl_xor_sync(kFull, sum, 4);
          sum += __shfl_xor_sync(kFull, sum, 8);
          sum += __shfl_xor_sync(kFull, sum, 16);
          l[nt][r] = sum;
        }
      if constexpr (S::kQSmem) {
        // the states overlie the Q fragments of every warp
        if (!consumer_sync(&sm.epi, epi_phase, lane)) {
          if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
          break;
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = nt * 8 + 2 * t + r;
          if (g == 0) {
            sm.red_m[warp][row] = l[nt][r] == 0.f ? -INFINITY : ref[nt][r];
            sm.red_l[warp][row] = l[nt][r];
          }
          float *dst = &sm.u.o[warp][row][(D / 8) * g];
#pragma unroll
          for (int i = 0; i < D / 16; i += 2)
            *reinterpret_cast<float4 *>(dst + 2 * i) =
                make_float4(o[i][nt][r], o[i][nt][2 + r], o[i + 1][nt][r],
                            o[i + 1][nt][2 + r]);
        }

      // ---- epilogue: merge the warps' states (as attention.cu) ----
      if (p.early) pdl_wait();  // outputs are written from here on
      if (!consumer_sync(&sm.epi, epi_phase, lane) || aborted) {
        if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
        break;
      }
      const bool single = ui.f == ui.l;
      const size_t pslot = (size_t)(2 * blockIdx.x + ui.slot);
      const int vrows = min(RB, p.rows - rg * RB);
      if (tid < vrows) {
        const int r = tid, w0 = r / RW, lr = r % RW;
        float M = -INFINITY;
#pragma unroll
        for (int w = w0; w < kWarps4; w += MT) M = fmaxf(M, sm.red_m[w][lr]);
        float Lsum = 0.f;
        float f[NSTREAM];
#pragma unroll
        for (int k = 0; k < NSTREAM; ++k) {
          const float mw = sm.red_m[w0 + k * MT][lr];
          f[k] = (mw == -INFINITY) ? 0.f : ex2(mw - M);
          Lsum = fmaf(f[k], sm.red_l[w0 + k * MT][lr], Lsum);
        }
        const float inv = Lsum == 0.f ? 0.f : 1.f / Lsum;
#pragma unroll
        for (int k = 0; k < NSTREAM; ++k) sm.wf[w0 + k * MT][r] = f[k] * inv;
        const float lse2 = Lsum == 0.f ? -INFINITY : M + log2f(Lsum);
        const int gr = rg * RB + r;
        if (single) {
          const int i = gr / p.group;
          const int h = kvh * p.group + gr % p.group;
          p.lse[((size_t)b * p.q_len + i) * p.num_q_heads + h] = lse2 * kLn2;
        } else {
          p.part_lse[pslot * RB + r] = lse2;
        }
      }
      if (!consumer_sync(&sm.epi, epi_phase, lane)) {
        if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
        break;
      }
      for (int e4 = tid; e4 < vrows * (D / 4); e4 += kWarps4 * 32) {
        const int r = e4 / (D / 4), d = (e4 % (D / 4)) * 4;
        const int w0 = r / RW, lr = r % RW;
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < NSTREAM; ++k) {
          const float f = sm.wf[w0 + k * MT][r];
          const float4 v =
              *reinterpret_cast<const float4 *>(&sm.u.o[w0 + k * MT][lr][d]);
          a.x = fmaf(f, v.x, a.x);
          a.y = fmaf(f, v.y, a.y);
          a.z = fmaf(f, v.z, a.z);
          a.w = fmaf(f, v.w, a.w);
        }
        a.x *= p.v_scale;
        a.y *= p.v_scale;
        a.z *= p.v_scale;
        a.w *= p.v_scale;
        if (single) {
          const int gr = rg * RB + r;
          const int i = gr / p.group;
          const int h = kvh * p.group + gr % p.group;
          uint16_t *dst = static_cast<uint16_t *>(p.out) +
                          (((size_t)b * p.q_len + i) * p.num_q_heads + h) * D + d;
          store_out(dst + 0, a.x);
          store_out(dst + 1, a.y);
          store_out(dst + 2, a.z);
          store_out(dst + 3, a.w);
        } else {
          *reinterpret_cast<float4 *>(p.part_o + (pslot * RB + r) * D + d) = a;
        }
      }
      if (!single && tid == 0) record_split(p, ui, blockIdx.x);
      if (!consumer_sync(&sm.epi, epi_phase, lane)) {
        if (lane == 0) { raise4(SVP_DEV_TIMEOUT); sm.abort_flag = 1; }
        break;
      }
      if (tid == 0) mbar_arrive(&sm.uempty[slot]);
      ++us;
    }
  }

  __syncthreads();  // no warp leaves while the others may use the barriers
}

// ---- host side ----

std::mutex g_mu4;
std::map<std::tuple<int, const void *, size_t>, int> g_occ4;

template <int D, int NT, int MT>
size_t smem4(int batch) {
  const size_t bucket = ((size_t)batch + 255) / 256 * 256;
  return sizeof(Smem4<D, NT, MT>) + sizeof(int) * (2 * bucket + 1) + 128;
}

// shared-memory attribute and occupancy, once per device and size; < 0 if
// the runtime refuses
template <int D, int NT, int MT>
int prepare4(int batch) {
  const size_t smem = smem4<D, NT, MT>(batch);
  auto kern = paged_attention_fp4_kernel<D, NT, MT>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return -1;
  const auto key = std::make_tuple(dev, (const void *)kern, smem);
  std::lock_guard<std::mutex> lk(g_mu4);
  auto it = g_occ4.find(key);
  if (it != g_occ4.end()) return it->second;
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess ||
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, Shape4<NT>::THREADS, smem) !=
          cudaSuccess)
    return -1;
  n = n > 0 ? n : 1;
  g_occ4[key] = n;
  return n;
}

#define SVP_DISPATCH4(CALL)                                   \
  do {                                                        \
    if (head_dim == 64) {                                     \
      switch (rb) {                                           \
        case 8: CALL(64, 1, 1); break;                        \
        case 16: CALL(64, 2, 1); break;                       \
        case 24: CALL(64, 3, 1); break;                       \
        case 32: CALL(64, 4, 1); break;                       \
        case 48: CALL(64, 3, 2); break;                       \
        default: CALL(64, 4, 2); break;                       \
      }                                                       \
    } else {                                                  \
      switch (rb) {                                           \
        case 8: CALL(128, 1, 1); break;                       \
        case 16: CALL(128, 2, 1); break;                      \
        case 24: CALL(128, 3, 1); break;                      \
        case 32: CALL(128, 4, 1); break;                      \
        case 48: CALL(128, 3, 2); break;                      \
        default: CALL(128, 4, 2); break;                      \
      }                                                       \
    }                                                         \
  } while (0)

template <int D, int NT, int MT>
cudaError_t launch4(const AttnParams &p, int grid, cudaStream_t st) {
  if (prepare4<D, NT, MT>(p.batch) < 0) return cudaErrorInvalidValue;
  return launch_pdl(paged_attention_fp4_kernel<D, NT, MT>, (unsigned)grid,
                    (unsigned)Shape4<NT>::THREADS, smem4<D, NT, MT>(p.batch), st, p);
}

}  // namespace

int attention_fp4_rows(int rows) {
  for (int rb : {8, 16, 24, 32, 48, 64})
    if (rows <= rb) return rb;
  // several units per group, each reading the pages again: the fewest rows
  // of padding, then the fewest units
  const int r48 = (rows + 47) / 48 * 48, r64 = (rows + 63) / 64 * 64;
  return r48 < r64 ? 48 : 64;
}

int attention_fp4_ctas_per_sm(int head_dim, int rb, int batch) {
  int n = 1;
#define SVP_CALL(D, NT, MT) n = prepare4<D, NT, MT>(batch)
  SVP_DISPATCH4(SVP_CALL);
#undef SVP_CALL
  return n > 0 ? n : 1;
}

cudaError_t launch_attention_fp4(const AttnParams &p, int grid,
                                 cudaStream_t stream) {
  const int head_dim = p.head_dim, rb = p.rb;
  cudaError_t e = cudaSuccess;
#define SVP_CALL(D, NT, MT) e = launch4<D, NT, MT>(p, grid, stream)
  SVP_DISPATCH4(SVP_CALL);
#undef SVP_CALL
  return e;
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
