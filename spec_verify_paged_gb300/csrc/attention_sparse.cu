// attention_sparse.cu -- attention over listed pages only
// (paged_sparse_attention, include/svp.h): every (sequence, kv head) has its
// own list of pages, each query row attends to the keys of those pages that
// causality or the draft tree lets it see.
//
// What bounds it: the listed K and V rows' bytes, each read once, while a kv
// head has few query rows; the chain of a page's products and softmax beyond.
//
// A cluster of 1 to 16 CTAs takes a unit: a (sequence, kv head) and up to 32 of
// its query rows (8 over an fp32 cache).  Its CTAs split the list and their
// warps deal out the pages; the results meet in distributed shared memory, so
// a call is one launch, without partials in memory.  Every warp copies its own
// pages (cp.async, a ring of three or four, in steps of one page or two), so
// no barrier joins the warps in between.  The 16-byte pieces are swizzled on
// the way so that the matrix operands are read without bank conflicts.  Rows of
// a page past the sequence's end are filled with zeros instead of being read.
//
//  * Keys are the M of mma.sync m16n8k16, query rows the N: S^T = K Q^T,
//    O^T = V^T P^T, so a page's operands are made once for all rows of the
//    unit, and 8 rows take half the products that 16 would.  P goes from S's
//    accumulators to the B operand by movmatrix.  (With the rows as M, each
//    row group of 16 to a warp converted every page for itself: 40 rows over
//    FP8 pages 30 us, against 22.)
//  * bf16: a weight is two bf16 terms, off by 2^-16 of itself, so that the
//    output's own rounding is what an output is off by (0.0017 of its norm
//    over random values, 0.0022 with one term of 2^-8).  The second product
//    costs 1 % where bytes bound the call and up to a fifth where the chain
//    does (32 x 8 lists of 128 pages, 4 rows 43.9 -> 44.3 us, 32 rows 50.7 ->
//    52.7; 4 x 8 of 256, 40 rows 20.7 -> 23.7).  Row sums are fp32.
//  * FP8 and 4-bit rows become fp16 operands between shared memory and the
//    matrix instruction (exact); P is fp16 at 2^6 times its weight, which
//    keeps weights down to 2^-20 normal.  q takes a power-of-two scale per row
//    (fp4.cuh).
//  * fp32: CUDA cores, fp32 throughout.
//  * Softmax in the log2 domain with a lazy reference: it moves only when a
//    score exceeds it by 2^8, so the usual page costs one vote.
//
// Measured (D = 128; of the listed rows' bytes at the copy rate): 32 sequences
// of 8 heads, 128 pages each, 4 query rows: bf16 44.3 us, 0.90; fp32 89, 0.90;
// FP8 29.6, 0.67; 4-bit 23.6, 0.48 (the conversion).  32 rows: bf16 53, FP8 and
// 4-bit 43, fp32 433 (four units).  4 sequences of 8 heads, 256 pages, 40 rows:
// bf16 23.7 us, FP8 22 and 4-bit 22, where the FP8 bytes take 5.1: about 7 us of
// start, look-ups and joining, and 16 pages a warp at 1.7 warps to a scheduler
// (FP8: issue active 40 %, tensor pipe 27 %, an instruction every 2.5 cycles of a
// warp); one unit of 40 rows spills (23), 128 or 168 registers for more warps
// spill more (33).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_sparse;

namespace {

namespace cg = cooperative_groups;

constexpr int kSpTiles = 4;         // most n8 tiles of query rows of a unit
constexpr int kListCap = 512;       // list entries a CTA looks up at once
constexpr int kNoPage = 0x7ffffff0; // first position of a page that is not there
constexpr float kSpNoRef = -3e38f;  // below any score

__device__ __forceinline__ void raise_sparse(unsigned f) {
  atomicOr(&g_status_sparse, f);
}

template <int DT, int D, int NT>
struct SpShape {
  static constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                              : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  static constexpr int PAGE = kBlockSize * ROWB;  // one side
  // warps of a CTA, of which an SM holds PER_SM: eight over small pages, whose
  // rings leave the room, while 128 registers are enough
  static constexpr int WARPS = PAGE < 4096 && DT != SVP_F32 && NT == 1 ? 8 : 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int STAGES = PAGE * WARPS >= 16384 ? 3 : 4;
  // pages that a warp takes at once: two where latency counts more than room
  // and registers (their products are independent chains, one vote serves both)
  static constexpr int AT_ONCE = PAGE < 4096 && DT != SVP_F32 && NT > 1 ? 2 : 1;
  static constexpr int ROWS = NT == 0 ? 4 : 8 * NT;  // of a unit
  static constexpr int WARP = STAGES * 2 * PAGE;  // a warp's ring
  // the warps' results take the rings' place at the end
  static constexpr int RES_ROW = 4 * D + 16;
  static constexpr int RES = WARPS * ROWS * (RES_ROW + 8);
  static constexpr int RING = WARPS * WARP > RES ? WARPS * WARP : RES;
  static constexpr int LIST = kListCap * 8;
  // query rows: with many tiles, as fragments for all warps; fp32 rows, and
  // each warp's weights
  static constexpr bool Q_SHARED = DT != SVP_F32 && NT > 2;
  static constexpr int QROW = 4 * D + 32;
  static constexpr int Q = DT == SVP_F32 ? ROWS * QROW + WARPS * ROWS * kBlockSize * 4
                           : Q_SHARED    ? NT * ((D / 16) * 256 + 32)
                                         : 0;
  static constexpr int SMEM = RING + LIST + 64 + (Q > ROWS * 8 ? Q : ROWS * 8);
  // an SM's 228 KB hold two CTAs, each with a KB of its own, or one over fp32
  // pages of D = 128 (204 and 207 KB)
  static constexpr int PER_SM = 2 * (SMEM + 1024) <= 228 * 1024 ? 2 : 1;
};

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Shared-memory reads by 32-bit address.  volatile keeps them behind the
// barriers, and nothing else in order.
__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a));
}
__device__ __forceinline__ void ldsm4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(a));
}
__device__ __forceinline__ uint4 ls128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 ls64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];"
               : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ls32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ls8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ float4 as_f4(uint4 v) {
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y),
                     __uint_as_float(v.z), __uint_as_float(v.w));
}

template <int DT>
__device__ __forceinline__ void mma16(float (&d)[4], const uint32_t (&a)[4],
                                      uint32_t b0, uint32_t b1) {
  if constexpr (DT == SVP_BF16) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    mma_f16(d, a, b0, b1);
  }
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (DT == SVP_BF16) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  } else {
    return pack_h2(lo, hi);
  }
}

// Where the 16-byte piece c of row r of a page stands in shared memory: rows
// that one access reads side by side lie in different banks.
template <int ROWB>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  if constexpr (ROWB == 64)
    return r * ROWB + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * ROWB + ((c ^ (r & 7)) << 4);
}

// K and V of a page into a ring stage, by a warp; rows past the sequence's end
// become zeros.  e: physical page, first position.
template <int DT, int D>
__device__ __forceinline__ void load_page(const SparseParams &p, uint32_t stage,
                                          int2 e, int head, int L, int lane) {
  using S = SpShape<DT, D, 1>;
  constexpr int PIECES = S::PAGE / 16;  // of a side
  const size_t at = ((size_t)e.x * p.num_kv_heads + head) * S::PAGE;
  const int rows = max(min(L - e.y, kBlockSize), 0);
#pragma unroll
  for (int i = 0; i < (2 * PIECES + 31) / 32; ++i) {
    const int x = i * 32 + lane;
    if (2 * PIECES % 32 != 0 && x >= 2 * PIECES) break;
    const int side = x / PIECES, y = x % PIECES;
    const char *src =
        static_cast<const char *>(side ? p.v_cache : p.k_cache) + at + y * 16;
    uint32_t dst = stage + side * S::PAGE;
    int bytes;
    if constexpr (DT == SVP_FP4_E2M1) {
      // pieces straddle the 36- or 72-byte rows
      dst += y * 16;
      bytes = min(max(rows * S::ROWB - y * 16, 0), 16);
    } else {
      constexpr int PPR = S::ROWB / 16;
      dst += piece<S::ROWB>(y / PPR, y % PPR);
      bytes = y / PPR < rows ? 16 : 0;
    }
    cp16(dst, src, bytes);
  }
}

// What a row may see: keys up to `t`; with a tree, of the keys from `base` on
// those whose bit is set.
struct RowMask {
  int t, base;
  uint32_t bits;
  __device__ __forceinline__ bool sees(int j) const {
    return j <= t && (j < base || ((bits >> ((j - base) & 31)) & 1u));
  }
};

__device__ __forceinline__ RowMask row_mask(const SparseParams &p, int b, int L,
                                            int row) {
  RowMask m;
  m.base = L - p.q_len;
  const int i = min(row, p.rows - 1) / p.group;
  m.t = m.base + i;
  m.bits = p.tree_mask ? p.tree_mask[(size_t)b * p.q_len + i] : 0xffffffffu;
  return m;
}

// A warp's state over 16-bit operands.  Lane (g, t) of S^T tile n: keys g and
// g + 8, query rows 8 n + 2 t and + 1; of O^T: two dimensions, the same rows.
template <int DT, int D, int NT>
struct WarpMma {
  using S = SpShape<DT, D, NT>;
  static constexpr int KS = D / 16, MT = D / 16, ROWB = S::ROWB;
  static constexpr float kOff = DT == SVP_BF16 ? 0.f : 6.f;
  static constexpr float kSlack = DT == SVP_BF16 ? 8.f : 14.f;
  static constexpr int kTerms = DT == SVP_BF16 ? 2 : 1;  // of a weight
  static constexpr bool Q_SHARED = S::Q_SHARED;
  uint2 q[Q_SHARED ? 1 : NT][Q_SHARED ? 1 : KS];
  float o[MT][NT][4];
  float ref[NT][2], sum[NT][2], factor[NT][2];
  int t_all;  // keys up to here are seen by all of the unit's rows

  // Key of row m (0..7) of half h of S^T.
  static __device__ __forceinline__ int key(int m, int h) {
    return DT == SVP_FP4_E2M1 ? fp4_key(m, h) : m + 8 * h;
  }
  // Dimension of row g of half h of O^T tile i.
  static __device__ __forceinline__ int dim(int i, int h, int g) {
    return DT == SVP_BF16       ? 16 * i + 8 * h + g
           : DT == SVP_FP8_E4M3 ? 16 * i + 2 * g + h
                                : (D / 8) * g + 2 * i + h;
  }

  // The B fragments of tile n and their rows' factor: lane (g, t) holds row
  // 8 n + g.
  __device__ __forceinline__ float fragments(const SparseParams &p, int b, int head,
                                             int row0, int n, uint2 (&w)[KS], int lane) {
    const int g = lane >> 2, t = lane & 3;
    const int row = row0 + 8 * n + g;
    const bool there = row < p.rows;
    const int r = there ? row : 0;
    const uint16_t *src = static_cast<const uint16_t *>(p.q) +
                          (((size_t)b * p.q_len + r / p.group) * p.num_q_heads +
                           (size_t)head * p.group + r % p.group) * D;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      if constexpr (DT == SVP_BF16) {
        w[ks].x = *reinterpret_cast<const uint32_t *>(src + 16 * ks + 2 * t);
        w[ks].y = *reinterpret_cast<const uint32_t *>(src + 16 * ks + 2 * t + 8);
      } else {
        w[ks] = *reinterpret_cast<const uint2 *>(src + (D / 4) * t + 4 * ks);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
      if (!there) w[ks] = make_uint2(0u, 0u);
    float f = p.qscale;
    if constexpr (DT != SVP_BF16) {
      float top = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint32_t x[2] = {w[ks].x, w[ks].y};
#pragma unroll
        for (int y = 0; y < 2; ++y)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(x[y] << 16)),
                                 fabsf(__uint_as_float(x[y] & 0xffff0000u))));
      }
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
      top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
      const int e = q_exponent(top);
      const float up = pow2i(14 - e);
      f *= pow2i(e - 14);
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
        w[ks] = make_uint2(pack_h2(__uint_as_float(w[ks].x << 16) * up,
                                   __uint_as_float(w[ks].x & 0xffff0000u) * up),
                           pack_h2(__uint_as_float(w[ks].y << 16) * up,
                                   __uint_as_float(w[ks].y & 0xffff0000u) * up));
    }
    return f;
  }

  // Before a barrier: the unit's query fragments, where they are shared a tile
  // to a warp, and their rows' factors behind them.
  __device__ __forceinline__ void load_query(const SparseParams &p, int b, int head,
                                             int row0, unsigned char *shared, int warp,
                                             int lane) {
    if constexpr (Q_SHARED) {
      for (int n = warp; n < NT; n += S::WARPS) {
        uint2 w[KS];
        const float f = fragments(p, b, head, row0, n, w, lane);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          reinterpret_cast<uint2 *>(shared)[(n * KS + ks) * 32 + lane] = w[ks];
        if (lane % 4 == 0)
          reinterpret_cast<float *>(shared + NT * KS * 256)[8 * n + lane / 4] = f;
      }
    } else {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float f = fragments(p, b, head, row0, n, q[n], lane);
#pragma unroll
        for (int e = 0; e < 2; ++e)  // this lane's rows of S^T: 2 t + e
          factor[n][e] = __shfl_sync(kFull, f, 4 * (2 * (lane & 3) + e));
      }
    }
  }

  // After it.
  __device__ __forceinline__ void start(const SparseParams &p, int L, int row0,
                                        const unsigned char *shared, int lane) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][n][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (Q_SHARED)
          factor[n][e] = reinterpret_cast<const float *>(
              shared + NT * KS * 256)[8 * n + 2 * (lane & 3) + e];
        ref[n][e] = kSpNoRef;
        sum[n][e] = 0.f;
      }
    }
    const int base = L - p.q_len;
    t_all = p.tree_mask ? base - 1 : base + min(row0, p.rows - 1) / p.group;
  }

  __device__ __forceinline__ uint2 query(const unsigned char *shared, int n, int ks,
                                         int lane) const {
    if constexpr (Q_SHARED)
      return reinterpret_cast<const uint2 *>(shared)[(n * KS + ks) * 32 + lane];
    else
      return q[n][ks];
  }

  // S^T of a page.  With one tile the even and the odd steps are two chains.
  __device__ __forceinline__ void scores(uint32_t kp, float (&s)[NT][4],
                                         const unsigned char *shared, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
    auto step = [&](int ks, const uint32_t (&a)[4]) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const uint2 b = query(shared, n, ks, lane);
        mma16<DT>(NT == 1 && ks % 2 ? odd : s[n], a, b.x, b.y);
      }
    };
    if constexpr (DT == SVP_BF16) {
      const int r = ((lane >> 3) & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t a[4];
        ldsm4(kp + piece<ROWB>(r, 2 * ks + c), a);
        step(ks, a);
      }
    } else if constexpr (DT == SVP_FP8_E4M3) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 w[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          w[h] = ls128(kp + piece<ROWB>(g + 8 * h, (D / 64) * t + c));
        const uint32_t x[2][4] = {{w[0].x, w[0].y, w[0].z, w[0].w},
                                  {w[1].x, w[1].y, w[1].z, w[1].w}};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t a[4] = {e4m3x2_f16x2(x[0][e]), e4m3x2_f16x2(x[1][e]),
                                 e4m3x2_f16x2(x[0][e] >> 16),
                                 e4m3x2_f16x2(x[1][e] >> 16)};
          step(4 * c + e, a);
        }
      }
    } else {
      constexpr int C = D / 64;  // scale blocks of a lane
      uint32_t w[2][C][2], sc[2][C];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t row = kp + key(g, h) * ROWB;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          if constexpr (D == 128) {
            const uint2 v = ls64(row + 16 * t + 8 * c);
            w[h][c][0] = v.x;
            w[h][c][1] = v.y;
          } else {
            w[h][c][0] = ls32(row + 8 * t);
            w[h][c][1] = ls32(row + 8 * t + 4);
          }
          sc[h][c] = e4m3x2_f16x2(ls8(row + D / 2 + C * t + c) * 0x101u);
        }
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t k0[4], k1[4];
          e2m1x8_h2(w[0][c][x], k0);
          e2m1x8_h2(w[1][c][x], k1);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a[4] = {
                hmul2(k0[2 * i], sc[0][c]), hmul2(k1[2 * i], sc[1][c]),
                hmul2(k0[2 * i + 1], sc[0][c]), hmul2(k1[2 * i + 1], sc[1][c])};
            step(4 * c + 2 * x + i, a);
          }
        }
    }
    if constexpr (NT == 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][e] += odd[e];
    }
  }

  // O^T += V^T P^T of a page; P in kTerms terms.
  __device__ __forceinline__ void values(uint32_t vp,
                                         const uint32_t (&pb)[kTerms][NT][2],
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
    auto step = [&](int i, const uint32_t (&a)[4]) {
#pragma unroll
      for (int x = 0; x < kTerms; ++x)
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16<DT>(o[i][n], a, pb[x][n][0], pb[x][n][1]);
    };
    if constexpr (DT == SVP_BF16) {
      const int r = (lane >> 4) * 8 + (lane & 7), c = (lane >> 3) & 1;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        uint32_t a[4];
        ldsm4_t(vp + piece<ROWB>(r, 2 * i + c), a);
        step(i, a);
      }
    } else if constexpr (DT == SVP_FP8_E4M3) {
      // a 16-bit element is two neighbouring dimensions of a key: the rows of
      // the two halves of a tile
      const int r = ((lane >> 3) & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
      for (int i = 0; i < MT / 2; ++i) {
        uint32_t v[4];
        ldsm4_t(vp + piece<ROWB>(r, 2 * i + c), v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t lo = __byte_perm(v[2 * x], 0, 0x3120);
          const uint32_t hi = __byte_perm(v[2 * x + 1], 0, 0x3120);
          const uint32_t a[4] = {e4m3x2_f16x2(lo), e4m3x2_f16x2(lo >> 16),
                                 e4m3x2_f16x2(hi), e4m3x2_f16x2(hi >> 16)};
          step(2 * i + x, a);
        }
      }
    } else {
      // keys 4 t .. 4 t + 3, dimensions (D / 8) g on
      constexpr int C = D / 64;
      constexpr uint32_t M = 0x0f0f0f0fu;
      uint32_t w[4][C], sc[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t row = vp + (4 * t + k) * ROWB;
        if constexpr (D == 128) {
          const uint2 v = ls64(row + 8 * g);
          w[k][0] = v.x;
          w[k][C - 1] = v.y;
        } else {
          w[k][0] = ls32(row + 4 * g);
        }
        sc[k] = ls8(row + D / 2 + (D / 8) * g / kFp4Group);
      }
      const uint32_t s01 = e4m3x2_f16x2(__byte_perm(sc[0], sc[1], 0x0040));
      const uint32_t s23 = e4m3x2_f16x2(__byte_perm(sc[2], sc[3], 0x0040));
#pragma unroll
      for (int x = 0; x < C; ++x) {
        uint32_t e01[4], d01[4], e23[4], d23[4];
        e2m1x8_h2((w[0][x] & M) | ((w[1][x] << 4) & ~M), e01);
        e2m1x8_h2(((w[0][x] >> 4) & M) | (w[1][x] & ~M), d01);
        e2m1x8_h2((w[2][x] & M) | ((w[3][x] << 4) & ~M), e23);
        e2m1x8_h2(((w[2][x] >> 4) & M) | (w[3][x] & ~M), d23);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t a[4] = {hmul2(e01[i], s01), hmul2(d01[i], s01),
                                 hmul2(e23[i], s23), hmul2(d23[i], s23)};
          step(4 * x + i, a);
        }
      }
    }
  }

  // The pages that stand at `at` in the ring (K, then V), first positions j0; one
  // at kNoPage has no visible key.
  template <int NP>
  __device__ __forceinline__ void pages(const SparseParams &p, const uint32_t (&at)[NP],
                                        const int (&j0)[NP], int b, int L, int row0,
                                        unsigned char *shared, int, int lane) {
    const int g = lane >> 2, t = lane & 3;
    float s[NP][NT][4];
#pragma unroll
    for (int x = 0; x < NP; ++x) scores(at[x], s[x], shared, lane);
    // in the log2 domain, masked; value 2 h + e: key of half h, row 2 t + e
#pragma unroll
    for (int x = 0; x < NP; ++x) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[x][n][e] *= factor[n][e & 1];
      if (j0[x] + kBlockSize - 1 > t_all) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const RowMask m = row_mask(p, b, L, row0 + 8 * n + 2 * t + e);
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (!m.sees(j0[x] + key(g, h))) s[x][n][2 * h + e] = -INFINITY;
          }
      }
    }
    bool over = false;
    float top[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[n][e] = fmaxf(s[0][n][e], s[0][n][2 + e]);
#pragma unroll
        for (int x = 1; x < NP; ++x)
          top[n][e] = fmaxf(top[n][e], fmaxf(s[x][n][e], s[x][n][2 + e]));
        over |= top[n][e] > ref[n][e] + (kSlack - kOff);
      }
    if (__any_sync(kFull, over)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int off = 4; off < 32; off <<= 1)
            top[n][e] = fmaxf(top[n][e], __shfl_xor_sync(kFull, top[n][e], off));
          if (top[n][e] > ref[n][e]) {
            const float f = ex2(ref[n][e] - top[n][e]);
            ref[n][e] = top[n][e];
            sum[n][e] *= f;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[i][n][e] *= f;
              o[i][n][2 + e] *= f;
            }
          }
        }
    }
#pragma unroll
    for (int x = 0; x < NP; ++x) {
      uint32_t pb[kTerms][NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[x][n][e] = ex2(s[x][n][e] - ref[n][e & 1] + kOff);
          sum[n][e & 1] += s[x][n][e];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float p0 = s[x][n][2 * h], p1 = s[x][n][2 * h + 1];
          const uint32_t w = pack2<DT>(p0, p1);
          pb[0][n][h] = transpose8(w);
          if constexpr (kTerms == 2)  // what the first term leaves
            pb[1][n][h] = transpose8(
                pack2<DT>(p0 - __uint_as_float(w << 16),
                          p1 - __uint_as_float(w & 0xffff0000u)));
        }
      }
      values(at[x] + S::PAGE, pb, lane);
    }
  }

  // The warp's rows to shared memory: values, then reference and sum.
  __device__ __forceinline__ void finish(float *res, float2 *stat, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int RR = S::RES_ROW / 4;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1)
          sum[n][e] += __shfl_xor_sync(kFull, sum[n][e], off);
        const int row = 8 * n + 2 * t + e;
        float *to = res + row * RR;
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) to[dim(i, h, g)] = o[i][n][2 * h + e];
        if (g == 0) stat[row] = make_float2(ref[n][e], sum[n][e]);
      }
  }
};

// A warp's state over an fp32 cache: R rows.  Scores: lane = key + 16 half of
// the dimensions; values: a lane owns 4 dimensions (of half the keys for D 64).
template <int D, int R>
struct WarpF32 {
  static constexpr int RPW = R;
  using S = SpShape<SVP_F32, D, R == 4 ? 0 : 1>;
  static constexpr int QROW = S::QROW, ROWB = S::ROWB;
  float4 o[RPW];
  float ref[RPW], sum[RPW];
  float factor;
  int t_all;

  // Byte of dimension 4 c of a query row: the second half lies 16 bytes on,
  // in other banks than the first.
  static __device__ __forceinline__ int q_at(int c) {
    return 16 * c + (c >= D / 8 ? 16 : 0);
  }

  // Before a barrier: the unit's query rows; behind them the warps' weights.
  __device__ __forceinline__ void load_query(const SparseParams &p, int b, int head,
                                             int row0, unsigned char *shared, int warp,
                                             int lane) {
    for (int x = warp * 32 + lane; x < RPW * (D / 4); x += S::THREADS) {
      const int r = x / (D / 4), c = x % (D / 4), row = row0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.rows)
        v = reinterpret_cast<const float4 *>(
            static_cast<const float *>(p.q) +
            (((size_t)b * p.q_len + row / p.group) * p.num_q_heads +
             (size_t)head * p.group + row % p.group) * D)[c];
      *reinterpret_cast<float4 *>(shared + r * QROW + q_at(c)) = v;
    }
  }

  __device__ __forceinline__ void start(const SparseParams &p, int L, int row0,
                                        const unsigned char *, int) {
    factor = p.qscale;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      ref[r] = kSpNoRef;
      sum[r] = 0.f;
    }
    const int base = L - p.q_len;
    t_all = p.tree_mask ? base - 1 : base + min(row0, p.rows - 1) / p.group;
  }

  template <int NP>
  __device__ __forceinline__ void pages(const SparseParams &p, const uint32_t (&at)[NP],
                                        const int (&first)[NP], int b, int L, int row0,
                                        unsigned char *shared, int warp, int lane) {
    static_assert(NP == 1, "");
    const int j0 = first[0];
    const uint32_t qs = smem_u32(shared), kp = at[0], vp = kp + S::PAGE;
    float *const ps = reinterpret_cast<float *>(shared + RPW * QROW) +
                      warp * RPW * kBlockSize;
    const int k = lane & 15, half = lane >> 4;
    float s[RPW];
#pragma unroll
    for (int r = 0; r < RPW; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const int c = half * (D / 8) + i;
      const float4 kv = as_f4(ls128(kp + piece<ROWB>(k, c)));
#pragma unroll
      for (int r = 0; r < RPW; ++r) {
        const float4 qv = as_f4(ls128(qs + r * QROW + q_at(c)));
        s[r] = fmaf(qv.x, kv.x, s[r]);
        s[r] = fmaf(qv.y, kv.y, s[r]);
        s[r] = fmaf(qv.z, kv.z, s[r]);
        s[r] = fmaf(qv.w, kv.w, s[r]);
      }
    }
    bool over = false;
    const bool check = j0 + kBlockSize - 1 > t_all;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      s[r] = (s[r] + __shfl_xor_sync(kFull, s[r], 16)) * factor;
      if (check && !row_mask(p, b, L, row0 + r).sees(j0 + k)) s[r] = -INFINITY;
      over |= s[r] > ref[r] + 8.f;
    }
    if (__any_sync(kFull, over)) {
#pragma unroll
      for (int r = 0; r < RPW; ++r) {
        float top = s[r];
#pragma unroll
        for (int off = 1; off < 16; off <<= 1)
          top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
        if (top > ref[r]) {
          const float f = ex2(ref[r] - top);
          ref[r] = top;
          sum[r] *= f;
          o[r].x *= f;
          o[r].y *= f;
          o[r].z *= f;
          o[r].w *= f;
        }
      }
    }
    __syncwarp();  // the previous page's weights have been read
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      const float w = ex2(s[r] - ref[r]);
      sum[r] += w;  // in both halves
      if (half == 0) ps[r * kBlockSize + k] = w;
    }
    __syncwarp();
    const uint32_t pw = smem_u32(ps);
    constexpr int SETS = D == 128 ? 4 : 2;  // of four keys for this lane
    const int c = D == 128 ? lane : k;
#pragma unroll
    for (int x = 0; x < SETS; ++x) {
      const int k0 = 4 * (x + (D == 128 ? 0 : 2 * half));
      float4 v[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) v[y] = as_f4(ls128(vp + piece<ROWB>(k0 + y, c)));
#pragma unroll
      for (int r = 0; r < RPW; ++r) {
        const float4 w = as_f4(ls128(pw + (r * kBlockSize + k0) * 4));
        const float ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          o[r].x = fmaf(ww[y], v[y].x, o[r].x);
          o[r].y = fmaf(ww[y], v[y].y, o[r].y);
          o[r].z = fmaf(ww[y], v[y].z, o[r].z);
          o[r].w = fmaf(ww[y], v[y].w, o[r].w);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(float *res, float2 *stat, int lane) {
    constexpr int RR = S::RES_ROW / 4;
    const int c = D == 128 ? lane : lane & 15;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
#pragma unroll
      for (int off = 1; off < 16; off <<= 1)
        sum[r] += __shfl_xor_sync(kFull, sum[r], off);
      float4 v = o[r];
      if constexpr (D == 64) {
        v.x += __shfl_xor_sync(kFull, v.x, 16);
        v.y += __shfl_xor_sync(kFull, v.y, 16);
        v.z += __shfl_xor_sync(kFull, v.z, 16);
        v.w += __shfl_xor_sync(kFull, v.w, 16);
      }
      if (lane < D / 4) *reinterpret_cast<float4 *>(res + r * RR + 4 * c) = v;
      if (lane == 0) stat[r] = make_float2(ref[r], sum[r]);
    }
  }
};

template <int DT, int D, int NT>
struct WarpOf {
  using T = WarpMma<DT, D, NT>;
};
template <int D, int NT>
struct WarpOf<SVP_F32, D, NT> {
  using T = WarpF32<D, NT == 0 ? 4 : 8>;
};

template <int DT, int D, int NT>
__global__ void __launch_bounds__(SpShape<DT, D, NT>::THREADS, SpShape<DT, D, NT>::PER_SM)
    sparse_attention_kernel(const SparseParams p) {
  using S = SpShape<DT, D, NT>;
  constexpr int RB = S::ROWS, STAGES = S::STAGES, W = S::WARPS, T = S::THREADS;
  extern __shared__ __align__(128) unsigned char smem[];
  int2 *const list = reinterpret_cast<int2 *>(smem + S::RING);
  int *const counts = reinterpret_cast<int *>(smem + S::RING + S::LIST);
  unsigned char *const shared = smem + S::RING + S::LIST + 64;
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned unit = blockIdx.x / (unsigned)nc;
  const unsigned bh = unit / (unsigned)p.n_rb;
  const int rb = (int)(unit - bh * (unsigned)p.n_rb);
  const int b = (int)(bh / (unsigned)p.num_kv_heads);
  const int head = (int)(bh - (unsigned)b * (unsigned)p.num_kv_heads);
  pdl_wait();
  pdl_launch_dependents();
  const int32_t *const entries = p.pages + (size_t)bh * p.n_select;
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  const int lo = (int)((long long)p.n_select * rank / nc);
  const int hi = (int)((long long)p.n_select * (rank + 1) / nc);
  // entries of the list that this thread looks up in a round
  constexpr int PER = kListCap / T;
  int page[PER];
  auto look = [&](int at) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = at + i * T + tid;
      page[i] = x < hi ? entries[x] : -1;
    }
  };
  look(lo);
  const int L = p.seq_lens[b];
  if (L < p.q_len || L > (long long)p.max_blocks * kBlockSize) {
    if (tid == 0) raise_sparse(SVP_DEV_BAD_SEQ_LEN);
    return;  // the whole cluster
  }
  const int n_pages = (int)(((long long)L + kBlockSize - 1) / kBlockSize);

  typename WarpOf<DT, D, NT>::T st;
  const int row0 = rb * RB;
  const uint32_t ring = smem_u32(smem) + warp * S::WARP;

  for (int at = lo; at < hi || at == lo; at += kListCap) {
    // the listed pages of this round, holes left out
    int phys[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      phys[i] = -1;
      if (page[i] >= n_pages) raise_sparse(SVP_DEV_BAD_BLOCK_ID);
      if (page[i] >= 0 && page[i] < n_pages) phys[i] = table[page[i]];
    }
    if (at == lo) st.load_query(p, b, head, row0, shared, warp, lane);
    else __syncthreads();  // the list of the round before is read
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const bool listed = page[i] >= 0 && page[i] < n_pages;
      if (listed && (phys[i] < 0 || phys[i] >= p.num_blocks)) {
        raise_sparse(SVP_DEV_BAD_BLOCK_ID);
        phys[i] = -1;
      }
      const unsigned m = __ballot_sync(kFull, phys[i] >= 0);
      if (lane == 0) counts[i * W + warp] = __popc(m);
    }
    __syncthreads();
    if (at == lo) st.start(p, L, row0, shared, lane);
    int count = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const unsigned m = __ballot_sync(kFull, phys[i] >= 0);
#pragma unroll
      for (int w = 0; w < W; ++w) {
        if (w == warp && phys[i] >= 0)
          list[count + __popc(m & ((1u << lane) - 1u))] =
              make_int2(phys[i], page[i] * kBlockSize);
        count += counts[i * W + w];
      }
    }
    if (at + kListCap < hi) look(at + kListCap);
    __syncthreads();
    // this warp's pages: every W-th
    const int n_mine = (count - warp + W - 1) / W;
    constexpr int NP = S::AT_ONCE, AHEAD = STAGES - NP;  // on their way at a time
    static_assert(STAGES % NP == 0, "a step's stages lie side by side");
    auto load = [&](int i) {  // pages i .. i + NP - 1; zeros for one that is not there
      if (i < n_mine) {
#pragma unroll
        for (int x = 0; x < NP; ++x)
          load_page<DT, D>(p, ring + (i + x) % STAGES * 2 * S::PAGE,
                           i + x < n_mine ? list[warp + (i + x) * W]
                                          : make_int2(0, kNoPage),
                           head, L, lane);
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < AHEAD; i += NP) load(i);
    for (int i = 0; i < n_mine; i += NP) {
      cp_wait<AHEAD / NP - 1>();
      __syncwarp();  // the pages are there, and the step before has been read
      load(i + AHEAD);
      uint32_t where[NP];
      int j0[NP];
#pragma unroll
      for (int x = 0; x < NP; ++x) {
        where[x] = ring + (i + x) % STAGES * 2 * S::PAGE;
        j0[x] = i + x < n_mine ? list[warp + (i + x) * W].y : kNoPage;
      }
      st.template pages<NP>(p, where, j0, b, L, row0, shared, warp, lane);
    }
    cp_wait<0>();
  }

  // ---- the warps' results meet, then the CTAs' ----
  __syncthreads();  // the rings are free
  constexpr int RR = S::RES_ROW / 4;
  float *const res = reinterpret_cast<float *>(smem);
  float2 *const stat = reinterpret_cast<float2 *>(res + W * RB * RR);
  float2 *const both = reinterpret_cast<float2 *>(shared);  // (the queries are used)
  st.finish(res + warp * RB * RR, stat + warp * RB, lane);
  __syncthreads();
  const int rows = min(RB, p.rows - row0);
  auto put = [&](int r, int c, float4 v, float top, float total) {
    // a row that sees nothing: zeros, and a log-sum-exp of -inf
    const float inv = total == 0.f ? 0.f : p.v_scale / total;
    const int row = row0 + r;
    const size_t to = ((size_t)b * p.q_len + row / p.group) * p.num_q_heads +
                      (size_t)head * p.group + row % p.group;
    if constexpr (DT == SVP_F32) {
      reinterpret_cast<float4 *>(static_cast<float *>(p.out) + to * D)[c] =
          make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    } else {
      reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + to * D)[c] =
          make_uint2(pack2<SVP_BF16>(v.x * inv, v.y * inv),
                     pack2<SVP_BF16>(v.z * inv, v.w * inv));
    }
    if (c == 0) {
      constexpr float off = DT == SVP_F32 || DT == SVP_BF16 ? 0.f : 6.f;
      p.lse[to] = total == 0.f ? -INFINITY : (top - off + log2f(total)) * kLn2;
    }
  };
  for (int x = tid; x < rows * (D / 4); x += T) {
    const int r = x / (D / 4), c = x % (D / 4);
    float2 f[W];
    float top = kSpNoRef, total = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = stat[w * RB + r];
      top = fmaxf(top, f[w].x);
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float s = ex2(f[w].x - top);
      const float4 y = *reinterpret_cast<const float4 *>(res + (w * RB + r) * RR + 4 * c);
      total = fmaf(f[w].y, s, total);
      v.x = fmaf(y.x, s, v.x);
      v.y = fmaf(y.y, s, v.y);
      v.z = fmaf(y.z, s, v.z);
      v.w = fmaf(y.w, s, v.w);
    }
    if (nc == 1) {
      put(r, c, v, top, total);
    } else {  // in the place of the first warp's, which no one else reads
      *reinterpret_cast<float4 *>(res + r * RR + 4 * c) = v;
      if (c == 0) both[r] = make_float2(top, total);
    }
  }
  if (nc == 1) return;
  cluster.sync();
  for (int x = rank * T + tid; x < rows * (D / 4); x += nc * T) {
    const int r = x / (D / 4), c = x % (D / 4);
    float top = kSpNoRef, total = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int k0 = 0; k0 < nc; k0 += 8) {
      float2 f[8];
      float4 y[8];
      float high = top;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        f[k] = make_float2(kSpNoRef, 0.f);
        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k0 + k < nc) {
          f[k] = cluster.map_shared_rank(both, k0 + k)[r];
          y[k] = *reinterpret_cast<const float4 *>(
              cluster.map_shared_rank(res, k0 + k) + r * RR + 4 * c);
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) high = fmaxf(high, f[k].x);
      const float was = ex2(top - high);
      total *= was;
      v = make_float4(v.x * was, v.y * was, v.z * was, v.w * was);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float s = ex2(f[k].x - high);
        total = fmaf(f[k].y, s, total);
        v.x = fmaf(y[k].x, s, v.x);
        v.y = fmaf(y[k].y, s, v.y);
        v.z = fmaf(y[k].z, s, v.z);
        v.w = fmaf(y[k].w, s, v.w);
      }
      top = high;
    }
    put(r, c, v, top, total);
  }
  cluster.sync();  // results may still be read
}

template <int DT, int D, int NT>
void sparse_config(int splits, cudaLaunchAttribute (&attr)[2], cudaLaunchConfig_t &cfg) {
  using S = SpShape<DT, D, NT>;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg = {};
  cfg.gridDim = dim3((unsigned)splits);
  cfg.blockDim = dim3(S::THREADS);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
}

// Whether the current device can place a cluster of sixteen CTAs of this kernel
// (a part or a partition with fewer SMs side by side cannot); asked once for
// each of the first devices.
template <int DT, int D, int NT>
bool sixteen_fit() {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];  // 0: not asked yet, 1: no, 2: yes
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return false;
  if (dev < kDevices) {
    const int k = known[dev].load(std::memory_order_relaxed);
    if (k) return k == 2;
  }
  auto kern = sparse_attention_kernel<DT, D, NT>;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  sparse_config<DT, D, NT>(kSpCluster, attr, cfg);
  int n = 0;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           SpShape<DT, D, NT>::SMEM) != cudaSuccess ||
      cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) !=
          cudaSuccess ||
      cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess)
    n = 0;
  (void)cudaGetLastError();  // a refused query leaves clusters of eight
  if (dev < kDevices) known[dev].store(n > 0 ? 2 : 1, std::memory_order_relaxed);
  return n > 0;
}

template <int DT, int D, int NT>
cudaError_t sparse_t(SparseParams p, int sms, cudaStream_t stream) {
  using S = SpShape<DT, D, NT>;
  static_assert(S::SMEM <= 227 * 1024, "shared memory");
  static_assert(S::PER_SM == 2 || DT == SVP_F32, "as measured");
  const int splits =
      sparse_splits((long long)p.batch * p.num_kv_heads * p.n_rb, p.n_select,
                    p.split_pages, sms, S::PER_SM, DT == SVP_F32,
                    sixteen_fit<DT, D, NT>);
  const long long grid =
      (long long)p.batch * p.num_kv_heads * p.n_rb * splits;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sparse_attention_kernel<DT, D, NT>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
  if (e == cudaSuccess && splits > 8)
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  cudaLaunchConfig_t cfg;
  sparse_config<DT, D, NT>(splits, attr, cfg);
  cfg.gridDim = dim3((unsigned)grid);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT, int D>
cudaError_t sparse_rows(SparseParams p, int sms, cudaStream_t stream) {
  // units of equal rows, as few as there can be
  constexpr int MOST = DT == SVP_F32 ? 8 : 8 * kSpTiles;
  p.n_rb = (p.rows + MOST - 1) / MOST;
  const int nt = ((p.rows + p.n_rb - 1) / p.n_rb + 7) / 8;
  const bool few = DT == SVP_F32 && p.rows <= 4;
  p.n_rb = few ? 1 : (p.rows + 8 * nt - 1) / (8 * nt);
  if constexpr (DT == SVP_F32)
    return few ? sparse_t<DT, D, 0>(p, sms, stream) : sparse_t<DT, D, 1>(p, sms, stream);
  else
    return nt == 1   ? sparse_t<DT, D, 1>(p, sms, stream)
           : nt == 2 ? sparse_t<DT, D, 2>(p, sms, stream)
           : nt == 3 ? sparse_t<DT, D, 3>(p, sms, stream)
                     : sparse_t<DT, D, 4>(p, sms, stream);
}

}  // namespace

cudaError_t launch_sparse_attention(const SparseParams &p, int dtype, int sms,
                                    cudaStream_t stream) {
  const bool d64 = p.head_dim == 64;
  switch (dtype) {
    case SVP_F32:
      return d64 ? sparse_rows<SVP_F32, 64>(p, sms, stream)
                 : sparse_rows<SVP_F32, 128>(p, sms, stream);
    case SVP_BF16:
      return d64 ? sparse_rows<SVP_BF16, 64>(p, sms, stream)
                 : sparse_rows<SVP_BF16, 128>(p, sms, stream);
    case SVP_FP8_E4M3:
      return d64 ? sparse_rows<SVP_FP8_E4M3, 64>(p, sms, stream)
                 : sparse_rows<SVP_FP8_E4M3, 128>(p, sms, stream);
    default:
      return d64 ? sparse_rows<SVP_FP4_E2M1, 64>(p, sms, stream)
                 : sparse_rows<SVP_FP4_E2M1, 128>(p, sms, stream);
  }
}

cudaError_t status_word_sparse(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_sparse);
}

}  // namespace svp
