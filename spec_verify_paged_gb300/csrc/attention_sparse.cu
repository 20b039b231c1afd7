// attention_sparse.cu -- attention over listed pages only
// (paged_sparse_attention, include/svp.h): every (sequence, kv head) has its
// own list of pages, each query row attends to the keys of those pages that
// causality or the draft tree lets it see.
//
// What bounds it: the listed K and V rows' bytes, each read once.
//
// A cluster of 1 to 8 CTAs takes a unit: a (sequence, kv head) and up to 64
// of its query rows (32 over an fp32 cache).  Its CTAs split the list; the
// results meet in distributed shared memory, so a call is one launch, without
// partials in memory.  A CTA's four warps form RG row groups (16 rows, 8 for
// fp32) times KG = 4 / RG key groups.  Four pages make a tile; tiles go
// through a ring of cp.async stages, whose 16-byte pieces are swizzled on the
// way so that the matrix operands are read without bank conflicts.  Rows of a
// page past the sequence's end are filled with zeros instead of being read.
//
//  * bf16: S = Q K^T and O = P V by mma.sync m16n8k16 with the query rows as
//    M: S's accumulators are, packed, the A operand of P V.  P is bf16: a
//    weight is off by half a bf16 step, 2^-8, as the output is; row sums are
//    fp32 and of the weights before that rounding.
//  * FP8 and 4-bit rows become fp16 operands (exact); P is fp16 at 2^6 times
//    its weight, which keeps weights down to 2^-20 normal.  q takes a
//    power-of-two scale per row (fp4.cuh).  With one row group that happens
//    between shared memory and the matrix instruction, in registers; with
//    several the four warps first expand a tile in shared memory, once for all
//    of them.
//  * fp32: CUDA cores, fp32 throughout.
//  * Softmax in the log2 domain with a lazy reference: it moves only when a
//    score exceeds it by 2^8, so the usual page costs one vote.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_sparse;

namespace {

namespace cg = cooperative_groups;

constexpr int kSpWarps = 4;
constexpr int kSpThreads = 32 * kSpWarps;
constexpr int kTilePages = 4;
static_assert(kTilePages == kSpWarps, "a warp expands a page");
constexpr int kListCap = 512;      // list entries a CTA looks up at once
constexpr int kNoPage = 0x7ffffff0; // first position of a page that is not there
constexpr float kSpNoRef = -3e38f; // below any score

__device__ __forceinline__ void raise_sparse(unsigned f) {
  atomicOr(&g_status_sparse, f);
}

template <int DT, int D>
struct SpShape {
  static constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                              : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  static constexpr int PAGE = kBlockSize * ROWB;       // one side
  static constexpr int STAGE = kTilePages * 2 * PAGE;
  static constexpr int STAGES = STAGE > 16384 ? 3 : 4;
  static constexpr int RPW = DT == SVP_F32 ? 8 : 16;   // query rows of a warp
  static constexpr int QROW = DT == SVP_F32 ? 4 * D + 32 : 0;
  static constexpr int LIST = kListCap * 8;
  // the warps' results take the ring's place at the end
  static constexpr int RES_ROW = 4 * D + 16;
  static constexpr int RES = kSpWarps * RPW * (RES_ROW + 8);
  static constexpr int RING = STAGES * STAGE > RES ? STAGES * STAGE : RES;
  static constexpr int SMEM =
      RING + LIST + 128 +
      (DT == SVP_F32 ? kSpWarps * RPW * (QROW + kBlockSize * 4) : 0);
};

// Whether a tile is expanded to fp16 in shared memory, behind everything else
// there: with several row groups, which would each convert it.
__host__ __device__ constexpr bool sp_expand(int dt, int rg) {
  return rg > 1 && (dt == SVP_FP8_E4M3 || dt == SVP_FP4_E2M1);
}
template <int DT, int D, int RG>
__host__ __device__ constexpr int sp_smem() {
  return SpShape<DT, D>::SMEM + (sp_expand(DT, RG) ? SpShape<SVP_BF16, D>::STAGE : 0);
}

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
template <int DT, int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  constexpr int ROWB = SpShape<DT, D>::ROWB;
  if constexpr (ROWB == 64)
    return r * ROWB + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * ROWB + ((c ^ (r & 7)) << 4);
}

// The tile's pages into a ring stage; pages past `count` and rows past the
// sequence's end become zeros.
template <int DT, int D>
__device__ __forceinline__ void load_tile(const SparseParams &p, uint32_t stage,
                                          const int2 *list, int tile, int count,
                                          int head, int L) {
  using S = SpShape<DT, D>;
  constexpr int PIECES = S::PAGE / 16;  // of a page's side
  constexpr int ALL = kTilePages * 2 * PIECES;
#pragma unroll
  for (int i = 0; i < (ALL + kSpThreads - 1) / kSpThreads; ++i) {
    const int x = i * kSpThreads + threadIdx.x;
    if (ALL % kSpThreads != 0 && x >= ALL) break;
    const int page = x / (2 * PIECES), side = x / PIECES % 2, y = x % PIECES;
    const int at = tile * kTilePages + page;
    const int2 e = at < count ? list[at] : make_int2(0, kNoPage);
    const char *src = static_cast<const char *>(side ? p.v_cache : p.k_cache) +
                      ((size_t)e.x * p.num_kv_heads + head) * S::PAGE + y * 16;
    uint32_t dst = stage + (page * 2 + side) * S::PAGE;
    int bytes = 16;
    if constexpr (DT == SVP_FP4_E2M1) {
      // pieces straddle the 36- or 72-byte rows
      dst += y * 16;
      const int valid = min(max(L - e.y, 0), kBlockSize) * S::ROWB - y * 16;
      bytes = min(max(valid, 0), 16);
    } else {
      constexpr int PPR = S::ROWB / 16;
      const int r = y / PPR;
      dst += piece<DT, D>(r, y % PPR);
      bytes = e.y + r < L ? 16 : 0;
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

// A warp's state over 16-bit operands: lane (g, t) holds rows g and g + 8.
template <int DT, int D, bool WIDE>  // WIDE: 16-bit elements in shared memory
struct WarpMma {
  static constexpr int KS = D / 16, NT = D / 8;
  static constexpr float kOff = DT == SVP_BF16 ? 0.f : 6.f;
  static constexpr float kSlack = DT == SVP_BF16 ? 8.f : 14.f;
  uint32_t q[KS][4];
  float o[NT][4];
  float ref[2], sum[2], factor[2];
  RowMask mask[2];
  int t_all;  // keys up to here are seen by all of the warp's rows

  __device__ __forceinline__ void start(const SparseParams &p, int b, int head,
                                        int L, int row0, unsigned char *, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    uint32_t w[2][KS][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = row0 + g + 8 * h;
      ref[h] = kSpNoRef;
      sum[h] = 0.f;
      mask[h] = row_mask(p, b, L, row);
      const bool there = row < p.rows;
      const size_t at = (((size_t)b * p.q_len + (there ? row : 0) / p.group) *
                             p.num_q_heads +
                         (size_t)head * p.group + (there ? row : 0) % p.group) * D;
      const uint16_t *src = static_cast<const uint16_t *>(p.q) + at;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        if constexpr (WIDE) {
          w[h][ks][0] = *reinterpret_cast<const uint32_t *>(src + 16 * ks + 2 * t);
          w[h][ks][1] = *reinterpret_cast<const uint32_t *>(src + 16 * ks + 2 * t + 8);
        } else {
          const uint2 v =
              *reinterpret_cast<const uint2 *>(src + (D / 4) * t + 4 * ks);
          w[h][ks][0] = v.x;
          w[h][ks][1] = v.y;
        }
        if (!there) w[h][ks][0] = w[h][ks][1] = 0u;
      }
      factor[h] = p.qscale;
      if constexpr (DT != SVP_BF16) {
        float top = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(w[h][ks][x] << 16)),
                                   fabsf(__uint_as_float(w[h][ks][x] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        const int e = q_exponent(top);
        const float up = pow2i(14 - e);
        factor[h] *= pow2i(e - 14);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            w[h][ks][x] = pack_h2(__uint_as_float(w[h][ks][x] << 16) * up,
                                  __uint_as_float(w[h][ks][x] & 0xffff0000u) * up);
      }
    }
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      q[ks][0] = w[0][ks][0];
      q[ks][1] = w[1][ks][0];
      q[ks][2] = w[0][ks][1];
      q[ks][3] = w[1][ks][1];
    }
    const int base = L - p.q_len;
    t_all = p.tree_mask ? base - 1 : base + min(row0, p.rows - 1) / p.group;
  }

  // Key of column n (0..7) of S tile j.
  static __device__ __forceinline__ int key(int j, int n) {
    return !WIDE && DT == SVP_FP4_E2M1 ? fp4_key(n, j) : 8 * j + n;
  }

  // S of a page: lane (g, t) gets rows g and g + 8, columns 2 t and 2 t + 1 of
  // two tiles of eight keys.
  __device__ __forceinline__ void scores(uint32_t kp, float (&s)[2][4], int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int ROWB = SpShape<DT, D>::ROWB;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[j][e] = 0.f;
    if constexpr (WIDE) {
      const int r = (lane >> 4) * 8 + (lane & 7), c = (lane >> 3) & 1;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        uint32_t k[4];
        ldsm4(kp + piece<SVP_BF16, D>(r, 2 * ks + c), k);
        mma16<DT>(s[0], q[ks], k[0], k[1]);
        mma16<DT>(s[1], q[ks], k[2], k[3]);
      }
    } else if constexpr (DT == SVP_FP8_E4M3) {
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 w[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
          w[j] = ls128(kp + piece<DT, D>(8 * j + g, (D / 64) * t + c));
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t x = e == 0 ? w[j].x : e == 1 ? w[j].y
                               : e == 2 ? w[j].z : w[j].w;
            mma16<DT>(s[j], q[4 * c + e], e4m3x2_f16x2(x), e4m3x2_f16x2(x >> 16));
          }
      }
    } else {
      constexpr int C = D / 64;  // scale blocks of a lane
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t row = kp + key(j, g) * ROWB;
#pragma unroll
        for (int c = 0; c < C; ++c) {
          uint32_t w[2];
          if constexpr (D == 128) {
            const uint2 v = ls64(row + 16 * t + 8 * c);
            w[0] = v.x;
            w[1] = v.y;
          } else {
            w[0] = ls32(row + 8 * t);
            w[1] = ls32(row + 8 * t + 4);
          }
          const uint32_t sc = e4m3x2_f16x2(ls8(row + D / 2 + C * t + c) * 0x101u);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t h[4];
            e2m1x8_h2(w[x], h);
            mma16<DT>(s[j], q[4 * c + 2 * x], hmul2(h[0], sc), hmul2(h[1], sc));
            mma16<DT>(s[j], q[4 * c + 2 * x + 1], hmul2(h[2], sc), hmul2(h[3], sc));
          }
        }
      }
    }
  }

  // O += P V of a page.
  __device__ __forceinline__ void values(uint32_t vp, const uint32_t (&pa)[4],
                                         int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int ROWB = SpShape<DT, D>::ROWB;
    if constexpr (WIDE) {
      const int r = ((lane >> 3) & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
      for (int i = 0; i < NT / 2; ++i) {
        uint32_t v[4];
        ldsm4_t(vp + piece<SVP_BF16, D>(r, 2 * i + c), v);
        mma16<DT>(o[2 * i], pa, v[0], v[1]);
        mma16<DT>(o[2 * i + 1], pa, v[2], v[3]);
      }
    } else if constexpr (DT == SVP_FP8_E4M3) {
      // a 16-bit element is two neighbouring dimensions of a key; tile 2 c + e
      // takes dimension 16 c + 2 n + e as column n
      const int r = ((lane >> 3) & 1) * 8 + (lane & 7), c = lane >> 4;
#pragma unroll
      for (int i = 0; i < NT / 4; ++i) {
        uint32_t v[4];
        ldsm4_t(vp + piece<DT, D>(r, 2 * i + c), v);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t lo = __byte_perm(v[2 * x], 0, 0x3120);
          const uint32_t hi = __byte_perm(v[2 * x + 1], 0, 0x3120);
          mma16<DT>(o[4 * i + 2 * x], pa, e4m3x2_f16x2(lo), e4m3x2_f16x2(hi));
          mma16<DT>(o[4 * i + 2 * x + 1], pa, e4m3x2_f16x2(lo >> 16),
                    e4m3x2_f16x2(hi >> 16));
        }
      }
    } else {
      // keys 4 t .. 4 t + 3; tile n takes dimension (D / 8) g + n as column g
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
          mma16<DT>(o[8 * x + 2 * i], pa, hmul2(e01[i], s01), hmul2(e23[i], s23));
          mma16<DT>(o[8 * x + 2 * i + 1], pa, hmul2(d01[i], s01), hmul2(d23[i], s23));
        }
      }
    }
  }

  // NP pages at `stage` (K, V, K, V, ..), their first positions j0; the products
  // of several pages are independent chains, and one vote serves them all.  A
  // page at kNoPage has no visible key.
  template <int NP>
  __device__ __forceinline__ void pages(const SparseParams &, uint32_t stage,
                                        const int (&j0)[NP], unsigned char *,
                                        int lane) {
    const int t = lane & 3;
    constexpr int PAGE = SpShape<WIDE ? SVP_BF16 : DT, D>::PAGE;
    float s[NP][2][4];
#pragma unroll
    for (int n = 0; n < NP; ++n) scores(stage + 2 * n * PAGE, s[n], lane);
    // in the log2 domain, masked; value e of tile j: row g + 8 (e / 2), column
    // 2 t + e % 2
    float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][j][e] *= factor[e >> 1];
      if (j0[n] + kBlockSize - 1 > t_all) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!mask[e >> 1].sees(j0[n] + key(j, 2 * t + (e & 1))))
              s[n][j][e] = -INFINITY;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
        top[h] = fmaxf(top[h], fmaxf(fmaxf(s[n][0][2 * h], s[n][0][2 * h + 1]),
                                     fmaxf(s[n][1][2 * h], s[n][1][2 * h + 1])));
    }
    if (__any_sync(kFull, top[0] > ref[0] + (kSlack - kOff) ||
                              top[1] > ref[1] + (kSlack - kOff))) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 1));
        top[h] = fmaxf(top[h], __shfl_xor_sync(kFull, top[h], 2));
        if (top[h] > ref[h]) {
          const float f = ex2(ref[h] - top[h]);
          ref[h] = top[h];
          sum[h] *= f;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            o[n][2 * h] *= f;
            o[n][2 * h + 1] *= f;
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NP; ++n) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[n][j][e] = ex2(s[n][j][e] - ref[e >> 1] + kOff);
          sum[e >> 1] += s[n][j][e];
        }
      const uint32_t pa[4] = {
          pack2<DT>(s[n][0][0], s[n][0][1]), pack2<DT>(s[n][0][2], s[n][0][3]),
          pack2<DT>(s[n][1][0], s[n][1][1]), pack2<DT>(s[n][1][2], s[n][1][3])};
      values(stage + (2 * n + 1) * PAGE, pa, lane);
    }
  }

  // Dimension of column n of O tile i.
  static __device__ __forceinline__ int dim(int i, int n) {
    return WIDE                 ? 8 * i + n
           : DT == SVP_FP8_E4M3 ? 16 * (i >> 1) + 2 * n + (i & 1)
                                : (D / 8) * n + i;
  }

  // The warp's rows to shared memory: values, then reference and sum.
  __device__ __forceinline__ void finish(float *res, float2 *stat, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr int RR = SpShape<DT, D>::RES_ROW / 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      sum[h] += __shfl_xor_sync(kFull, sum[h], 1);
      sum[h] += __shfl_xor_sync(kFull, sum[h], 2);
      float *to = res + (g + 8 * h) * RR;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) to[dim(i, 2 * t + e)] = o[i][2 * h + e];
      if (t == 0) stat[g + 8 * h] = make_float2(ref[h], sum[h]);
    }
  }
};

// A warp's state over an fp32 cache: 8 rows.  Scores: lane = key + 16 half of
// the dimensions; values: a lane owns 4 dimensions (of half the keys for D 64).
template <int D>
struct WarpF32 {
  static constexpr int RPW = 8;
  static constexpr int QROW = SpShape<SVP_F32, D>::QROW;
  float4 o[RPW];
  float ref[RPW], sum[RPW];
  float factor;
  int row0, t_all, L, b;

  // Byte of dimension 4 c of a query row: the second half lies 16 bytes on,
  // in other banks than the first.
  static __device__ __forceinline__ int q_at(int c) {
    return 16 * c + (c >= D / 8 ? 16 : 0);
  }

  __device__ __forceinline__ void start(const SparseParams &p, int b_, int head,
                                        int L_, int row0_, unsigned char *own,
                                        int lane) {
    b = b_;
    L = L_;
    row0 = row0_;
    factor = p.qscale;
#pragma unroll
    for (int r = 0; r < RPW; ++r) {
      o[r] = make_float4(0.f, 0.f, 0.f, 0.f);
      ref[r] = kSpNoRef;
      sum[r] = 0.f;
    }
    for (int x = lane; x < RPW * (D / 4); x += 32) {
      const int r = x / (D / 4), c = x % (D / 4), row = row0 + r;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row < p.rows)
        v = reinterpret_cast<const float4 *>(
            static_cast<const float *>(p.q) +
            (((size_t)b * p.q_len + row / p.group) * p.num_q_heads +
             (size_t)head * p.group + row % p.group) * D)[c];
      *reinterpret_cast<float4 *>(own + r * QROW + q_at(c)) = v;
    }
    __syncwarp();
    const int base = L - p.q_len;
    t_all = p.tree_mask ? base - 1 : base + min(row0, p.rows - 1) / p.group;
  }

  template <int NP>
  __device__ __forceinline__ void pages(const SparseParams &p, uint32_t stage,
                                        const int (&first)[NP], unsigned char *own,
                                        int lane) {
    constexpr int PAGE = SpShape<SVP_F32, D>::PAGE;
#pragma unroll 1
    for (int n = 0; n < NP; ++n)
      if (first[n] < kNoPage)
        page(p, stage + 2 * n * PAGE, stage + (2 * n + 1) * PAGE, first[n], own, lane);
  }

  __device__ __forceinline__ void page(const SparseParams &p, uint32_t kp,
                                       uint32_t vp, int j0, unsigned char *own,
                                       int lane) {
    const uint32_t qs = smem_u32(own);
    float *const ps = reinterpret_cast<float *>(own + RPW * QROW);
    const int k = lane & 15, half = lane >> 4;
    float s[RPW];
#pragma unroll
    for (int r = 0; r < RPW; ++r) s[r] = 0.f;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const int c = half * (D / 8) + i;
      const float4 kv = as_f4(ls128(kp + piece<SVP_F32, D>(k, c)));
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
      for (int y = 0; y < 4; ++y) v[y] = as_f4(ls128(vp + piece<SVP_F32, D>(k0 + y, c)));
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
    constexpr int RR = SpShape<SVP_F32, D>::RES_ROW / 4;
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

template <int DT, int D, bool WIDE>
struct WarpOf {
  using T = WarpMma<DT, D, WIDE>;
};
template <int D>
struct WarpOf<SVP_F32, D, false> {
  using T = WarpF32<D>;
};

// A page's side of FP8 or 4-bit rows as fp16, by a warp.
template <int DT, int D>
__device__ __forceinline__ void expand_side(uint32_t from, uint32_t to, int lane) {
  constexpr int BLOCKS = D / 16;  // of 16 elements, of a row
#pragma unroll
  for (int i = 0; i < kBlockSize * BLOCKS / 32; ++i) {
    const int y = i * 32 + lane, r = y / BLOCKS, c = y % BLOCKS;
    uint32_t h[8];
    if constexpr (DT == SVP_FP8_E4M3) {
      const uint4 w = ls128(from + piece<DT, D>(r, c));
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        h[2 * e] = e4m3x2_f16x2(x[e]);
        h[2 * e + 1] = e4m3x2_f16x2(x[e] >> 16);
      }
    } else {
      const uint32_t row = from + r * fp4_row_bytes(D);
      uint32_t w[2], v[4];
      if constexpr (D == 128) {
        const uint2 u = ls64(row + 8 * c);
        w[0] = u.x;
        w[1] = u.y;
      } else {
        w[0] = ls32(row + 8 * c);
        w[1] = ls32(row + 8 * c + 4);
      }
      const uint32_t sc = e4m3x2_f16x2(ls8(row + D / 2 + c) * 0x101u);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        e2m1x8_h2(w[x], v);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[4 * x + e] = hmul2(v[e], sc);
      }
    }
#pragma unroll
    for (int x = 0; x < 2; ++x)
      asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                       to + piece<SVP_BF16, D>(r, 2 * c + x)),
                   "r"(h[4 * x]), "r"(h[4 * x + 1]), "r"(h[4 * x + 2]),
                   "r"(h[4 * x + 3])
                   : "memory");
  }
}

template <int DT, int D, int RG>
__global__ void __launch_bounds__(kSpThreads)
    sparse_attention_kernel(const SparseParams p) {
  using S = SpShape<DT, D>;
  constexpr int KG = kSpWarps / RG, RPW = S::RPW, RB = RG * RPW;
  constexpr bool EXPAND = sp_expand(DT, RG);
  using W16 = SpShape<SVP_BF16, D>;
  extern __shared__ __align__(128) unsigned char smem[];
  int2 *const list = reinterpret_cast<int2 *>(smem + S::RING);
  int *const counts = reinterpret_cast<int *>(smem + S::RING + S::LIST);
  cg::cluster_group cluster = cg::this_cluster();
  const int nc = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rg = warp / KG, kg = warp % KG;
  unsigned char *const own =
      smem + S::RING + S::LIST + 64 + warp * RPW * (S::QROW + kBlockSize * 4);
  const unsigned unit = blockIdx.x / (unsigned)nc;
  const unsigned bh = unit / (unsigned)p.n_rb;
  const int rb = (int)(unit - bh * (unsigned)p.n_rb);
  const int b = (int)(bh / (unsigned)p.num_kv_heads);
  const int head = (int)(bh - (unsigned)b * (unsigned)p.num_kv_heads);
  pdl_wait();
  pdl_launch_dependents();
  const int L = p.seq_lens[b];
  if (L < p.q_len || L > (long long)p.max_blocks * kBlockSize) {
    if (tid == 0) raise_sparse(SVP_DEV_BAD_SEQ_LEN);
    return;  // the whole cluster
  }
  const int32_t *const entries = p.pages + (size_t)bh * p.n_select;
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  const int lo = (int)((long long)p.n_select * rank / nc);
  const int hi = (int)((long long)p.n_select * (rank + 1) / nc);
  const int n_pages = (int)(((long long)L + kBlockSize - 1) / kBlockSize);

  typename WarpOf<DT, D, EXPAND || DT == SVP_BF16>::T st;
  st.start(p, b, head, L, rb * RB + rg * RPW, own, lane);
  const bool idle = rb * RB + rg * RPW >= p.rows;  // a row group without rows

  for (int at = lo; at < hi; at += kListCap) {
    // the listed pages of this round, holes left out
    constexpr int PER = kListCap / kSpThreads;
    int page[PER], phys[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int x = at + i * kSpThreads + tid;
      page[i] = x < hi ? entries[x] : -1;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      phys[i] = -1;
      if (page[i] >= n_pages) raise_sparse(SVP_DEV_BAD_BLOCK_ID);
      if (page[i] >= 0 && page[i] < n_pages) {
        phys[i] = table[page[i]];
        if (phys[i] < 0 || phys[i] >= p.num_blocks) {
          raise_sparse(SVP_DEV_BAD_BLOCK_ID);
          phys[i] = -1;
        }
      }
    }
    int count = 0;
    __syncthreads();  // the list and the ring of the round before are read
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const unsigned m = __ballot_sync(kFull, phys[i] >= 0);
      if (lane == 0) counts[i * kSpWarps + warp] = __popc(m);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const unsigned m = __ballot_sync(kFull, phys[i] >= 0);
#pragma unroll
      for (int w = 0; w < kSpWarps; ++w) {
        if (w == warp && phys[i] >= 0)
          list[count + __popc(m & ((1u << lane) - 1u))] =
              make_int2(phys[i], page[i] * kBlockSize);
        count += counts[i * kSpWarps + w];
      }
    }
    __syncthreads();
    const int tiles = (count + kTilePages - 1) / kTilePages;
    const uint32_t ring = smem_u32(smem);
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) {
      if (s < tiles) load_tile<DT, D>(p, ring + s * S::STAGE, list, s, count, head, L);
      cp_commit();
    }
    for (int tile = 0; tile < tiles; ++tile) {
      cp_wait<S::STAGES - 2>();
      __syncthreads();  // the tile is there, and the one before has been read
      const int ahead = tile + S::STAGES - 1;
      if (ahead < tiles)
        load_tile<DT, D>(p, ring + ahead % S::STAGES * S::STAGE, list, ahead, count,
                         head, L);
      cp_commit();
      uint32_t stage = ring + tile % S::STAGES * S::STAGE;
      if constexpr (EXPAND) {
        const uint32_t wide = ring + S::SMEM;
#pragma unroll
        for (int side = 0; side < 2; ++side)
          expand_side<DT, D>(stage + (2 * warp + side) * S::PAGE,
                             wide + (2 * warp + side) * W16::PAGE, lane);
        __syncthreads();
        stage = wide;
      }
      constexpr int PAGE = EXPAND ? W16::PAGE : S::PAGE;
      // a warp's pages of the tile lie side by side
      constexpr int MINE = kTilePages / KG, NP = MINE < 2 ? MINE : 2;
#pragma unroll 1
      for (int x = kg * MINE; x < (kg + 1) * MINE; x += NP) {
        const int e = tile * kTilePages + x;
        if (e >= count || idle) break;
        int j0[NP];
#pragma unroll
        for (int n = 0; n < NP; ++n) j0[n] = e + n < count ? list[e + n].y : kNoPage;
        st.template pages<NP>(p, stage + 2 * x * PAGE, j0, own, lane);
      }
    }
    cp_wait<0>();
  }

  // ---- the warps' results meet ----
  __syncthreads();  // the ring is free
  constexpr int RR = S::RES_ROW / 4;
  float *const res = reinterpret_cast<float *>(smem);
  float2 *const stat = reinterpret_cast<float2 *>(res + kSpWarps * RPW * RR);
  st.finish(res + warp * RPW * RR, stat + warp * RPW, lane);
  if (nc > 1) cluster.sync(); else __syncthreads();
  const int rows = min(RB, p.rows - rb * RB);
  for (int x = rank * kSpThreads + tid; x < rows * (D / 4); x += nc * kSpThreads) {
    const int r = x / (D / 4), c = x % (D / 4);
    const int w0 = r / RPW * KG, rr = r % RPW;
    float top = kSpNoRef;
    for (int k = 0; k < nc; ++k) {
      const float2 *from = nc > 1 ? cluster.map_shared_rank(stat, k) : stat;
#pragma unroll
      for (int w = 0; w < KG; ++w) top = fmaxf(top, from[(w0 + w) * RPW + rr].x);
    }
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    for (int k = 0; k < nc; ++k) {
      const float2 *from = nc > 1 ? cluster.map_shared_rank(stat, k) : stat;
      const float *val = nc > 1 ? cluster.map_shared_rank(res, k) : res;
#pragma unroll
      for (int w = 0; w < KG; ++w) {
        const float2 f = from[(w0 + w) * RPW + rr];
        const float s = ex2(f.x - top);
        const float4 y =
            *reinterpret_cast<const float4 *>(val + ((w0 + w) * RPW + rr) * RR + 4 * c);
        total = fmaf(f.y, s, total);
        v.x = fmaf(y.x, s, v.x);
        v.y = fmaf(y.y, s, v.y);
        v.z = fmaf(y.z, s, v.z);
        v.w = fmaf(y.w, s, v.w);
      }
    }
    // a row that sees nothing: zeros, and a log-sum-exp of -inf
    const float inv = total == 0.f ? 0.f : p.v_scale / total;
    const int row = rb * RB + r;
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
  }
  if (nc > 1) cluster.sync();  // results may still be read
}

template <int DT, int D, int RG>
cudaError_t sparse_t(SparseParams p, int splits, cudaStream_t stream) {
  using S = SpShape<DT, D>;
  p.n_rb = (p.rows + RG * S::RPW - 1) / (RG * S::RPW);
  const long long grid =
      (long long)p.batch * p.num_kv_heads * p.n_rb * splits;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  auto kern = sparse_attention_kernel<DT, D, RG>;
  cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, sp_smem<DT, D, RG>());
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(kSpThreads);
  cfg.dynamicSmemBytes = sp_smem<DT, D, RG>();
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

template <int DT, int D>
cudaError_t sparse_rows(const SparseParams &p, int sms, cudaStream_t stream) {
  constexpr int RPW = SpShape<DT, D>::RPW;
  const int rg = p.rows <= RPW ? 1 : p.rows <= 2 * RPW ? 2 : 4;
  const long long units = (long long)p.batch * p.num_kv_heads *
                          ((p.rows + rg * RPW - 1) / (rg * RPW));
  // split a list while the CTAs all find room and keep two tiles each, or to
  // the caller's pages per CTA
  const long long least = p.split_pages > 0 ? p.split_pages : 2 * kTilePages;
  int splits = 1;
  while (splits < 8 && 2LL * splits * least <= p.n_select &&
         (p.split_pages > 0 || units * splits * 2 <= 2LL * sms))
    splits *= 2;
  return rg == 1   ? sparse_t<DT, D, 1>(p, splits, stream)
         : rg == 2 ? sparse_t<DT, D, 2>(p, splits, stream)
                   : sparse_t<DT, D, 4>(p, splits, stream);
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

cudaError_t read_status_sparse(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_sparse, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_sparse, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
