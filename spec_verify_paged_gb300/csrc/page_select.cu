// page_select.cu -- which pages of a long context attention needs to read:
// bounds of the keys of every page (kv_page_bounds), what a query's products
// with a page's keys can be at most (paged_page_scores) and the choice of
// pages by such a score (paged_select_pages).  include/svp.h has the calls.
//
// For a page with keys K_j and a query row q, every product is
//   <q, K_j> = sum_d q_d K_j,d <= sum_d max(q_d, 0) hi_d + min(q_d, 0) lo_d
// with lo and hi the elementwise smallest and largest key: 4 D bytes of
// bounds (bf16) stand for 16 keys, an eighth of what bf16 keys take.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_pages;

namespace {

__device__ __forceinline__ void raise_pages(unsigned f) {
  atomicOr(&g_status_pages, f);
}

// ---- bounds ----
// A warp takes one head's page: a lane holds V consecutive elements (16 bytes
// of a row; 8 bytes of codes of a 4-bit row), so one access of the warp covers
// 32 V / D rows and all rows are in flight at once.  The lanes that hold the
// same elements of other rows are then joined by shuffles.
// Bound by the keys' bytes in 16 and 32 bits, by their conversion in fewer.
// Whole prompts of 8 heads, D = 128, of the bytes at the copy rate: bf16 0.93,
// fp32 0.96, FP8 0.85 (420 MB: 72.5 us; 0.70 by way of fp16 values), 4-bit 0.57.
// The newest row of 32 sequences of 32 heads: 2.4 us a call.
constexpr int kBoundWarps = 8;

template <int DT>
struct BoundType;
// packed pairs with their NaN-propagating extremes; ident: nothing seen yet
struct PairBf16 {
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static constexpr uint32_t kPosInf = 0x7f807f80u, kNegInf = 0xff80ff80u;
  // as a bf16 pair
  static __device__ __forceinline__ uint32_t out(uint32_t a, bool) { return a; }
};
struct PairF16 {
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  static constexpr uint32_t kPosInf = 0x7c007c00u, kNegInf = 0xfc00fc00u;
  // codes and code * scale have at most 6 significant bits: exact in bf16
  static __device__ __forceinline__ uint32_t out(uint32_t a, bool) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
};
// E4M3 codes as unsigned numbers of the same order (the sign bit flipped, all
// bits of a negative code), each in the high byte of a 16-bit half, where the
// byte below it only breaks ties.  So a word of four codes makes two registers
// by three instructions and no conversion, and three-operand minima and maxima
// take two rows at a time.  A NaN is the largest or the smallest.
struct PairE4m3 {
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    return __vminu2(a, b);
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    return __vmaxu2(a, b);
  }
  static constexpr uint32_t kPosInf = 0xffffffffu, kNegInf = 0u;
  // codes 0 and 2 of a word, codes 1 and 3
  static __device__ __forceinline__ void split(uint32_t w, uint32_t &even,
                                               uint32_t &odd) {
    uint32_t sign;  // of each byte, in all of its bits
    asm("prmt.b32 %0, %1, 0, 0xba98;" : "=r"(sign) : "r"(w));
    odd = w ^ (sign | 0x80808080u);
    even = odd << 8;
  }
  // the bounds' codes in the high bytes as bf16, low half and high half
  static __device__ __forceinline__ uint32_t out(uint32_t l, uint32_t h, bool upper) {
    const uint32_t x = upper ? h : l;
    uint32_t sign;
    asm("prmt.b32 %0, %1, 0, 0xba98;" : "=r"(sign) : "r"(x));
    const uint32_t code = x ^ (~sign | 0x80808080u);
    const uint32_t two = e4m3x2_f16x2(__byte_perm(code, 0, 0x4431));
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&two));
    __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
    uint32_t r = *reinterpret_cast<const uint32_t *>(&v);
    // a NaN among them
    if ((h & 0xff00u) == 0xff00u || (l & 0xff00u) == 0u) r |= 0x7fffu;
    if (h >= 0xff000000u || l < 0x01000000u) r |= 0x7fff0000u;
    return r;
  }
};
struct OneF32 {
  static __device__ __forceinline__ uint32_t lo(uint32_t a, uint32_t b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;"
        : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
  static __device__ __forceinline__ uint32_t hi(uint32_t a, uint32_t b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;"
        : "=f"(r) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    return __float_as_uint(r);
  }
  static constexpr uint32_t kPosInf = 0x7f800000u, kNegInf = 0xff800000u;
};
template <> struct BoundType<SVP_BF16> { using P = PairBf16; };
template <> struct BoundType<SVP_FP8_E4M3> { using P = PairE4m3; };
template <> struct BoundType<SVP_FP4_E2M1> { using P = PairF16; };
template <> struct BoundType<SVP_F32> { using P = OneF32; };

// fp32 -> bf16 bits, away from zero where `out` says so (a lower bound is
// rounded down, an upper bound up), NaN as the quiet NaN.
__device__ __forceinline__ uint32_t bf16_outward(float x, bool up) {
  const uint32_t u = __float_as_uint(x);
  if (x != x) return 0x7fffu;
  const bool away = (u & 0xffffu) != 0 && ((u >> 31) == 0) == up;
  return (u >> 16) + (away ? 1u : 0u);
}

template <int DT, int D>
__global__ void __launch_bounds__(32 * kBoundWarps)
    page_bounds_kernel(const BoundsParams p) {
  using P = typename BoundType<DT>::P;
  constexpr int V = DT == SVP_F32 ? 4 : DT == SVP_BF16 ? 8 : 16;
  constexpr int LPR = D / V;         // lanes of a row
  constexpr int RPA = 32 / LPR;      // rows of an access
  constexpr int NA = kBlockSize / RPA;  // accesses
  constexpr int NR = DT == SVP_F32 ? 4 : V / 2;  // registers of V elements
  constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                       : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  pdl_wait();
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const int lane = threadIdx.x & 31;
  const unsigned item = blockIdx.x * kBoundWarps + (threadIdx.x >> 5);
  const unsigned shares = (unsigned)(p.num_kv_heads + p.heads - 1) / (unsigned)p.heads;
  const unsigned i = item / shares;
  const int g0 = (int)(item - i * shares) * p.heads;  // this warp's heads
  // (rows of 256 bytes and more: one, and no loop)
  const int g1 = ROWB >= 256 ? g0 + 1 : min(g0 + p.heads, p.num_kv_heads);
  const int L = p.seq_lens[b];
  if (L < 0 || L > (long long)p.max_blocks * kBlockSize) {
    if (threadIdx.x == 0) raise_pages(SVP_DEV_BAD_SEQ_LEN);
    return;
  }
  const int first = max(L - p.n_new, 0) / kBlockSize;
  const int page = first + (int)i;
  if (i >= (unsigned)p.max_pages || (long long)page * kBlockSize >= L) return;
  const int phys = p.block_table[(size_t)b * p.max_blocks + page];
  if (phys < 0 || phys >= p.num_blocks) {
    if (lane == 0) raise_pages(SVP_DEV_BAD_BLOCK_ID);
    return;
  }
  const int rows = min(L - page * kBlockSize, kBlockSize);
  const int r0 = lane / LPR, c = lane % LPR;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    const unsigned char *src =
        static_cast<const unsigned char *>(p.k_cache) +
        ((size_t)phys * p.num_kv_heads + g) * (size_t)(kBlockSize * ROWB);
    uint32_t lo[NR], hi[NR];
#pragma unroll
    for (int e = 0; e < NR; ++e) {
      lo[e] = P::kPosInf;
      hi[e] = P::kNegInf;
    }
    auto take = [&](const uint32_t (&w)[NR]) {
#pragma unroll
      for (int e = 0; e < NR; ++e) {
        lo[e] = P::lo(lo[e], w[e]);
        hi[e] = P::hi(hi[e], w[e]);
      }
    };
    if constexpr (DT == SVP_FP4_E2M1) {
      uint32_t w[NA][2], sc[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int r = min(a * RPA + r0, rows - 1);  // rows past the end: the last
        const uint32_t *row = reinterpret_cast<const uint32_t *>(src + r * ROWB);
        w[a][0] = row[2 * c];
        w[a][1] = row[2 * c + 1];
        sc[a] = src[r * ROWB + D / 2 + c];
      }
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        uint32_t v[NR], h[4];
        const uint32_t s2 = e4m3x2_f16x2(sc[a] * 0x101u);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          e2m1x8_h2(w[a][x], h);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[4 * x + e] = hmul2(h[e], s2);
        }
        take(v);
      }
    } else {
      uint4 w[NA];
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const int r = min(a * RPA + r0, rows - 1);
        w[a] = *(reinterpret_cast<const uint4 *>(src + r * ROWB) + c);
      }
      if constexpr (DT == SVP_FP8_E4M3) {
#pragma unroll
        for (int a = 0; a < NA; a += 2) {
          const uint32_t x[4] = {w[a].x, w[a].y, w[a].z, w[a].w};
          const uint32_t y[4] = {w[a + 1].x, w[a + 1].y, w[a + 1].z, w[a + 1].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t u[2], v[2];
            P::split(x[e], u[0], u[1]);
            P::split(y[e], v[0], v[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              lo[2 * e + h] = __vimin3_u16x2(lo[2 * e + h], u[h], v[h]);
              hi[2 * e + h] = __vimax3_u16x2(hi[2 * e + h], u[h], v[h]);
            }
          }
        }
      } else {
#pragma unroll
        for (int a = 0; a < NA; ++a) {
          const uint32_t x[4] = {w[a].x, w[a].y, w[a].z, w[a].w};
          take(x);
        }
      }
    }
    // Lanes that hold the same elements of other rows: in each step a lane hands
    // half of its registers to its partner and keeps the other half, so at the
    // end it has the bounds of NR / RPA (of one if there are fewer) registers.
    int base = 0;  // the first register's place among the row's
#pragma unroll
    for (int off = 16, left = NR; off >= LPR; off >>= 1) {
      const bool up = (lane & off) != 0;
      if (left > 1) {
        left /= 2;
#pragma unroll
        for (int e = 0; e < NR / 2; ++e) {
          if (e >= left) break;
          const uint32_t l = up ? lo[e] : lo[e + left], h = up ? hi[e] : hi[e + left];
          const uint32_t ml = up ? lo[e + left] : lo[e], mh = up ? hi[e + left] : hi[e];
          lo[e] = P::lo(ml, __shfl_xor_sync(kFull, l, off));
          hi[e] = P::hi(mh, __shfl_xor_sync(kFull, h, off));
        }
        base += up ? left : 0;
      } else {
        lo[0] = P::lo(lo[0], __shfl_xor_sync(kFull, lo[0], off));
        hi[0] = P::hi(hi[0], __shfl_xor_sync(kFull, hi[0], off));
      }
    }
    constexpr int LEFT = NR / RPA > 1 ? NR / RPA : 1;
    unsigned char *dst = static_cast<unsigned char *>(p.bounds) +
                         ((size_t)phys * p.num_kv_heads + g) * (4 * D) + c * (2 * V);
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint32_t *from = side ? hi : lo;
      unsigned char *to = dst + side * (2 * D);
      if constexpr (DT == SVP_F32) {
        uint16_t *const t16 = reinterpret_cast<uint16_t *>(to) + base;
        if constexpr (LEFT == 4)
          *reinterpret_cast<uint2 *>(t16) = make_uint2(
              bf16_outward(__uint_as_float(from[0]), side) |
                  (bf16_outward(__uint_as_float(from[1]), side) << 16),
              bf16_outward(__uint_as_float(from[2]), side) |
                  (bf16_outward(__uint_as_float(from[3]), side) << 16));
        else
          *reinterpret_cast<uint32_t *>(t16) =
              bf16_outward(__uint_as_float(from[0]), side) |
              (bf16_outward(__uint_as_float(from[1]), side) << 16);
      } else if constexpr (DT == SVP_FP8_E4M3) {
        // registers come in pairs: elements 0 and 2, elements 1 and 3 of a word
        uint16_t *const t16 = reinterpret_cast<uint16_t *>(to) + base / 2 * 4;
        if constexpr (LEFT == 2) {
          const uint32_t even = P::out(lo[0], hi[0], side), odd = P::out(lo[1], hi[1], side);
          *reinterpret_cast<uint2 *>(t16) = make_uint2(__byte_perm(even, odd, 0x5410),
                                                       __byte_perm(even, odd, 0x7632));
        } else {
          const uint32_t v = P::out(lo[0], hi[0], side);
          t16[base & 1] = (uint16_t)v;
          t16[(base & 1) + 2] = (uint16_t)(v >> 16);
        }
      } else {
        uint32_t *const t32 = reinterpret_cast<uint32_t *>(to) + base;
        if constexpr (LEFT >= 2)
          *reinterpret_cast<uint2 *>(t32) =
              make_uint2(P::out(from[0], side), P::out(from[1], side));
        else
          *t32 = P::out(from[0], side);
        static_assert(LEFT <= 2, "pairs at most");
      }
    }
  }
}

// ---- scores ----
// The bound is a matrix product: pages as M, query rows as N, and 2 D terms,
// hi with the positive parts of q and lo with the negative ones.  mma.sync
// m16n8k16 takes 16 pages; the order of the terms does not matter, so they
// are dealt such that lane (g, t) takes 16 consecutive bytes of pages g and
// g + 8 for two steps.  A lane copies its own pieces of a tile of 16 pages
// through shared memory, so the next tile is on its way while one is
// multiplied, and no warp waits for another; the query rows' parts are in
// shared memory as well.
// bf16 products are exact in fp32, the sums are fp32; an fp32 q is taken as
// three bf16 terms of 8 bits each.
// Bound by the bounds' bytes, which lie 512 to a page and head, with few query
// rows; by the query parts' shared-memory reads and the products with many.
// 32 sequences of 8 heads, up to 32,768 positions, 4 rows: 32.6 us, 0.77 of the
// copy rate (64 sequences: 0.85); 4 sequences of 131,072, 8 rows 25, 0.80, 40
// rows 36, 0.55 (issue active 34 %, tensor pipe 27 %).  fp32 rows, with three
// times the products and query parts: 37, 29 and 92.
constexpr int kPScoreWarps = 4;

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1,
                                         uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

template <int D, int S>  // S: bf16 terms of a q value
__host__ __device__ constexpr int pscore_row() {
  return 2 * S * 2 * D + 16;  // positive and negative parts; no bank conflicts
}

// The parts of eight elements of a query row, from dimension 8 c on.
template <int D, int S>
__device__ __forceinline__ void stage_query(const PageScoreParams &p, unsigned char *to,
                                            size_t at, int c, bool there) {
  // the negative parts (for lo), then the positive ones
  if constexpr (S == 1) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (there)
      v = *(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(p.q) + at) + c);
    const uint32_t flip = p.negate ? 0x80008000u : 0u;
    const uint32_t w[4] = {v.x ^ flip, v.y ^ flip, v.z ^ flip, v.w ^ flip};
    uint32_t neg[4], pos[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      neg[e] = PairBf16::lo(w[e], 0u);
      pos[e] = PairBf16::hi(w[e], 0u);
    }
    *reinterpret_cast<uint4 *>(to + 16 * c) = make_uint4(neg[0], neg[1], neg[2], neg[3]);
    *reinterpret_cast<uint4 *>(to + 2 * D + 16 * c) =
        make_uint4(pos[0], pos[1], pos[2], pos[3]);
  } else {
    float x[8] = {};
    if (there) {
      const float4 *from =
          reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at) + 2 * c;
      const float4 u = from[0], v = from[1];
      x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
      x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
    }
    uint32_t neg[S][4] = {}, pos[S][4] = {};
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = p.negate ? -x[e] : x[e];
      const bool up = v > 0.f, nan = v != v;
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const float h = __bfloat162float(__float2bfloat16_rn(v));
        const uint32_t bits = __float_as_uint(h) >> 16 << (16 * (e & 1));
        if (up || nan) pos[s][e / 2] |= bits;
        if (!up) neg[s][e / 2] |= bits;
        v = isfinite(h) ? v - h : 0.f;  // what is left; nothing of an infinity
      }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
      *reinterpret_cast<uint4 *>(to + s * 2 * D + 16 * c) =
          make_uint4(neg[s][0], neg[s][1], neg[s][2], neg[s][3]);
      *reinterpret_cast<uint4 *>(to + (S + s) * 2 * D + 16 * c) =
          make_uint4(pos[s][0], pos[s][1], pos[s][2], pos[s][3]);
    }
  }
}

template <int D, int S>
__global__ void __launch_bounds__(32 * kPScoreWarps)
    page_scores_kernel(const PageScoreParams p) {
  constexpr int NC = D / 32;  // 16-byte chunks of a lane on one side
  constexpr int ROW = pscore_row<D, S>();
  extern __shared__ __align__(16) unsigned char sq[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  // heads side by side: their bounds of a page lie next to one another
  const unsigned bc = blockIdx.x / (unsigned)p.num_kv_heads;
  const int head = (int)(blockIdx.x - bc * (unsigned)p.num_kv_heads);
  const int b = (int)(bc / (unsigned)p.chunks);
  const int chunk = (int)(bc - (unsigned)b * (unsigned)p.chunks);
  const size_t unit = (size_t)b * p.num_kv_heads + head;
  pdl_wait();
  pdl_launch_dependents();
  const int L = p.seq_lens[b];
  int n = (int)(((long long)L + kBlockSize - 1) / kBlockSize);
  if (L < 0 || L > (long long)p.max_blocks * kBlockSize) {
    if (threadIdx.x == 0 && chunk == 0) raise_pages(SVP_DEV_BAD_SEQ_LEN);
    n = 0;
  }
  const int tiles = (p.max_blocks + 15) / 16;
  const int first = chunk * p.tiles_per_cta;
  const int last = min(first + p.tiles_per_cta, tiles);
  float *const out = p.scores + unit * p.max_blocks;
  const int32_t *const table = p.block_table + (size_t)b * p.max_blocks;
  // lane r < 16: the physical page of page r of a tile, or -1
  auto page_ids = [&](int tile) {
    const int at = tile * 16 + lane;
    int id = -1;
    if (lane < 16 && tile < last && at < n) {
      id = table[at];
      if (id < 0 || id >= p.num_blocks) {
        raise_pages(SVP_DEV_BAD_BLOCK_ID);
        id = -1;
      }
    }
    return id;
  };
  // this lane's pieces of a tile, [page g, g + 8][lo, hi][NC]
  constexpr int PIECES = 4 * NC;
  const uint32_t ring = smem_u32(sq) + (unsigned)((p.rows + 7) / 8 * 8) * ROW +
                        (warp * PIECES * 32 + lane) * 16;
  auto load = [&](int id) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int page = __shfl_sync(kFull, id, g + 8 * h);
      const uint4 *src = reinterpret_cast<const uint4 *>(
          static_cast<const unsigned char *>(p.bounds) +
          ((size_t)(page < 0 ? 0 : page) * p.num_kv_heads + head) * (4 * D));
#pragma unroll
      for (int x = 0; x < 2 * NC; ++x)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                         ring + (h * 2 * NC + x) * 512),
                     "l"(src + x / NC * (D / 8) + 4 * (x % NC) + t),
                     "r"(page < 0 ? 0 : 16)  // (a page that is not there: zeros)
                     : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // the first tiles' bounds are on their way while the query rows are laid out
  constexpr int W = kPScoreWarps;
  int id[2];  // of this warp's next tiles
#pragma unroll
  for (int i = 0; i < 2; ++i) id[i] = page_ids(first + warp + i * W);
  if (first * 16 < n) {
    load(id[0]);
    // row r of this launch is (position, head of the group) row0 + r
    const int padded = (p.rows + 7) / 8 * 8;
#pragma unroll 4
    for (int i = threadIdx.x; i < padded * (D / 8); i += 32 * kPScoreWarps) {
      const int r = i / (D / 8), c = i % (D / 8);
      const int row = p.row0 + min(r, p.rows - 1);
      const size_t at = (((size_t)b * p.q_len + row / p.group) * p.num_q_heads +
                         (size_t)head * p.group + row % p.group) * D;
      stage_query<D, S>(p, sq + r * ROW, at, c, r < p.rows);
    }
    __syncthreads();
  }
  const int n_nt = (p.rows + 7) / 8;
  for (int tile = first + warp; tile < last; tile += W) {
    const int page0 = tile * 16;
    if (page0 >= n) {  // nothing here: -inf, so that a score is always there
      if (lane < 16 && page0 + lane < p.max_blocks && !p.more)
        out[page0 + lane] = -INFINITY;
      continue;
    }
    const int next = page_ids(tile + 2 * W);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    uint4 w[2][2][NC];
#pragma unroll
    for (int x = 0; x < PIECES; ++x)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[x / (2 * NC)][x / NC % 2][x % NC].x),
                     "=r"(w[x / (2 * NC)][x / NC % 2][x % NC].y),
                     "=r"(w[x / (2 * NC)][x / NC % 2][x % NC].z),
                     "=r"(w[x / (2 * NC)][x / NC % 2][x % NC].w)
                   : "r"(ring + x * 512)
                   : "memory");
    const int now = id[0];
    id[0] = id[1];
    id[1] = next;
    load(id[0]);
    float best[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
    for (int nt = 0; nt < n_nt; ++nt) {
      float acc[2][2][4] = {};  // four chains of products
      const unsigned char *qr = sq + (nt * 8 + g) * ROW + 16 * t;
#pragma unroll
      for (int s = 0; s < S; ++s)
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int side = 0; side < 2; ++side) {
            const uint4 q = *reinterpret_cast<const uint4 *>(
                qr + (side * S + s) * 2 * D + 64 * c);
            const uint4 &a = w[0][side][c], &e = w[1][side][c];
            mma_bf16(acc[side][0], a.x, e.x, a.y, e.y, q.x, q.y);
            mma_bf16(acc[side][1], a.z, e.z, a.w, e.w, q.z, q.w);
          }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (nt * 8 + 2 * t + (e & 1) < p.rows)
          best[e >> 1] = max_nan(best[e >> 1], (acc[0][0][e] + acc[0][1][e]) +
                                                   (acc[1][0][e] + acc[1][1][e]));
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      best[h] = max_nan(best[h], __shfl_xor_sync(kFull, best[h], 1));
      best[h] = max_nan(best[h], __shfl_xor_sync(kFull, best[h], 2));
      const int at = page0 + g + 8 * h;
      const bool there = __shfl_sync(kFull, now, g + 8 * h) >= 0;
      if (t == 0 && at < p.max_blocks) {
        float v = there ? best[h] * p.scale : -INFINITY;
        if (p.more && there) v = max_nan(v, out[at]);
        out[at] = v;
      }
    }
  }
  // (the zeros of a tile that is not there may still be on their way)
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// ---- selection ----
// The k-th largest of a list's scores: a histogram of 1024 equal parts of the
// keys' range tells which part holds it, and how many it is from that part's
// top; of a part with few keys those are ranked by counting, one with many
// is cut into 1024 again (three times at most: keys have 32 bits).  Then the
// kept pages are numbered in order.  Bound by that chain of about ten
// barriers: 256 lists of up to 2048 scores 6.3 us a call, 32 of 8192 8.2 (bit by
// bit, 32 counts and barriers: 13.8 and 20.2).
constexpr int kPickMax = 1024;   // threads
constexpr int kPickKeys = 16;    // keys of a thread held in registers
constexpr int kPickBins = 1024;
constexpr int kPickFew = 128;    // keys ranked by counting

struct PickShared {
  uint4 hist4[kPickBins / 4];
  alignas(16) unsigned few[kPickFew + 4];
  unsigned warp_a[32], warp_b[32];
  unsigned cells[kPickMax * kPickKeys / 32];
  unsigned bin, above, in_bin, n_few, edge, ties;
};

// Ascending unsigned order; NaN above everything, -0 as +0.  Never 0.
__device__ __forceinline__ unsigned pick_key(float x) {
  if (x != x) return 0xffffffffu;
  const unsigned u = __float_as_uint(x + 0.f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Exclusive prefix sum over the block; buf holds one value per warp.
__device__ __forceinline__ unsigned pick_scan(unsigned v, unsigned *buf) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  unsigned incl = v;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, incl, off);
    if (lane >= off) incl += y;
  }
  if (lane == 31) buf[warp] = incl;
  __syncthreads();
  return __reduce_add_sync(kFull, lane < warp ? buf[lane] : 0u) + incl - v;
}

template <int KEYS>  // keys of a thread in registers; 0: read again each time
__global__ void __launch_bounds__(kPickMax)
    pick_pages_kernel(const PickParams p) {
  __shared__ PickShared sm;
  unsigned *const hist = reinterpret_cast<unsigned *>(sm.hist4);
  const int tid = threadIdx.x, T = blockDim.x;
  const int warp = tid >> 5, lane = tid & 31, n_warps = T >> 5;
  const unsigned unit = blockIdx.x;
  const int b = (int)(unit / (unsigned)p.heads);
  pdl_wait();
  pdl_launch_dependents();
  int32_t *const pages = p.pages + (size_t)unit * p.n_select;
  const float *const scores = p.scores + (size_t)unit * p.max_blocks;
  const int L = p.seq_lens[b];
  float x[KEYS ? KEYS : 1];
  if constexpr (KEYS > 0) {
#pragma unroll
    for (int i = 0; i < KEYS; ++i)
      x[i] = i * T + tid < p.max_blocks ? scores[i * T + tid] : 0.f;
  }
  int n = (int)(((long long)L + kBlockSize - 1) / kBlockSize);
  if (L < 0 || n > p.max_blocks) {
    if (tid == 0) raise_pages(SVP_DEV_BAD_SEQ_LEN);
    n = 0;
  }
  if (n <= p.n_select) {
    for (int i = tid; i < p.n_select; i += T) pages[i] = i < n ? i : -1;
    return;
  }
  // candidates [c0, c1) compete for k places
  const int c0 = p.n_sink, c1 = n - p.n_recent;
  const unsigned k = (unsigned)(p.n_select - p.n_sink - p.n_recent);
  unsigned key[KEYS ? KEYS : 1];
  if constexpr (KEYS > 0) {
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const int j = i * T + tid;
      key[i] = j >= c0 && j < c1 ? pick_key(x[i]) : 0u;
    }
  }
  auto each = [&](auto f) {  // f(key) of every candidate
    if constexpr (KEYS > 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i)
        if (key[i] != 0u) f(key[i]);
    } else {
      for (int j = c0 + tid; j < c1; j += T) f(pick_key(scores[j]));
    }
  };
  unsigned edge = 0xffffffffu, ties = 0;  // kept: above the edge, and ties at it
  if (k > 0) {
    unsigned lo = 0xffffffffu, hi = 0u;
    each([&](unsigned y) {
      lo = min(lo, y);
      hi = max(hi, y);
    });
    lo = __reduce_min_sync(kFull, lo);
    hi = __reduce_max_sync(kFull, hi);
    if (lane == 0) {
      sm.warp_a[warp] = lo;
      sm.warp_b[warp] = hi;
    }
    for (int i = tid; i < kPickBins / 4; i += T) sm.hist4[i] = make_uint4(0, 0, 0, 0);
    if (tid == 0) sm.n_few = 0;
    __syncthreads();
    lo = __reduce_min_sync(kFull, lane < n_warps ? sm.warp_a[lane] : 0xffffffffu);
    hi = __reduce_max_sync(kFull, lane < n_warps ? sm.warp_b[lane] : 0u);
    unsigned need = k;
    while (true) {
      // keys in [lo, hi], `need` of them wanted
      const unsigned range = hi - lo;
      const int shift = range < kPickBins ? 0 : 22 - __clz(range);
      each([&](unsigned y) {
        if (y >= lo && y <= hi) atomicAdd(&hist[(hi - y) >> shift], 1u);
      });
      __syncthreads();
      // from the top: a thread takes kPickBins / T bins, one to eight
      const int per = kPickBins / T;
      unsigned c[8];
      if (per >= 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 q = 4 * i < per ? sm.hist4[tid * (per / 4) + i]
                                      : make_uint4(0, 0, 0, 0);
          c[4 * i] = q.x;
          c[4 * i + 1] = q.y;
          c[4 * i + 2] = q.z;
          c[4 * i + 3] = q.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = i < per ? hist[tid * per + i] : 0u;
      }
      unsigned mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) mine += c[i];
      unsigned before = pick_scan(mine, sm.warp_a);
      if (before < need && before + mine >= need) {  // exactly one thread
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (before < need && before + c[i] >= need) {
            sm.bin = (unsigned)(tid * per + i);
            sm.above = before;
            sm.in_bin = c[i];
            before = need;  // found
          } else {
            before += c[i];
          }
        }
      }
      __syncthreads();
      const unsigned in_bin = sm.in_bin;
      need -= sm.above;
      hi -= sm.bin << shift;
      lo = hi - min(hi - lo, (1u << shift) - 1u);
      if (shift == 0 || need == in_bin) {
        // equal keys, or all of the part's
        edge = shift == 0 ? hi : lo - 1u;
        ties = shift == 0 ? need : 0u;
        break;
      }
      if (in_bin <= kPickFew) {
        each([&](unsigned y) {
          if (y >= lo && y <= hi) sm.few[atomicAdd(&sm.n_few, 1u)] = y;
        });
        if (tid < 4) sm.few[in_bin + tid] = 0u;  // below every key
        __syncthreads();
        for (unsigned c = tid; c < in_bin; c += T) {
          const unsigned y = sm.few[c];
          unsigned above = 0, same = 0;
          for (unsigned o = 0; o < in_bin; o += 4) {
            const uint4 q = *reinterpret_cast<const uint4 *>(sm.few + o);
            above += (q.x > y) + (q.y > y) + (q.z > y) + (q.w > y);
            same += (q.x == y) + (q.y == y) + (q.z == y) + (q.w == y);
          }
          if (above < need && above + same >= need) {  // (equal keys agree)
            sm.edge = y;
            sm.ties = need - above;
          }
        }
        __syncthreads();
        edge = sm.edge;
        ties = sm.ties;
        break;
      }
      for (int i = tid; i < kPickBins / 4; i += T) sm.hist4[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
  }
  // number the kept pages: T positions a row, warp after warp
  const unsigned lower = (1u << lane) - 1u;
  auto look = [&](int j, unsigned y, unsigned &sure, unsigned &tied) {
    const bool forced = j < c0 || (j >= c1 && j < n);
    sure = __ballot_sync(kFull, forced || y > edge);
    tied = __ballot_sync(kFull, y != 0u && y == edge);
  };
  auto put = [&](int j, unsigned sure, unsigned tied, unsigned s0, unsigned t0) {
    const bool a = (sure >> lane) & 1u, t = (tied >> lane) & 1u;
    t0 += __popc(tied & lower);
    if (a || (t && t0 < ties)) pages[s0 + __popc(sure & lower) + min(t0, ties)] = j;
  };
  if constexpr (KEYS > 0) {
    if (k == 0) {
#pragma unroll
      for (int i = 0; i < KEYS; ++i) key[i] = 0u;
    }
    unsigned sure[KEYS], tied[KEYS];
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      look(i * T + tid, key[i], sure[i], tied[i]);
      if (lane == 0)
        sm.cells[i * n_warps + warp] = (__popc(sure[i]) << 16) | __popc(tied[i]);
    }
    __syncthreads();
    // at most T cells: both counts' prefix sums at once
    const unsigned c = tid < KEYS * n_warps ? sm.cells[tid] : 0u;
    const unsigned before = pick_scan(c, sm.warp_b);
    if (tid < KEYS * n_warps) sm.cells[tid] = before;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < KEYS; ++i) {
      const unsigned y = sm.cells[i * n_warps + warp];
      put(i * T + tid, sure[i], tied[i], y >> 16, y & 0xffffu);
    }
  } else {
    unsigned n_sure = 0, n_tied = 0;
    for (int i = 0, j0 = 0; j0 < n; ++i, j0 += T) {
      const int j = j0 + tid;
      unsigned sure, tied;
      look(j, k > 0 && j >= c0 && j < c1 ? pick_key(scores[j]) : 0u, sure, tied);
      unsigned *const row = sm.cells + 32 * (i & 1);
      if (lane == 0) row[warp] = (__popc(sure) << 16) | __popc(tied);
      __syncthreads();
      const unsigned all = lane < n_warps ? row[lane] : 0u;
      const unsigned y = __reduce_add_sync(kFull, lane < warp ? all : 0u);
      put(j, sure, tied, n_sure + (y >> 16), n_tied + (y & 0xffffu));
      const unsigned sum = __reduce_add_sync(kFull, all);
      n_sure += sum >> 16;
      n_tied += sum & 0xffffu;
    }
  }
}

template <int DT>
cudaError_t bounds_t(const BoundsParams &p, dim3 grid, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(32 * kBoundWarps);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return p.head_dim == 64 ? cudaLaunchKernelEx(&cfg, page_bounds_kernel<DT, 64>, p)
                          : cudaLaunchKernelEx(&cfg, page_bounds_kernel<DT, 128>, p);
}

template <int D, int S>
cudaError_t scores_t(const PageScoreParams &p, unsigned grid, cudaStream_t stream) {
  constexpr int kRing = kPScoreWarps * 16 * 4 * D;
  constexpr int kRows = S == 1 ? kPageScoreRows : kPageScoreRowsF32;
  static_assert(kRows * pscore_row<D, S>() + kRing <= 227 * 1024, "shared memory");
  const size_t smem = (size_t)((p.rows + 7) / 8 * 8) * pscore_row<D, S>() + kRing;
  if (smem > 48 * 1024) {
    // always the most that any launch takes: launches in other host threads
    // may need more than this one
    const cudaError_t e = cudaFuncSetAttribute(
        page_scores_kernel<D, S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kRows * pscore_row<D, S>() + kRing);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(page_scores_kernel<D, S>, grid, 32 * kPScoreWarps, smem, stream, p);
}

}  // namespace

cudaError_t launch_page_bounds(BoundsParams p, int sms, cudaStream_t stream) {
  // a warp takes heads of a page of 4 KB in all, so that its look-ups serve more
  // than 1 KB, once there are enough warps all the same
  const int row = p.dtype == SVP_F32        ? 4 * p.head_dim
                  : p.dtype == SVP_BF16     ? 2 * p.head_dim
                  : p.dtype == SVP_FP8_E4M3 ? p.head_dim
                                            : fp4_row_bytes(p.head_dim);
  p.heads = std::max(1, 256 / row);
  if ((long long)p.batch * p.max_pages * p.num_kv_heads < 256LL * sms) p.heads = 1;
  const long long items =
      (long long)p.max_pages * ((p.num_kv_heads + p.heads - 1) / p.heads);
  const long long blocks = (items + kBoundWarps - 1) / kBoundWarps;
  if (blocks > 0x7fffffffLL / kBoundWarps) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)blocks, (unsigned)p.batch);
  switch (p.dtype) {
    case SVP_F32: return bounds_t<SVP_F32>(p, grid, stream);
    case SVP_BF16: return bounds_t<SVP_BF16>(p, grid, stream);
    case SVP_FP8_E4M3: return bounds_t<SVP_FP8_E4M3>(p, grid, stream);
    default: return bounds_t<SVP_FP4_E2M1>(p, grid, stream);
  }
}

cudaError_t launch_page_scores(PageScoreParams p, int sms, cudaStream_t stream) {
  const long long tiles = ((long long)p.max_blocks + 15) / 16;
  const long long units = (long long)p.batch * p.num_kv_heads;
  // One wave of CTAs (four to an SM, or what its shared memory holds) if that is
  // at most 12 tiles to a warp: the
  // query rows are laid out once in each.  Else shorter parts, which even out
  // ragged lengths (5 tiles to a warp 33 us where 16 take 38: 32 sequences of 8
  // heads, up to 32,768 positions), not as short with many rows (40 rows over
  // 131,072 positions of 8 sequences: 8 tiles 72 us, 3 tiles 79).
  constexpr int W = kPScoreWarps;
  const int splits = p.f32 ? 3 : 1;
  const long long smem = (p.rows + 7) / 8 * 8LL * (4 * splits * p.head_dim + 16) +
                         64LL * W * p.head_dim + 1024;
  const long long fit = std::max(1LL, std::min(4LL, (228 << 10) / smem));
  long long per = std::max(1LL, fit * sms / units);
  per = std::max<long long>((tiles + per - 1) / per, W);
  if (per > 12 * W) per = (p.rows > 32 ? 8 : 5) * W;
  const long long chunks = (tiles + per - 1) / per;
  if (chunks * units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  p.tiles_per_cta = (int)per;
  p.chunks = (int)chunks;
  const unsigned grid = (unsigned)(chunks * units);
  if (p.f32)
    return p.head_dim == 64 ? scores_t<64, 3>(p, grid, stream)
                            : scores_t<128, 3>(p, grid, stream);
  return p.head_dim == 64 ? scores_t<64, 1>(p, grid, stream)
                          : scores_t<128, 1>(p, grid, stream);
}

cudaError_t launch_pick_pages(const PickParams &p, cudaStream_t stream) {
  const long long units = (long long)p.batch * p.heads;
  if (units > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // eight keys to a thread, sixteen where that takes more threads than there are
  const int most = p.max_blocks;
  const int threads = most <= 1024 ? 128 : most <= 2048 ? 256 : most <= 4096 ? 512 : kPickMax;
  if (most <= 8 * threads)
    return launch_pdl(pick_pages_kernel<8>, (unsigned)units, threads, 0, stream, p);
  if (most <= kPickKeys * threads)
    return launch_pdl(pick_pages_kernel<kPickKeys>, (unsigned)units, threads, 0, stream, p);
  return launch_pdl(pick_pages_kernel<0>, (unsigned)units, threads, 0, stream, p);
}

cudaError_t status_word_pages(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_pages);
}

}  // namespace svp
