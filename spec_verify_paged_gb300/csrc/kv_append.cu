// kv_append.cu -- scatter the new tokens' K/V rows into the paged cache, and
// the inverse (kv_gather).
//
// Page: "KV cache & Flash Attention", sections "KV cache" (store K and V of
// every token once) and "PagedAttention" (logical position -> physical
// block via the page table).  Row (b, k, g) of k_new/v_new goes to logical
// position pos = seq_lens[b] - n_new + k, i.e. page block_table[b][pos/16],
// row pos % 16, kv head g.  A byte copy: one warp moves one K row and one V
// row with 16-byte vector accesses.  Into an FP8 E4M3 cache each bf16 value
// x becomes the code of x / scale (round to nearest even, saturating).  Into
// a 4-bit cache a lane takes one block of 16 values: the block's scale is
// the E4M3 value of max|y| / 6 (y = x / k_scale), so the largest value maps
// to the largest code, and the codes are E2M1 of y / scale.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "fp4.cuh"
#include "ptx.cuh"
#include "svp.h"
#include "svp_internal.h"

namespace svp {

static __device__ unsigned int g_status_append;

constexpr int kAppendWarps = 8;

// 8 bf16 values -> E4M3 codes of x / s.
__device__ __forceinline__ uint2 quant_fp8(uint4 w, float s) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t packed = 0;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint32_t u = in[2 * h + t];
      const float2 f = make_float2(__uint_as_float(u << 16) / s,
                                   __uint_as_float(u & 0xffff0000u) / s);
      packed |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3)
                << (16 * t);
    }
    out[h] = packed;
  }
  return make_uint2(out[0], out[1]);
}

__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_append_kernel(const AppendParams p) {
  // the attention kernel that usually follows may set itself up meanwhile;
  // it reads the caches only after this grid has completed
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const long long n_rows = (long long)p.batch * p.n_new * p.num_kv_heads;
  if (row >= n_rows) return;
  const int g = (int)(row % p.num_kv_heads);
  const int k = (int)((row / p.num_kv_heads) % p.n_new);
  const int b = (int)(row / ((long long)p.num_kv_heads * p.n_new));
  const int L = p.seq_lens[b];
  if (L < p.n_new || L > (long long)p.max_blocks * kBlockSize) {
    if (lane == 0) atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_SEQ_LEN);
    return;
  }
  const int pos = L - p.n_new + k;
  const int phys = p.block_table[(size_t)b * p.max_blocks + pos / kBlockSize];
  if (phys < 0 || phys >= p.num_blocks) {
    if (lane == 0) atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_BLOCK_ID);
    return;
  }
  if (p.fp8) {
    // 8 bf16 values (16 bytes) in, 8 codes (8 bytes) out per lane step
    const size_t dst = ((((size_t)phys * p.num_kv_heads + g) * kBlockSize) +
                        pos % kBlockSize) * (size_t)p.head_dim;
    const size_t src = (size_t)row * p.head_dim * 2;
    for (int c = lane; c < p.head_dim / 8; c += 32) {
      const uint4 kv = reinterpret_cast<const uint4 *>(
          static_cast<const char *>(p.k_new) + src)[c];
      const uint4 vv = reinterpret_cast<const uint4 *>(
          static_cast<const char *>(p.v_new) + src)[c];
      reinterpret_cast<uint2 *>(static_cast<char *>(p.k_cache) + dst)[c] =
          quant_fp8(kv, p.k_scale);
      reinterpret_cast<uint2 *>(static_cast<char *>(p.v_cache) + dst)[c] =
          quant_fp8(vv, p.v_scale);
    }
    return;
  }
  const size_t row_bytes = (size_t)p.head_dim * p.elem_bytes;
  const size_t dst = ((((size_t)phys * p.num_kv_heads + g) * kBlockSize) +
                      pos % kBlockSize) * row_bytes;
  const size_t src = (size_t)row * row_bytes;
  const int chunks = (int)(row_bytes / 16);
  for (int c = lane; c < chunks; c += 32) {
    const uint4 kv = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(p.k_new) + src)[c];
    const uint4 vv = reinterpret_cast<const uint4 *>(
        static_cast<const char *>(p.v_new) + src)[c];
    reinterpret_cast<uint4 *>(static_cast<char *>(p.k_cache) + dst)[c] = kv;
    reinterpret_cast<uint4 *>(static_cast<char *>(p.v_cache) + dst)[c] = vv;
  }
}

// Logical position `pos` of sequence b: its page, or -1 with the flag
// raised for a page id outside the cache.
__device__ __forceinline__ int page_of(const int32_t *table, int max_blocks,
                                       int num_blocks, int b, int pos) {
  const int phys = table[(size_t)b * max_blocks + pos / kBlockSize];
  if (phys >= 0 && phys < num_blocks) return phys;
  atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_BLOCK_ID);
  return -1;
}

// 16 bf16 values as a block of a 4-bit row: E2M1 codes and, returned, their
// E4M3 scale.
__device__ __forceinline__ __nv_fp8_storage_t quant_fp4(const uint4 (&in)[2],
                                                        float factor,
                                                        uint32_t (&code)[2]) {
  float x[kFp4Group], top = 0.f;
  const uint32_t w[8] = {in[0].x, in[0].y, in[0].z, in[0].w,
                         in[1].x, in[1].y, in[1].z, in[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    top = fmaxf(top, fmaxf(fabsf(x[2 * i]), fabsf(x[2 * i + 1])));
  }
  top /= factor;  // division is monotonic: the largest |y|
  __nv_fp8_storage_t sc =
      __nv_cvt_float_to_fp8(top / 6.f, __NV_SATFINITE, __NV_E4M3);
  if (sc == 0) sc = 1;  // the smallest scale, 2^-9: finer than no scale
  const float s =
      __half2float(__half(__nv_cvt_fp8_to_halfraw(sc, __NV_E4M3)));
  // The codes are those of r = (x / factor) / s, both quotients rounded to
  // fp32.  Two divisions an element would be most of this kernel's time, so
  // r is taken as x c, c = (1 / factor) (1 / s), which is within 2^-21 of it,
  // and looked at where that could matter, next to E2M1's midpoints:
  //  * factor a power of two: x / factor keeps x's 8 bits and s has 4, so a
  //    quotient that is no midpoint is at least 2^-12 away from it, and
  //    rounding x c to 16 bits (Veltkamp's splitting) restores every one
  //    that is;
  //  * else: if x c (1 - 2^-20) and x c (1 + 2^-20) have the same code, that
  //    is r's; a block with one that has not (one in 10^4) divides.
  // So do blocks whose largest value saturates the scale, and factors so far
  // from 1 that c might leave fp32's range.
  const float c = (1.f / factor) * (1.f / s);
  code[0] = code[1] = 0u;
  bool sure = c > 0x1p-100f && c < 0x1p100f && top <= 8.f * s;
  if (sure && (__float_as_uint(factor) & 0x7fffffu) == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float r[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float q = x[2 * i + e] * c;
        const float t = __fmul_rn(q, 257.f);
        r[e] = __fsub_rn(t, __fsub_rn(t, q));
      }
      code[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(
                          make_float2(r[0], r[1]), __NV_E2M1, cudaRoundNearest)
                      << (8 * (i & 3));
    }
  } else if (sure) {
    uint32_t high[2] = {0u, 0u};
    const float c0 = c * (1.f - 0x1p-20f), c1 = c * (1.f + 0x1p-20f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 v = make_float2(x[2 * i], x[2 * i + 1]);
      code[i >> 2] |=
          (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v.x * c0, v.y * c0),
                                             __NV_E2M1, cudaRoundNearest)
          << (8 * (i & 3));
      high[i >> 2] |=
          (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(v.x * c1, v.y * c1),
                                             __NV_E2M1, cudaRoundNearest)
          << (8 * (i & 3));
    }
    sure = code[0] == high[0] && code[1] == high[1];
  }
  if (!sure) {
    code[0] = code[1] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      code[i >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(
                          make_float2(x[2 * i] / factor / s,
                                      x[2 * i + 1] / factor / s),
                          __NV_E2M1, cudaRoundNearest)
                      << (8 * (i & 3));
  }
  return sc;
}

// Rows into a 4-bit cache: one lane per block of 16 elements, the K and V
// blocks of a row on neighbouring lanes; a sequence's rows along x, the
// sequences along y.  Bound by one chain of loads -- row, length, page id,
// then the stores -- and the launch.  64 rows of 64 sequences, 8 heads (22 MB):
// 6.3 us as a graph node, 0.5 of the copy rate, 8.4 as a call; a decode step's
// 32 rows of 32 heads: 2.0 and 4.1.
template <int NB>  // blocks of a row
__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_append_fp4_kernel(const AppendParams p) {
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const unsigned idx = blockIdx.x * (32 * kAppendWarps) + threadIdx.x;
  const unsigned row = idx / (2 * NB), r = idx % (2 * NB);  // row: (k, g)
  if (row >= (unsigned)(p.n_new * p.num_kv_heads)) return;
  const bool is_v = r >= NB;
  const int blk = is_v ? r - NB : r;
  const int k = row / p.num_kv_heads, g = row % p.num_kv_heads;
  // the new values do not depend on the table: load them first
  const uint4 *src = reinterpret_cast<const uint4 *>(
      static_cast<const uint16_t *>(is_v ? p.v_new : p.k_new) +
      ((size_t)b * p.n_new * p.num_kv_heads + row) * (NB * kFp4Group) +
      blk * kFp4Group);
  const uint4 in[2] = {src[0], src[1]};
  const int L = p.seq_lens[b];
  if (L < p.n_new || L > (long long)p.max_blocks * kBlockSize) {
    if (r == 0) atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_SEQ_LEN);
    return;
  }
  const int pos = L - p.n_new + k;
  const int phys = page_of(p.block_table, p.max_blocks, p.num_blocks, b, pos);
  if (phys < 0) return;
  const float factor = is_v ? p.v_scale : p.k_scale;
  uint32_t code[2];
  const __nv_fp8_storage_t sc = quant_fp4(in, factor, code);
  unsigned char *dst =
      static_cast<unsigned char *>(is_v ? p.v_cache : p.k_cache) +
      (((size_t)phys * p.num_kv_heads + g) * kBlockSize + pos % kBlockSize) *
          (size_t)fp4_row_bytes(NB * kFp4Group);
  uint32_t *d32 = reinterpret_cast<uint32_t *>(dst + 8 * blk);
  d32[0] = code[0];  // rows are 4-byte aligned (36 or 72 bytes)
  d32[1] = code[1];
  dst[NB * 8 + blk] = sc;
}

// Packed rows to their slots.  A thread takes U items of K and the same of V,
// 16 bytes of new values each (a block of 32 bytes for a 4-bit cache), all in
// flight; a slot is looked up once for its item.  Bound by the rows' bytes:
// 65,568 rows of 8 bf16 heads (537 MB in and out) take 75-78 us, the copy rate,
// fp32 155, too; FP8 81 (0.74) and 4-bit 71 (0.72), which convert every value.
template <int DT, int D>
__global__ void __launch_bounds__(256) kv_append_slots_kernel(const AppendSlotsParams p) {
  constexpr bool FP4 = DT == SVP_FP4_E2M1;
  constexpr int U = FP4 ? 1 : 2;
  constexpr int PIECES = FP4 ? D / kFp4Group : DT == SVP_F32 ? D / 4 : D / 8;
  constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                       : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  pdl_wait();
  pdl_launch_dependents();
  // items: (token, head, piece); the block's first in 64 bits, the rest from it
  const unsigned per = (unsigned)p.num_kv_heads * PIECES;
  const unsigned long long first = (unsigned long long)blockIdx.x * (256 * U);
  const unsigned long long token0 = first / per;
  const unsigned rest = (unsigned)(first - token0 * per);
  uint4 in[U][2][FP4 ? 2 : 1];
  long long slot[U];
  unsigned at[U];  // piece of the token
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned x = rest + u * 256 + threadIdx.x;
    const unsigned long long token = token0 + x / per;
    at[u] = x % per;
    slot[u] = -1;
    if (token >= (unsigned long long)p.n_rows) continue;
    const size_t from = ((size_t)token * per + at[u]) * (FP4 ? 2 : 1);
#pragma unroll
    for (int side = 0; side < 2; ++side)
#pragma unroll
      for (int h = 0; h < (FP4 ? 2 : 1); ++h)
        in[u][side][h] =
            static_cast<const uint4 *>(side ? p.v_new : p.k_new)[from + h];
    slot[u] = p.slots[token];
    if (slot[u] >= (long long)p.num_blocks * kBlockSize) {
      atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_BLOCK_ID);
      slot[u] = -1;
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (slot[u] < 0) continue;
    const unsigned g = at[u] / PIECES, c = at[u] % PIECES;
    const size_t to = (((size_t)(slot[u] / kBlockSize) * p.num_kv_heads + g) *
                           kBlockSize + (size_t)(slot[u] % kBlockSize)) * ROWB;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      unsigned char *const row =
          static_cast<unsigned char *>(side ? p.v_cache : p.k_cache) + to;
      const float factor = side ? p.v_scale : p.k_scale;
      if constexpr (FP4) {
        uint32_t code[2];
        const __nv_fp8_storage_t sc = quant_fp4(in[u][side], factor, code);
        uint32_t *const d32 = reinterpret_cast<uint32_t *>(row + 8 * c);
        d32[0] = code[0];
        d32[1] = code[1];
        row[D / 2 + c] = sc;
      } else if constexpr (DT == SVP_FP8_E4M3) {
        reinterpret_cast<uint2 *>(row)[c] = quant_fp8(in[u][side][0], factor);
      } else {
        reinterpret_cast<uint4 *>(row)[c] = in[u][side][0];
      }
    }
  }
}

template <int DT, int D>
static cudaError_t slots_t(const AppendSlotsParams &p, cudaStream_t stream) {
  constexpr int U = DT == SVP_FP4_E2M1 ? 1 : 2;
  constexpr int PIECES = DT == SVP_FP4_E2M1 ? D / kFp4Group
                         : DT == SVP_F32    ? D / 4 : D / 8;
  const long long items = p.n_rows * p.num_kv_heads * PIECES;
  const long long grid = (items + 256 * U - 1) / (256 * U);
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  return launch_pdl(kv_append_slots_kernel<DT, D>, (unsigned)grid, 256, 0, stream, p);
}

cudaError_t launch_append_slots(const AppendSlotsParams &p, cudaStream_t stream) {
  const bool d64 = p.head_dim == 64;
  switch (p.dtype) {
    case SVP_F32:
      return d64 ? slots_t<SVP_F32, 64>(p, stream) : slots_t<SVP_F32, 128>(p, stream);
    case SVP_BF16:
      return d64 ? slots_t<SVP_BF16, 64>(p, stream) : slots_t<SVP_BF16, 128>(p, stream);
    case SVP_FP8_E4M3:
      return d64 ? slots_t<SVP_FP8_E4M3, 64>(p, stream)
                 : slots_t<SVP_FP8_E4M3, 128>(p, stream);
    default:
      return d64 ? slots_t<SVP_FP4_E2M1, 64>(p, stream)
                 : slots_t<SVP_FP4_E2M1, 128>(p, stream);
  }
}

// Rows back as values: a warp to a position (or to a share of its heads), so
// that the page is looked up once; a lane writes 16 bytes (8 bf16 or 4 fp32
// elements) of a K row and of the V row beside it.  Positions along x, the
// sequences along y.  Bound by the output bytes: 16,384 rows of 32 groups of
// a 4-bit cache (75 MB in, 268 MB out) take 58 us, 0.88 of the copy rate.
template <int DT, int D>
__global__ void __launch_bounds__(32 * kAppendWarps)
    kv_gather_kernel(const GatherParams p, int shares) {
  constexpr int PER = DT == SVP_F32 ? 4 : 8;  // elements of a lane
  constexpr int NC = D / PER;                 // lanes of a row
  constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                       : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  pdl_launch_dependents();
  const int b = blockIdx.y;
  const unsigned item = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
  const unsigned i = item / shares, share = item % shares;
  if (i >= (unsigned)p.n_rows) return;
  const int L = p.seq_lens[b];
  int phys = -1;
  long long pos = 0;
  if (L < 0 || L > (long long)p.max_blocks * kBlockSize) {
    if (threadIdx.x % 32 == 0)
      atomicOr(&g_status_append, (unsigned)SVP_DEV_BAD_SEQ_LEN);
  } else {
    pos = (p.starts ? (long long)p.starts[b] : (long long)L - p.n_rows) + i;
    if (pos >= 0 && pos < L)
      phys = page_of(p.block_table, p.max_blocks, p.num_blocks, b, (int)pos);
  }
  // head g's row, 16 rows further on for the next head
  const size_t first =
      ((size_t)(phys < 0 ? 0 : phys) * p.num_kv_heads * kBlockSize +
       (size_t)(pos & (kBlockSize - 1))) * ROWB;
  const size_t to0 = ((size_t)b * p.n_rows + i) * p.num_kv_heads * NC;
#pragma unroll 2
  for (int j = share * 32 + threadIdx.x % 32; j < p.num_kv_heads * NC;
       j += 32 * shares) {
    const int g = j / NC, c = j % NC;
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (phys >= 0) {
      const size_t at = first + (size_t)g * (kBlockSize * ROWB);
      const unsigned char *const src[2] = {
          static_cast<const unsigned char *>(p.k_cache) + at,
          static_cast<const unsigned char *>(p.v_cache) + at};
      if constexpr (DT == SVP_F32 || DT == SVP_BF16) {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          out[s] = __ldg(reinterpret_cast<const uint4 *>(src[s]) + c);
      } else {
        uint32_t h[2][4];  // fp16 pairs of the 8 values before the factor
        if constexpr (DT == SVP_FP8_E4M3) {
          uint2 w[2];
#pragma unroll
          for (int s = 0; s < 2; ++s)
            w[s] = __ldg(reinterpret_cast<const uint2 *>(src[s]) + c);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            h[s][0] = e4m3x2_f16x2(w[s].x);
            h[s][1] = e4m3x2_f16x2(w[s].x >> 16);
            h[s][2] = e4m3x2_f16x2(w[s].y);
            h[s][3] = e4m3x2_f16x2(w[s].y >> 16);
          }
        } else {
          uint32_t w[2], sc[2];
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            w[s] = __ldg(reinterpret_cast<const uint32_t *>(src[s]) + c);
            sc[s] = __ldg(src[s] + D / 2 + c / 2);
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint32_t s2 = e4m3x2_f16x2(sc[s] * 0x101u);
            e2m1x8_h2(w[s], h[s]);
#pragma unroll
            for (int x = 0; x < 4; ++x) h[s][x] = hmul2(h[s][x], s2);
          }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const float scale = s ? p.v_scale : p.k_scale;
          uint32_t o[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 f =
                __half22float2(*reinterpret_cast<const __half2 *>(&h[s][x]));
            const __nv_bfloat162 v =
                __floats2bfloat162_rn(f.x * scale, f.y * scale);
            o[x] = *reinterpret_cast<const uint32_t *>(&v);
          }
          out[s] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
    static_cast<uint4 *>(p.k_out)[to0 + j] = out[0];
    static_cast<uint4 *>(p.v_out)[to0 + j] = out[1];
  }
}

template <int DT, int D>
static cudaError_t gather_t(const GatherParams &p, cudaStream_t stream) {
  // one warp to a position when there are many, else as many as its lanes
  // fill (a decode step's few rows: the latency of one round of loads)
  const int full = (p.num_kv_heads * (D / (DT == SVP_F32 ? 4 : 8)) + 31) / 32;
  const long long positions = (long long)p.batch * p.n_rows;
  const int shares = positions >= 4096 ? 1
                     : (int)(4096 / positions < full ? 4096 / positions : full);
  const long long blocks =
      ((long long)p.n_rows * shares + kAppendWarps - 1) / kAppendWarps;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kv_gather_kernel<DT, D><<<dim3((unsigned)blocks, (unsigned)p.batch),
                            32 * kAppendWarps, 0, stream>>>(p, shares);
  return cudaGetLastError();
}

cudaError_t launch_kv_gather(const GatherParams &p, cudaStream_t stream) {
  const bool d64 = p.head_dim == 64;
  switch (p.dtype) {
    case SVP_F32:
      return d64 ? gather_t<SVP_F32, 64>(p, stream) : gather_t<SVP_F32, 128>(p, stream);
    case SVP_BF16:
      return d64 ? gather_t<SVP_BF16, 64>(p, stream) : gather_t<SVP_BF16, 128>(p, stream);
    case SVP_FP8_E4M3:
      return d64 ? gather_t<SVP_FP8_E4M3, 64>(p, stream)
                 : gather_t<SVP_FP8_E4M3, 128>(p, stream);
    default:
      return d64 ? gather_t<SVP_FP4_E2M1, 64>(p, stream)
                 : gather_t<SVP_FP4_E2M1, 128>(p, stream);
  }
}

cudaError_t launch_kv_append(const AppendParams &p, cudaStream_t stream) {
  const long long n_rows = (long long)p.batch * p.n_new * p.num_kv_heads;
  if (n_rows == 0) return cudaSuccess;
  if (p.fp4) {
    const int nb = p.head_dim / kFp4Group;
    const long long lanes = (long long)p.n_new * p.num_kv_heads * 2 * nb;
    constexpr int T = 32 * kAppendWarps;
    const dim3 grid((unsigned)((lanes + T - 1) / T), (unsigned)p.batch);
    if (nb == 4)
      kv_append_fp4_kernel<4><<<grid, T, 0, stream>>>(p);
    else
      kv_append_fp4_kernel<8><<<grid, T, 0, stream>>>(p);
    return cudaGetLastError();
  }
  const long long grid = (n_rows + kAppendWarps - 1) / kAppendWarps;
  kv_append_kernel<<<(unsigned)grid, 32 * kAppendWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t status_word_append(unsigned **word) {
  return cudaGetSymbolAddress(reinterpret_cast<void **>(word), g_status_append);
}

}  // namespace svp
