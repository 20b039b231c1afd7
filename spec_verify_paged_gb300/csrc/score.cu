// score.cu -- accumulated attention weight of every cached key
// (paged_score_update, include/svp.h).
//
// With the log-sum-exp of every query row known from the attention call, the
// weight a row gave key j is exp(scale <q, K_j> - lse): a key's total needs
// its own K row and the query rows only.  So a page is finished by the one
// warp that reads it -- no split merge, no atomics, no shared state between
// CTAs -- and K is read once, V not at all.
//
// What bounds it: K's bytes for few rows -- 32 sequences of 32 heads, up to
// 4096 tokens, one row: bf16 101 us, 0.91 of the copy rate, fp32 181, FP8 74.
// With many rows over a 4-bit cache the start of the CTAs (lengths, page ids,
// query rows: 3-4 us each, five resident per SM) and the conversion and
// exponentials of a page (about 200 warp instructions at 20 rows): 16
// sequences of 8 heads, up to 8192 tokens, 20 rows: 28.4 us where the bytes
// take 7.9.  Fewer, longer CTAs with pages fetched three ahead left SMs idle
// at ragged lengths (53 pages a CTA: 40 us).  Design:
//  * K goes from global memory to registers as matrix operands: keys are M,
//    query rows N (m16n8k16, one page per tile), and the k positions are
//    dealt to the dimensions so that a lane's operands are consecutive
//    bytes of its key's row (16 bytes of bf16 or FP8, 8 bytes of FP4 codes).
//    There is no reuse of a page beyond its warp, so shared memory would
//    only add a copy; the next page's loads are in flight while a page is
//    multiplied.
//  * The query rows wait in shared memory as B operands (bf16 as they are;
//    fp16 with a power-of-two scale per row against FP8 and FP4 keys, whose
//    values are exact in fp16), one copy for the CTA's four warps.  Sums,
//    weights and scores are fp32.
//  * fp32 caches use fp32 FMAs in the same lane layout.
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "fp4.cuh"

namespace svp {

static __device__ unsigned int g_status_score;

namespace {

constexpr int kScoreWarps = 4;
constexpr int kScoreThreads = 32 * kScoreWarps;
constexpr int kScoreMaxPages = 32 * kScoreWarps;  // of one CTA

struct ScoreRows {
  // score scale (log2 domain) and log2-domain LSE (+inf: the row adds
  // nothing, whatever its products -- a padding row's zeros make NaN of an
  // infinite key): two rows are one 16-byte read
  alignas(16) float2 ql[kScoreRows];
  int pos[kScoreRows];        // query position within the new rows
  uint32_t bits[kScoreRows];  // ancestor bits (all ones without a tree)
};

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4],
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// This lane's part of a page's K rows (keys g and g + 8) and the A operand
// of k-step ks.  dim(ks, t): first of the four dims (slots 0..3) that lane t
// supplies in that step.
template <int DT, int D>
struct KPage;

template <int D>
struct KPage<SVP_BF16, D> {
  uint4 r[2][D / 32];
  static __device__ int dim(int ks, int t) {
    return 32 * (ks >> 1) + 8 * t + 4 * (ks & 1);
  }
  __device__ void load(const unsigned char *page, int g, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < D / 32; ++c)
        r[h][c] = __ldg(reinterpret_cast<const uint4 *>(
            page + (g + 8 * h) * (2 * D) + 64 * c + 16 * t));
  }
  __device__ void operand(int ks, int, uint32_t (&a)[4]) const {
    const uint4 x = r[0][ks >> 1], y = r[1][ks >> 1];
    a[0] = ks & 1 ? x.z : x.x;
    a[1] = ks & 1 ? y.z : y.x;
    a[2] = ks & 1 ? x.w : x.y;
    a[3] = ks & 1 ? y.w : y.y;
  }
};

template <int D>
struct KPage<SVP_FP8_E4M3, D> {
  uint4 r[2][D / 64];
  static __device__ int dim(int ks, int t) {
    return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3);
  }
  __device__ void load(const unsigned char *page, int g, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        r[h][c] = __ldg(reinterpret_cast<const uint4 *>(
            page + (g + 8 * h) * D + 64 * c + 16 * t));
  }
  __device__ void operand(int ks, int, uint32_t (&a)[4]) const {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 x = r[h][ks >> 2];
      w[h] = (ks & 3) == 0 ? x.x : (ks & 3) == 1 ? x.y
             : (ks & 3) == 2 ? x.z : x.w;
    }
    a[0] = e4m3x2_f16x2(w[0]);
    a[1] = e4m3x2_f16x2(w[1]);
    a[2] = e4m3x2_f16x2(w[0] >> 16);
    a[3] = e4m3x2_f16x2(w[1] >> 16);
  }
};

template <int D>
struct KPage<SVP_FP4_E2M1, D> {
  uint2 r[2][D / 64];
  uint32_t s[2][D / 64];
  static __device__ int dim(int ks, int t) {
    return 64 * (ks >> 2) + 16 * t + 4 * (ks & 3);
  }
  __device__ void load(const unsigned char *page, int g, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const unsigned char *row = page + (g + 8 * h) * fp4_row_bytes(D);
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        const unsigned char *q = row + 8 * (t + 4 * c);
        if constexpr (D == 128) {
          r[h][c] = __ldg(reinterpret_cast<const uint2 *>(q));
        } else {
          r[h][c] = make_uint2(__ldg(reinterpret_cast<const uint32_t *>(q)),
                               __ldg(reinterpret_cast<const uint32_t *>(q) + 1));
        }
        s[h][c] = __ldg(reinterpret_cast<const uint32_t *>(row + D / 2 + 4 * c));
      }
    }
  }
  __device__ void operand(int ks, int t, uint32_t (&a)[4]) const {
    uint32_t h[2][4];
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint2 w = r[x][ks >> 2];
      e2m1x8_h2((ks & 2) ? w.y : w.x, h[x]);
      const uint32_t sc = e4m3x2_f16x2(__byte_perm(s[x][ks >> 2], 0, t * 0x11));
      a[x] = hmul2(h[x][2 * (ks & 1)], sc);
      a[2 + x] = hmul2(h[x][2 * (ks & 1) + 1], sc);
    }
  }
};

template <int D>
struct KPage<SVP_F32, D> {
  float4 r[2][D / 16];
  __device__ void load(const unsigned char *page, int g, int t) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
        r[h][c] = __ldg(reinterpret_cast<const float4 *>(
            page + (g + 8 * h) * (4 * D) + 64 * c + 16 * t));
  }
};

template <int DT, int D>
__global__ void __launch_bounds__(kScoreThreads)
    score_kernel(const ScoreParams p, int pages_per_cta, int chunks) {
  constexpr int KS = D / 16;
  constexpr int ROWB = DT == SVP_F32 ? 4 * D : DT == SVP_BF16 ? 2 * D
                       : DT == SVP_FP8_E4M3 ? D : fp4_row_bytes(D);
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ ScoreRows rows;
  uint2 *const qf = reinterpret_cast<uint2 *>(smem_raw);   // [nt][KS][32]
  float *const qf32 = reinterpret_cast<float *>(smem_raw);  // [row][D]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int chunk = blockIdx.x % chunks;
  const int group = blockIdx.x / chunks;
  const int b = group / p.num_kv_heads, kvh = group % p.num_kv_heads;

  pdl_wait();  // the attention call that wrote lse, the append before it
  pdl_launch_dependents();
  const int L = p.seq_lens[b];
  if (L < p.q_len || L > (long long)p.max_blocks * kBlockSize) {
    if (tid == 0) atomicOr(&g_status_score, (unsigned)SVP_DEV_BAD_SEQ_LEN);
    return;
  }
  UnitInfo ui;
  int n_pages;
  visible_pages(L, p.q_len, p.n_sink, p.window, ui.n_a, ui.b_start, n_pages);
  const int page0 = chunk * pages_per_cta;
  const int page1 = min(page0 + pages_per_cta, n_pages);
  if (page0 >= n_pages) return;
  const int t0 = L - p.q_len;

  // this warp's pages: page0 + warp, + 4, ...; lane i holds the i-th's id
  const int mine = (page1 - page0 - warp + kScoreWarps - 1) / kScoreWarps;
  int phys = -1;
  if (lane < mine) {
    const int pidx = page0 + warp + lane * kScoreWarps;
    phys = __ldg(p.block_table + (size_t)b * p.max_blocks +
                 logical_block(ui, pidx));
    if (phys < 0 || phys >= p.num_blocks) {
      atomicOr(&g_status_score, (unsigned)SVP_DEV_BAD_BLOCK_ID);
      phys = -1;
    }
  }

  // ---- the query rows ----
  const int n_tiles = (p.rows + 7) / 8;
  for (int nt = warp; nt < n_tiles; nt += kScoreWarps) {
    const int r = nt * 8 + g;  // this lane's row
    const bool valid = r < p.rows;
    const int gr = p.row0 + (valid ? r : 0);
    const int i = gr / p.group;
    const int h = kvh * p.group + gr % p.group;
    const size_t qrow = ((size_t)b * p.q_len + i) * p.num_q_heads + h;
    float qs = p.qscale;
    if constexpr (DT == SVP_F32) {
      const float4 *src = reinterpret_cast<const float4 *>(p.q) + qrow * (D / 4);
      for (int c = t; c < D / 4; c += 4)
        reinterpret_cast<float4 *>(qf32)[r * (D / 4) + c] =
            valid ? __ldg(src + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      const uint16_t *src = static_cast<const uint16_t *>(p.q) + qrow * D;
      uint2 w[KS];
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        w[ks] = __ldg(reinterpret_cast<const uint2 *>(
            src + KPage<DT, D>::dim(ks, t)));
        if (!valid) w[ks] = make_uint2(0, 0);
      }
      if constexpr (DT != SVP_BF16) {
        uint32_t top = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          top = max(max(top, max(w[ks].x & 0x7fffu, (w[ks].x >> 16) & 0x7fffu)),
                    max(w[ks].y & 0x7fffu, (w[ks].y >> 16) & 0x7fffu));
        top = max(top, __shfl_xor_sync(kFull, top, 1));
        top = max(top, __shfl_xor_sync(kFull, top, 2));
        const int e = q_exponent(__uint_as_float(top << 16));
        const float f = pow2i(14 - e);
        qs *= pow2i(e - 14);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
          w[ks] = make_uint2(pack_h2(__uint_as_float(w[ks].x << 16) * f,
                                     __uint_as_float(w[ks].x & 0xffff0000u) * f),
                             pack_h2(__uint_as_float(w[ks].y << 16) * f,
                                     __uint_as_float(w[ks].y & 0xffff0000u) * f));
      }
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) qf[(nt * KS + ks) * 32 + lane] = w[ks];
    }
    if (t == 0) {
      const float lse = valid ? __ldg(p.lse + qrow) : -INFINITY;
      rows.ql[r] = make_float2(
          qs, lse == -INFINITY ? INFINITY : lse * 1.4426950408889634f);
      rows.pos[r] = i;
      rows.bits[r] = row_tree_bits(p.tree_mask, p.q_len, b, i);
    }
  }
  __syncthreads();

  // positions of the launch's first and last row: a page between them and
  // inside the last one's window needs no per-key test
  const int t_min = p.tree_mask ? t0 - 1 : t0 + p.row0 / p.group;
  const int t_max = t0 + (p.row0 + p.rows - 1) / p.group;

  auto page_at = [&](int k) {
    return __shfl_sync(kFull, phys, k & 31);
  };
  auto k_of = [&](int ph) {
    return static_cast<const unsigned char *>(p.k_cache) +
           ((size_t)ph * p.num_kv_heads + kvh) * (size_t)(kBlockSize * ROWB);
  };
  // lane t = 0 of a quad keeps key g's score, t = 1 key g + 8's
  auto score_of = [&](int ph) {
    return p.scores + ((size_t)ph * p.num_kv_heads + kvh) * kBlockSize +
           g + 8 * (t & 1);
  };
  KPage<DT, D> cur;
  float old = 0.f;
  int ph = page_at(0);
  if (mine > 0 && ph >= 0) {
    cur.load(k_of(ph), g, t);
    old = t < 2 ? *score_of(ph) : 0.f;
  }
  for (int k = 0; k < mine; ++k) {
    const int here = ph;
    KPage<DT, D> now = cur;
    const float was = old;
    ph = page_at(k + 1);
    if (k + 1 < mine && ph >= 0) {
      cur.load(k_of(ph), g, t);
      old = t < 2 ? *score_of(ph) : 0.f;
    }
    if (here < 0) continue;  // warp-uniform
    const int j0 = logical_block(ui, page0 + warp + k * kScoreWarps) * kBlockSize;
    const bool all_vis = j0 + kBlockSize - 1 <= t_min &&
                         (p.window == 0 || j0 + kBlockSize - 1 < p.n_sink ||
                          j0 > t_max - p.window);
    float sum[2] = {0.f, 0.f};
    if constexpr (DT == SVP_F32) {
      for (int r = 0; r < p.rows; ++r) {
        const float2 ql = rows.ql[r];
        const float4 *q4 = reinterpret_cast<const float4 *>(qf32) + r * (D / 4) + t;
        float d[2] = {0.f, 0.f};
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const float4 q = q4[4 * c];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            d[h] = fmaf(q.x, now.r[h][c].x, d[h]);
            d[h] = fmaf(q.y, now.r[h][c].y, d[h]);
            d[h] = fmaf(q.z, now.r[h][c].z, d[h]);
            d[h] = fmaf(q.w, now.r[h][c].w, d[h]);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          d[h] += __shfl_xor_sync(kFull, d[h], 1);
          d[h] += __shfl_xor_sync(kFull, d[h], 2);
          const float w = ex2(fmaf(d[h], ql.x, -ql.y));
          if (ql.y == INFINITY) continue;
          if (all_vis || key_visible(j0 + g + 8 * h, t0 + rows.pos[r],
                                     rows.bits[r], t0, p.n_sink, p.window))
            sum[h] += w;
        }
      }
    } else {
      uint32_t a[KS][4];  // converted once for all row tiles
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) now.operand(ks, t, a[ks]);
      auto multiply = [&](int nt, float (&acc)[4]) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint2 q = qf[(nt * KS + ks) * 32 + lane];
          if constexpr (DT == SVP_BF16)
            mma_bf16(acc, a[ks], q.x, q.y);
          else
            mma_f16(acc, a[ks], q.x, q.y);
        }
      };
      auto weigh = [&](int nt, const float (&acc)[4]) {
        const float4 ql =  // rows 2t and 2t + 1 of the tile
            *reinterpret_cast<const float4 *>(&rows.ql[nt * 8 + 2 * t]);
        float w[4] = {ex2(fmaf(acc[0], ql.x, -ql.y)), ex2(fmaf(acc[1], ql.z, -ql.w)),
                      ex2(fmaf(acc[2], ql.x, -ql.y)), ex2(fmaf(acc[3], ql.z, -ql.w))};
        if (ql.y == INFINITY) w[0] = w[2] = 0.f;
        if (ql.w == INFINITY) w[1] = w[3] = 0.f;
        if (!all_vis) {  // warp-uniform
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = nt * 8 + 2 * t + (e & 1);
            if (!key_visible(j0 + g + 8 * (e >> 1), t0 + rows.pos[r], rows.bits[r],
                             t0, p.n_sink, p.window))
              w[e] = 0.f;
          }
        }
        sum[0] += w[0] + w[1];
        sum[1] += w[2] + w[3];
      };
      // two row tiles at a time: two independent chains
      int nt = 0;
      for (; nt + 1 < n_tiles; nt += 2) {
        float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
        multiply(nt, x);
        multiply(nt + 1, y);
        weigh(nt, x);
        weigh(nt + 1, y);
      }
      if (nt < n_tiles) {
        float x[4] = {0.f, 0.f, 0.f, 0.f};
        multiply(nt, x);
        weigh(nt, x);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sum[h] += __shfl_xor_sync(kFull, sum[h], 1);
        sum[h] += __shfl_xor_sync(kFull, sum[h], 2);
      }
    }
    const int j = j0 + g + 8 * t;
    if (t < 2 && j < L)
      *score_of(here) = (j >= L - p.n_fresh ? 0.f : was) + (t ? sum[1] : sum[0]);
  }
}

template <int DT, int D>
cudaError_t launch_score_t(const ScoreParams &p, int sms, cudaStream_t stream) {
  const long long groups = (long long)p.batch * p.num_kv_heads;
  // pages of a CTA: about four waves of the CTAs an SM holds, so that the
  // hardware evens out ragged lengths, within what a warp's lanes can name
  long long per = groups * p.max_pages / ((long long)sms * 16);
  per = (per + kScoreWarps - 1) / kScoreWarps * kScoreWarps;
  if (per < kScoreWarps) per = kScoreWarps;
  if (per > kScoreMaxPages) per = kScoreMaxPages;
  const long long chunks = (p.max_pages + per - 1) / per;
  if (groups * chunks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  const int tiles = (p.rows + 7) / 8;
  const size_t smem = (size_t)tiles * 8 * D * (DT == SVP_F32 ? 4 : 2);
  auto kern = score_kernel<DT, D>;
  if (smem > 40 * 1024) {  // fp32 rows; idempotent, so no state is kept
    const cudaError_t e = cudaFuncSetAttribute(
        kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kScoreRows * D * 4);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kern, (unsigned)(groups * chunks), (unsigned)kScoreThreads,
                    smem, stream, p, (int)per, (int)chunks);
}

}  // namespace

cudaError_t launch_score_update(const ScoreParams &p, int sms,
                                cudaStream_t stream) {
  const bool d64 = p.head_dim == 64;
  switch (p.dtype) {
    case SVP_F32:
      return d64 ? launch_score_t<SVP_F32, 64>(p, sms, stream)
                 : launch_score_t<SVP_F32, 128>(p, sms, stream);
    case SVP_BF16:
      return d64 ? launch_score_t<SVP_BF16, 64>(p, sms, stream)
                 : launch_score_t<SVP_BF16, 128>(p, sms, stream);
    case SVP_FP8_E4M3:
      return d64 ? launch_score_t<SVP_FP8_E4M3, 64>(p, sms, stream)
                 : launch_score_t<SVP_FP8_E4M3, 128>(p, sms, stream);
    default:
      return d64 ? launch_score_t<SVP_FP4_E2M1, 64>(p, sms, stream)
                 : launch_score_t<SVP_FP4_E2M1, 128>(p, sms, stream);
  }
}

cudaError_t read_status_score(cudaStream_t s, unsigned *flags) {
  unsigned v = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(&v, g_status_score, sizeof v, 0,
                                            cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e != cudaSuccess) return e;
  const unsigned zero = 0;
  e = cudaMemcpyToSymbolAsync(g_status_score, &zero, sizeof zero, 0,
                              cudaMemcpyHostToDevice, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *flags |= v;
  return e;
}

}  // namespace svp
