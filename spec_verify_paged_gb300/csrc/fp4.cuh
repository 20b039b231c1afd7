// fp4.cuh -- reading 4-bit cache rows as matrix-instruction operands.
//
// A row of D elements is D/2 bytes of E2M1 codes (element 2i in the low
// nibble of byte i) and D/16 E4M3 scales, one per 16 elements, so a row is
// one run of 9D/16 bytes and a head's 16-row page one run of 9D bytes.
// code * scale has at most 2 + 4 significant bits and lies in
// [2^-10, 2688]: it is exact in fp16, so operands are built as fp16 with no
// rounding at all and the products are summed in fp32.
//
// mma.m16n8k16 with the keys as M: lane (g = lane / 4, t = lane % 4) holds
// rows g and g + 8.  The sum over k has no order, so the k positions are
// dealt to the head dimensions in the way that lets a lane take 16
// consecutive codes -- one scale block, 8 bytes -- for four k-steps: no
// shuffles, no shared-memory round trip between the code and the MMA.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace svp {

constexpr int kFp4Group = 16;

__host__ __device__ constexpr int fp4_row_bytes(int d) {
  return d / 2 + d / kFp4Group;
}

// The four bytes of w (two E2M1 codes each) as four fp16 pairs, exact.
__device__ __forceinline__ void e2m1x8_h2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 bytes (low 16 bits) -> fp16 pair, exact.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
      (__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4],
                                        uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same into fresh accumulators.
__device__ __forceinline__ void mma_f16_first(float (&d)[4],
                                              const uint32_t (&a)[4],
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1),
        "f"(0.f));
}

// Exchange of an 8x8 fp16 tile held as MMA rows for the same tile held as
// MMA columns.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(r) : "r"(x));
  return r;
}

// Key of MMA row m (0..7) in half h (rows m and m + 8) of a 16-key page:
// transposing the scores' fp16 pairs then leaves lane t with keys 4t .. 4t+3
// of P, the keys whose V rows it reads; rows 4t + s (s fixed) start 8 banks
// apart in a page of 72-byte rows, so the V reads have no bank conflicts.
__device__ __forceinline__ int fp4_key(int m, int h) {
  return 4 * (m >> 1) + (m & 1) + 2 * h;
}

// A query row's fp16 scale: bf16 values times 2^(14 - e), e the exponent of
// the row's largest magnitude, keep their 8 bits in fp16 down to 2^-28 of
// that magnitude, and lie below 2^15.  The inverse goes into the score
// scale.  e is kept above -100 so that both powers are finite.
__device__ __forceinline__ int q_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 0xff) - 127;
  return e < -100 ? -100 : e;
}
__device__ __forceinline__ float pow2i(int e) {  // 2^e, -126 <= e <= 127
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

}  // namespace svp
