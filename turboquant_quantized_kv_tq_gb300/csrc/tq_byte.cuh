// Device helpers shared by the byte cache's kernels: where the codes of a block lie, e4m3
// conversions and power-of-two scales.
#pragma once

#include <cuda_fp8.h>

#include "tq_byte.h"
#include "tq_device.cuh"

namespace tqb {

using tqd::kFull;

// Byte of 16-byte chunk c of token t's K row.  The chunks of a row are exchanged by the row's
// index, so that eight rows read at the same chunk touch all shared-memory banks, and a block
// copied as it is into shared memory is a 128-byte-swizzled matrix operand (64-byte at d = 64).
template <int D>
__device__ __forceinline__ int k_chunk(int t, int c) {
  if constexpr (D == 64) return t * 64 + ((c ^ ((t >> 1) & 3)) << 4);
  return (c >> 3) * 2048 + t * 128 + (((c & 7) ^ (t & 7)) << 4);
}
// Place of token t among the 16 bytes of one V coordinate: tokens 2u, 2u + 1, 2u + 8, 2u + 9 are
// side by side, the order in which thread u of a quad holds the probabilities of a 16-token product.
__host__ __device__ __forceinline__ int v_slot(int t) { return ((t & 7) >> 1) * 4 + (t >> 3) * 2 + (t & 1); }

__device__ __forceinline__ long long pool_block(const Pool& P, int page, int h) {
  return (long long)page * P.heads + h;
}

// Page of block `tile` of sequence b; anything outside the table or the pool goes to the redirect
// page and is recorded.
__device__ __forceinline__ int page_of(const Pool& P, int b, long long tile) {
  int page = -1;
  if (tile >= 0 && tile < P.max_blocks) page = __ldg(P.table + (long long)b * P.max_blocks + tile);
  if ((unsigned)page >= (unsigned)P.num_pages) {
    if (P.err) atomicExch(P.err, TQ_DEVERR_BAD_PAGE);
    page = P.num_pages;
  }
  return page;
}

// 2^e as fp32, |e| <= 126
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((unsigned)(e + 127) << 23); }
// exponent of a power of two
__device__ __forceinline__ int log2i(float s) { return (int)((__float_as_uint(s) >> 23) & 255u) - 127; }

// Smallest e in [kEMin, kEMax] with amax <= 448 * 2^e = 1.75 * 2^(e + 8).
__device__ __forceinline__ int scale_exponent(float amax) {
  const unsigned u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(kEMax, max(kEMin, e));
}

// |x| where it is finite, else 0.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.402823466e38f ? a : 0.f;
}

// Two codes (a in the low byte), to nearest even, saturating; a NaN becomes 0.
__device__ __forceinline__ uint32_t encode2(float a, float b) {
  a = a == a ? a : 0.f;
  b = b == b ? b : 0.f;
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ uint32_t encode4(const float* x) { return encode2(x[0], x[1]) | (encode2(x[2], x[3]) << 16); }

// The same of finite values.
__device__ __forceinline__ uint32_t encode4_finite(const float* x) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3) |
         ((uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3) << 16);
}

// Two codes (low 16 bits) as fp16 pairs: exact, e4m3 values are fp16 values.
__device__ __forceinline__ uint32_t codes_half2(uint32_t two) {
  uint32_t r;
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %1;\ncvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ void codes_half4(uint32_t four, uint32_t& a, uint32_t& b) {
  asm("{\n.reg .b16 lo, hi;\nmov.b32 {lo, hi}, %2;\ncvt.rn.f16x2.e4m3x2 %0, lo;\ncvt.rn.f16x2.e4m3x2 %1, hi;\n}\n"
      : "=r"(a), "=r"(b)
      : "r"(four));
}
__device__ __forceinline__ float decode1(unsigned char c) {
  const uint32_t h = codes_half2(c);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

}  // namespace tqb
