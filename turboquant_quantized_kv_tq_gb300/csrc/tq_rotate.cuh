// One pass over a row of D coordinates: RMS norm and position rotation (fp32).
//
// D / 16 threads share a row; thread l holds two chunks of 8 coordinates.  With r = rotary_dim,
// threads l < r / 16 hold chunks l and l + r / 16 -- with "halves" pairing the two members of
// eight pairs, with "interleaved" pairing two groups of four whole pairs -- and the other threads
// the unrotated rest.  So a rotation never needs a neighbour's value, and every load and store is
// 16 bytes (16-bit types) of a contiguous run.
//
// The angle of a pair is position * frequency in turns modulo 1, in 64-bit fixed point: the product
// of the 64-bit fraction with the position wraps exactly, its top 32 bits are the signed fraction
// of a turn to 2^-32 (an angle error of 2^-33 turns for any position, plus the frequency's own
// rounding of 2^-63 turns per position), and sincospi of the fp32 rest to a quarter turn needs no
// range reduction.  A table of cosines by position would be 64 MB at 131072 positions and d = 128; the
// cosines of a token are instead computed once per block and shared by all its heads.
#pragma once

#include <type_traits>

#include "tq_byte.h"
#include "tq_device.cuh"

namespace tqb {

using tqd::kFull;

template <typename T>
struct Raw8 {  // 8 elements as loaded
  uint4 v[sizeof(T) * 8 / 16];
};

template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) * 8 / 16); ++i) r.v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
// (no read-only path: a buffer that the same launch may overwrite, row by row)
template <typename T>
__device__ __forceinline__ Raw8<T> load8_rw(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)(sizeof(T) * 8 / 16); ++i) r.v[i] = *(reinterpret_cast<const uint4*>(p) + i);
  return r;
}

__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x);
    x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z);
    x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__nv_bfloat16>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<__half>& r, float (&x)[8]) {
  const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store8(__half* p, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = tqd::pack_half2(x[2 * i], x[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// The chunks (of 8 coordinates) that thread l of a row holds.
__device__ __forceinline__ int chunk_a(int l, int r) { return l < r / 16 ? l : r / 8 + 2 * (l - r / 16); }
__device__ __forceinline__ int chunk_b(int l, int r) { return l < r / 16 ? l + r / 16 : r / 8 + 2 * (l - r / 16) + 1; }

// Cosines and sines of one token lie in shared memory as [4][r / 16] groups of two pairs
// (cos, cos, sin, sin): group j of thread l at j * (r / 16) + l, so that the threads of a row read
// consecutive 16-byte words.  Index of pair p's cosine (its sine is 2 floats on):
__device__ __forceinline__ int pair_slot(int p, int r, int interleaved) {
  int l, j;
  if (!interleaved) {
    l = p >> 3;
    j = (p & 7) >> 1;
  } else {
    const int hi = p >= r / 4;
    const int u = p - (hi ? r / 4 : 0);
    l = u >> 2;
    j = 2 * hi + ((u & 3) >> 1);
  }
  return 4 * (j * (r / 16) + l) + (p & 1);
}

// (cos, sin) of one pair at the token whose positions on axis a are pos(a).
template <typename F>
__device__ __forceinline__ float2 pair_angle(uint64_t entry, F pos) {
  const long long at = pos((int)(entry & 3u));
  const uint64_t turns = (entry & ~3ull) * (uint64_t)at;              // modulo one turn
  // nearest quarter turn and the signed rest in [-1/8, 1/8] turns, in half-turns for sincospi: as fp32 the
  // rest is off by 2^-27 half-turns at most, a quarter of what the whole fraction would be
  const uint32_t frac = (uint32_t)((turns + 0x80000000ull) >> 32);
  const uint32_t quarter = (frac + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(frac - (quarter << 30)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(x, &s, &c);
  const float cc = quarter & 1 ? s : c, ss = quarter & 1 ? c : s;
  return make_float2((quarter + 1) & 2 ? -cc : cc, quarter & 2 ? -ss : ss);
}

// Pairs of fp32 values in one instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;\n" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 1 / sqrt(ms) for 2^-126 <= ms < infinity (one Newton step: the approximation's last bit would cost codes at rounding
// borders); NaN elsewhere (below 2^-126 the approximation flushes to 1 / 0).
__device__ __forceinline__ float norm_factor(float ms) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(ms));
  return fmaf(0.5f * r, fmaf(-ms, r * r, 1.f), r);
}

// The factor of rows whose mean square is out of that range (far; the warp's other rows come along unchanged).  With c
// the power of two that brings the larger of max |x| and sqrt(eps) to [1, 2), the values become c x and their factor is
// 1 / sqrt(mean((c x)^2) + c^2 eps).  A row with an infinity gets 0 (finite coordinates become 0, the infinite ones
// NaN), a row of zeros without eps infinity (NaN, as 0 / 0 is).
template <int TPR>
__device__ __forceinline__ float far_norm_factor(uint64_t (&a2)[4], uint64_t (&b2)[4], int D, float eps, bool far) {
  float top = sqrtf(eps), x, y;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpair(a2[i], x, y);
    top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
    unpair(b2[i], x, y);
    top = fmaxf(top, fmaxf(fabsf(x), fabsf(y)));
  }
#pragma unroll
  for (int m = 1; m < TPR; m <<= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, m));
  const int e = min(126, max(-126, (int)(__float_as_uint(top) >> 23) - 127));
  const float c = far ? __uint_as_float((unsigned)(127 - e) << 23) : 1.f;
  uint64_t s2 = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a2[i] = mul2(a2[i], pair(c, c));
    b2[i] = mul2(b2[i], pair(c, c));
    s2 = fma2(b2[i], b2[i], fma2(a2[i], a2[i], s2));
  }
  unpair(s2, x, y);
  float ss = x + y;
#pragma unroll
  for (int m = 1; m < TPR; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
  const float ms = ss / (float)D + eps * c * c;
  return ms == INFINITY ? 0.f : ms == 0.f ? INFINITY : norm_factor(ms);
}

// Norm (norm: with wa, wb the row's weights) and rotation of one row's values.  Rows whose squares leave fp32's range
// are seen to at once (kAll), or only reported (kNear: true, the row's values mean nothing) and taken again from their
// input by kFar.  Measured: seen to at once in every row of a pass of queries, the append of 4096 tokens takes 38.5 us,
// with the second pass behind the rows in flight 37.4 (36.8 without either; the code of two kinds of block is more than
// the instruction cache holds).
enum RowRange { kAll, kNear, kFar };
template <int TPR, RowRange RANGE>
__device__ __forceinline__ bool norm_rotate_row(float (&a)[8], float (&b)[8], int l, bool norm, const float (&wa)[8],
                                                const float (&wb)[8], int D, float eps, const float4* cs, int r,
                                                int interleaved) {
  uint64_t a2[4], b2[4];
  bool far = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a2[i] = pair(a[2 * i], a[2 * i + 1]);
    b2[i] = pair(b[2 * i], b[2 * i + 1]);
  }
  if (norm) {
    float rs;
    if constexpr (RANGE == kFar) {
      rs = far_norm_factor<TPR>(a2, b2, D, eps, true);
    } else {
      uint64_t s2 = mul2(a2[0], a2[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) s2 = fma2(a2[i], a2[i], s2);
#pragma unroll
      for (int i = 0; i < 4; ++i) s2 = fma2(b2[i], b2[i], s2);
      float ss, s1;
      unpair(s2, ss, s1);
      ss += s1;
#pragma unroll
      for (int m = 1; m < TPR; m <<= 1) ss += __shfl_xor_sync(kFull, ss, m);
      const float ms = ss / (float)D + eps;
      rs = norm_factor(ms);
      far = !(rs > 0.f);
      if (RANGE == kAll && __any_sync(kFull, far)) {
        const float other = far_norm_factor<TPR>(a2, b2, D, eps, far);
        if (far) rs = other;
      }
    }
    const uint64_t rs2 = pair(rs, rs);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a2[i] = mul2(mul2(a2[i], rs2), pair(wa[2 * i], wa[2 * i + 1]));
      b2[i] = mul2(mul2(b2[i], rs2), pair(wb[2 * i], wb[2 * i + 1]));
    }
  }
  if (l < r / 16 && !interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = cs[j * (r / 16) + l];
      const uint64_t c = pair(v.x, v.y), s = pair(v.z, v.w), ns = pair(-v.z, -v.w), x = a2[j];
      a2[j] = fma2(b2[j], ns, mul2(x, c));
      b2[j] = fma2(b2[j], c, mul2(x, s));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    unpair(a2[i], a[2 * i], a[2 * i + 1]);
    unpair(b2[i], b[2 * i], b[2 * i + 1]);
  }
  if (l < r / 16 && interleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = cs[j * (r / 16) + l];
      float* m = j < 2 ? a + 4 * j : b + 4 * (j - 2);
      const float x = m[0], y = m[1], z = m[2], w = m[3];
      m[0] = x * v.x - y * v.z;
      m[1] = x * v.z + y * v.x;
      m[2] = z * v.y - w * v.w;
      m[3] = z * v.w + w * v.y;
    }
  }
  return far;
}

// Position of token j of batch entry b on axis a.
__device__ __forceinline__ long long token_position(const Positions& P, int axis, int b, int j, int B, int n) {
  if (P.pos) return __ldg(P.pos + ((long long)axis * B + b) * n + j);
  return (long long)(P.start ? __ldg(P.start + b) : 0) + j;
}

}  // namespace tqb
