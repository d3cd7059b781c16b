// What the byte cache's tensor-memory attention kernels share: operands, rows of the output, a block's maximum and
// probabilities.  The mathematics stands in tq_byte_tc.cu.
#pragma once

#include "tq_byte_attn.cuh"
#include "tq_tc05.cuh"

namespace tqb {

constexpr int kTok = 128;          // tokens per tile
constexpr int kThreads = 512;
constexpr int kRowRegs = 192, kOtherRegs = 64;  // 256 * 192 + 256 * 64 = 512 * 128, the launch's registers
constexpr float kTop = 7.f;        // M lies this far below the maximum it was set from
constexpr float kSlack = 15.f;     // M is raised when the maximum passes it by this: P <= 2^15

struct TcParams {
  AttnArgs a;
  int G, rows, groups;  // groups: row groups of a slab
  JoinHead* heads;  // [grid]
  float* part;      // [grid][first stretch, last](M[ROWS], l[ROWS], O[ROWS][D]); tree_kernel's: see its Plan
  int grid;
};
// Fills p (but for the groups and the grid); the device's SMs, and its index.
int tc_params(const AttnArgs& a, TcParams* p, int* dev);

// 128-byte-swizzled K-major operand: rows of 128 bytes in groups of 8 (1024 bytes).
__device__ __forceinline__ uint64_t sdesc128(uint32_t addr) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n.reg .pred e;\nelect.sync _|e, 0xffffffff;\nselp.u32 %0, 1, 0, e;\n}\n" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int tiles_of(int limit) { return (limit + kTok - 1) / kTok; }
__device__ __forceinline__ int range_of(int total, int grid) { return (total + grid - 1) / grid; }

template <int D, typename T>
__device__ __forceinline__ T* out_row(const TcParams& p, int b, int h, int row) {
  const int i = row / p.G, hd = h * p.G + row - i * p.G;
  return reinterpret_cast<T*>(p.a.out) + (((long long)b * p.a.nq + i) * p.a.Hq + hd) * D;
}

__device__ __forceinline__ void store16(__nv_bfloat16* dst, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
}
__device__ __forceinline__ void store16(__half* dst, const float* x) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = tqd::pack_half2(x[2 * i], x[2 * i + 1]);
  reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
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
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// 32 columns of this thread's lane, without the wait for the load.
__device__ __forceinline__ void ld32_async(uint32_t taddr, float* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
        "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
        "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
        "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
// The wait for the loads before it, tied to the N values it makes valid.
template <int N>
__device__ __forceinline__ void ld_wait(float* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+f"(v[i]));
}
// 8 columns stored, without the wait.
__device__ __forceinline__ void st8_async(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// The largest s + e of one block's 16 scores (left: those the row attends to, when EDGE).
template <bool EDGE>
__device__ __forceinline__ float block_top(float* v, int left, float a, float e) {
  if (EDGE) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k >= left) v[k] = -INFINITY;
  }
  float m = v[0];
#pragma unroll
  for (int k = 1; k < 15; k += 2) m = fmaxf(m, fmaxf(v[k], v[k + 1]));
  m = fmaxf(m, v[15]);
  const float top = fmaf(m, a, e);
  // (a block without a token of the row stays out: its scale may be anything)
  return EDGE && m == -INFINITY ? -INFINITY : top;
}
// P of one block as fp16 pairs in V's stored token order; the sum of its 16 values is returned.
template <bool EDGE>
__device__ __forceinline__ float block_p(const float* v, int left, float a, float b, uint32_t* w) {
  const uint64_t a2 = pair(a, a), b2 = pair(b, b);
  float x[16];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    unpair(fma2(pair(v[2 * k], v[2 * k + 1]), a2, b2), x[2 * k], x[2 * k + 1]);
    x[2 * k] = ex2(x[2 * k]);
    x[2 * k + 1] = ex2(x[2 * k + 1]);
  }
  if (EDGE) {
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (k >= left) x[k] = 0.f;
  }
  uint64_t s0 = pair(x[0], x[1]), s1 = pair(x[2], x[3]);
#pragma unroll
  for (int k = 2; k < 8; k += 2) {
    s0 = add2(s0, pair(x[2 * k], x[2 * k + 1]));
    s1 = add2(s1, pair(x[2 * k + 2], x[2 * k + 3]));
  }
  float t0, t1;
  unpair(add2(s0, s1), t0, t1);
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    w[2 * m] = tqd::pack_half2(x[2 * m], x[2 * m + 1]);
    w[2 * m + 1] = tqd::pack_half2(x[2 * m + 8], x[2 * m + 9]);
  }
  return t0 + t1;
}

}  // namespace tqb
