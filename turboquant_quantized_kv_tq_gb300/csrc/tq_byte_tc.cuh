// What the byte cache's tensor-memory attention kernels share: the plan of their ranges, queries as e4m3
// terms, a tile's maximum and probabilities.  The mathematics stands in tq_byte_tc.cu.
#pragma once

#include "tq_byte_attn.cuh"
#include "tq_tc05.cuh"

namespace tqb {

constexpr int kTok = 128;          // tokens per tile
constexpr int kThreads = 512;
constexpr int kRowRegs = 192, kOtherRegs = 64;  // 256 * 192 + 256 * 64 = 512 * 128, the launch's registers
constexpr int kGroupCost = 8;      // virtual tiles of a row group: what a range costs beside its tiles (4: 125 us for
                                   // the last 64 positions, 8: 122, 14: 124)
constexpr float kTop = 7.f;        // M lies this far below the maximum it was set from
constexpr float kSlack = 15.f;     // M is raised when the maximum passes it by this: P <= 2^15

struct TcParams {
  AttnArgs a;
  int G, rows, groups;  // groups: row groups of a slab
  JoinHead* heads;  // [grid]
  float* part;      // [grid][first stretch, last](M[ROWS], l[ROWS], O[ROWS][D])
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
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Tokens that the rows of group rg of an entry attend to at most, and tiles.  (A tree's drafts may attend to any of
// the entry's last tokens.)
template <bool TREE>
__device__ __forceinline__ int group_limit(const TcParams& p, int rows_per, int rg, int len, int cnt) {
  const int last = min((rg + 1) * rows_per, p.rows) - 1;
  const int i = min(cnt - 1, last / p.G);
  return i * p.G + p.G - 1 < rg * rows_per ? 0 : TREE ? len : row_limit(i, len, cnt);
}
__device__ __forceinline__ int tiles_of(int limit) { return (limit + kTok - 1) / kTok; }
__device__ __forceinline__ int cost_of(int tiles) { return tiles > 0 ? tiles + kGroupCost : 0; }

// Costs before each entry (order: entry, row group, head); written by warp 0.
template <bool TREE>
__device__ __forceinline__ void fill_plan(const TcParams& p, int rows_per, int* pre, int32_t* err) {
  const int lane = threadIdx.x & 31, most = p.a.pool.max_blocks * 16;
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.a.B; b0 += 32) {
      const int b = b0 + lane;
      int t = 0;
      if (b < p.a.B) {
        const int len = clamped_len(p.a.seq_len, b, most, err), cnt = clamped_count(p.a.count, b, p.a.nq);
        for (int rg = 0; rg < p.groups; ++rg) t += cost_of(tiles_of(group_limit<TREE>(p, rows_per, rg, len, cnt)));
        t *= p.a.Hkv;
      }
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(kFull, t, m);
        if (lane >= m) t += o;
      }
      if (b < p.a.B) pre[b + 1] = run + t;
      run += __shfl_sync(kFull, t, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
}

struct Seg {
  int b, h, rg, len, cnt, limit;
  int t0, t1, tiles;
  int start, next;  // of the slab's group, of the stretch after this one
};
template <bool TREE>
__device__ __forceinline__ Seg seg_at(const TcParams& p, int rows_per, const int* pre, int at, int end) {
  Seg s;
  int lo = 0, hi = p.a.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] <= at) lo = mid + 1;
    else hi = mid;
  }
  s.b = lo;
  const int most = p.a.pool.max_blocks * 16;
  s.len = clamped_len(p.a.seq_len, s.b, most, nullptr);
  s.cnt = clamped_count(p.a.count, s.b, p.a.nq);
  int x = at - pre[s.b], span = 1;
  s.rg = 0;
  for (;; ++s.rg) {
    s.limit = group_limit<TREE>(p, rows_per, s.rg, s.len, s.cnt);
    s.tiles = tiles_of(s.limit);
    span = cost_of(s.tiles);
    if (x < span * p.a.Hkv || s.rg + 1 >= p.groups) break;
    x -= span * p.a.Hkv;
  }
  span = max(span, 1);
  s.h = x / span;
  x -= s.h * span;
  s.start = at - x;
  s.t0 = min(x, s.tiles);
  s.t1 = min(s.tiles, x + (end - at));
  s.next = min(end, at + span - x);
  return s;
}

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

// One query row as NT e4m3 terms in the swizzled operand tiles at q (term t at q + 128 D t); returns
// the factor of its scores, log2(e) |scale| 2^e (the sign of `scale` goes into the terms).
template <int D, int NT, typename T>
__device__ __forceinline__ float query_row(const T* src, bool live, float scale, unsigned char* q, int r) {
  uint4 raw[D / 8];
#pragma unroll
  for (int c = 0; c < D / 8; ++c) raw[c] = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float x[16];
    unpack16(Raw16<T>{{raw[2 * c], raw[2 * c + 1]}}, x, src);
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
  }
  const bool odd = !(amax <= 3.402823466e38f);  // an infinity: the row's result is NaN, as the formula's is
  const unsigned u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // amax <= 448 2^e
  e = min(120, max(-120, e));
  if (amax == 0.f || odd) e = 0;
  const float inv = scale < 0.f ? -exp2i(-e) : exp2i(-e);
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float x[16];
    unpack16(Raw16<T>{{raw[2 * c], raw[2 * c + 1]}}, x, src);
    const int at = k_chunk<D>(r, c);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= inv;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t two[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float &a = x[4 * k + 2 * m], &b = x[4 * k + 2 * m + 1];
          two[m] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
          const uint32_t back = codes_half2(two[m]);
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
          a -= f.x;
          b -= f.y;
        }
        w[k] = two[0] | (two[1] << 16);
      }
      *reinterpret_cast<uint4*>(q + 128 * D * t + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return odd ? __uint_as_float(0x7fc00000u) : fabsf(scale) * kLog2e * exp2i(e);
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

// 32 W scores from column t_s of this thread's lane to -infinity where the row (draft i of entry b) does not attend to
// the token; j0: the draft at the first (negative: a token before the drafts).  Their factors are positive, so it hides them.
template <int W>
__device__ __forceinline__ void hide_scores(uint32_t t_s, const TreeMasks& M, int b, int i, bool asks, int cnt, int j0) {
  const uint32_t* m = M.row(b, i);
  uint32_t w[W];
#pragma unroll
  for (int x = 0; x < W; ++x) w[x] = asks ? tree_word(m, M.words, cnt, j0 + 32 * x) : 0u;
#pragma unroll 1
  for (int g = 0; g < W; ++g, t_s += 32) {
    const uint32_t bits = w[0];
#pragma unroll
    for (int x = 1; x < W; ++x) w[x - 1] = w[x];
    if (!__any_sync(kFull, bits != 0xffffffffu)) continue;
    float v[32];
    tqd::tc_ld32(t_s, v);
#pragma unroll
    for (int k = 0; k < 32; ++k) v[k] = bits >> k & 1u ? v[k] : -INFINITY;
    tqd::tc_st32(t_s, v);
  }
}

// query_row for a tree's kernels, which keep their code small: what a block runs once a stretch waits for its
// instructions.  The row is loaded ahead (request), so that it does not wait behind the next tiles' copies; its
// words are then put through 64 (D / 2) columns of tensor memory from t_raw on, so that a loop can take them 16 values at a
// time: put(t, c, w) takes codes 16 c .. of term t, for chunks c in [c0, c1).  The factor is never so small that a scaled
// one of -infinity is not.
template <int D>
struct QueryRow {
  uint4 raw[D / 8];
  __device__ __forceinline__ void request(const void* src, bool live) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) raw[c] = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
  }
};
template <int D, int NT, typename T, typename F>
__device__ __forceinline__ float query_terms(const QueryRow<D>& q, float scale, uint32_t t_raw, int c0, int c1, F put) {
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < D / 16; ++c) {
    float x[16];
    unpack16(Raw16<T>{{q.raw[2 * c], q.raw[2 * c + 1]}}, x, (const T*)nullptr);
#pragma unroll
    for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
    const uint32_t w[8] = {q.raw[2 * c].x, q.raw[2 * c].y, q.raw[2 * c].z, q.raw[2 * c].w,
                           q.raw[2 * c + 1].x, q.raw[2 * c + 1].y, q.raw[2 * c + 1].z, q.raw[2 * c + 1].w};
    st8_async(t_raw + 8 * c, w);
  }
  const bool odd = !(amax <= 3.402823466e38f);  // an infinity: the row's result is NaN, as the formula's is
  const unsigned u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // amax <= 448 2^e
  e = min(120, max(-120, e));
  if (amax == 0.f || odd) e = 0;
  const float inv = scale < 0.f ? -exp2i(-e) : exp2i(-e);
  asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    Raw16<T> raw;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\ntcgen05.wait::ld.sync.aligned;\n"
                 : "=r"(raw.v[0].x), "=r"(raw.v[0].y), "=r"(raw.v[0].z), "=r"(raw.v[0].w), "=r"(raw.v[1].x), "=r"(raw.v[1].y),
                   "=r"(raw.v[1].z), "=r"(raw.v[1].w)
                 : "r"(t_raw + 8 * c) : "memory");
    float x[16];
    unpack16(raw, x, (const T*)nullptr);
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= inv;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float &a = x[2 * k], &b = x[2 * k + 1];
        const uint32_t two = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t back = codes_half2(two);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
        a -= f.x;
        b -= f.y;
        w[k >> 1] = k & 1 ? w[k >> 1] | (two << 16) : two;
      }
      put(t, c, w);
    }
  }
  const float f = fabsf(scale) * kLog2e * exp2i(e);
  return odd ? __uint_as_float(0x7fc00000u) : fmaxf(f, 8.07793567e-28f);  // 2^-90
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
