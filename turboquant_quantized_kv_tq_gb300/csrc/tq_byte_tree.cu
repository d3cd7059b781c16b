// Attention of a tree's drafts over the byte cache on the 5th-generation tensor cores: up to 128 (query, head) rows
// of a slab (batch entry, KV head) at a time, head dims 64 and 128, bf16 and fp16 queries.
//
// The mathematics, the products and the softmax are those of tq_byte_tc.cu, where two tiles of 128 rows take turns
// on one token tile, so that one's softmax runs beside the other's products.  A tree has rarely more than 128 rows
// (16 drafts of 4 heads per KV head: 64), and a lone row tile would leave the tensor cores idle through its softmax.
// Here the two groups of row warps hold the same rows and take turns on the token tiles: group i takes tiles
// n = i (mod 2) with scores S_i, and both add to one O.  So a row has one reference M, which goes from tile to tile
// (through shared memory, posted as soon as a tile's maximum is known); the group that raises it rescales O between
// the products of the tile before and its own.  Each group sums its own l.
// The queries' terms lie in tensor memory, which a second O would fill: a score product reads only its keys from
// shared memory, and the room that they took there holds tiles in flight.  Rows that do not exist cost nothing:
// their warps only pass the barriers.
//
// F = 2, up to 64 rows: a row has two lanes, r and r + 64, one for each half of a tile's tokens.  Each has an M and an O
// of its own; its P holds zeros for the other half's tokens, and the lanes join as partials of a range do.  So all four
// warps of a group work on 64 rows, each on half as many scores.  8 x 32768 tokens, two lanes / one: d = 64, 64 rows 73 / 78 us, 72
// rows (two groups of 64) 132 / 80; d = 128, 32 rows 94 / 94, 64 rows 97 / 95, 96 rows 185 / 99.  More than 128 rows are groups of 128,
// and the pool is read once for each: 256 rows of 8 x 1024 tokens 25 us, of 8 x 32768 215.
//
// Which drafts a row sees matters only in the last tiles: there a pass over the scores puts -infinity where a mask's
// bit is clear, from a window of 32 bits at a time, before the tile's softmax, which is the same for all tiles.
//
// Bits: a query is exact but for what lies below 2^-18 of its row's largest value (the split kernel, up to 8 rows: 2^-39): the
// price of scores on the codes as they are stored, which the tensor cores take at twice fp16's rate and nothing has to unpack.
// A weight is one fp16 number.  Its rounding is what moves a bf16 result from the fp32 form's, by 8e-4 in the 2-norm (bf16's own
// rounding: 1.7e-3); a second term would double the readout's products.  M, l and the joins are fp32, O the tensor cores' fp32
// for up to kMostTiles tiles.
//
// Measured (us, bf16, 32 / 8 heads, 8 x 32768 tokens, pools out of L2): 16 rows 94, 64 rows 97, 128 rows 103; fp16 106 and 121
// for 64 and 128 rows; d = 64 71 and 80.  At d = 128 and up to 64 rows that meets what HBM gives (5.5 TB/s of 6.8).  Otherwise no
// pipe is near its limit (tensor 36 to 42 %, issue 30 to 46 %): the time is the chain of a tile -- scores to registers, maximum,
// P, readout, next scores -- on two row groups.  The code has to stay well below 128 KB (poll, below).
//
// Warps: 0-7 rows, 8-11 V to fp16, 12 K copies, 13 MMA issue, 14 V copies (15 only completes the warpgroup).
#include <atomic>

#include "tq_byte_tc.cuh"

namespace tqb {
namespace {

// tqd::mbar_wait as a loop that stays one: unrolled four times at each of its places it made up 50 of the kernel's 126 KB of
// code, and from 128 KB on every form slowed down, as from an instruction cache of that size.  Unrolled / here: 64 unlike
// lengths, 91 rows 45 / 35 us; d = 64, 192 rows of 16 x 16384 tokens 55 / 47; 64 and 128 rows of 8 x 32768 tokens 101 / 98 and 119 /
// 112 (135 KB of code: 102, 147).
__device__ __forceinline__ bool poll(uint32_t bar, uint32_t parity) {
#pragma unroll 1
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    if (done) return true;
  }
  return false;
}

template <int D>
struct Plan {
  static constexpr int BLK = 32 * D + 32;
  static constexpr int TILE = 128 * D;                            // bytes of a tile's codes
  static constexpr int FIRST = 6;                                 // blocks of a tile in the first part of P
  static constexpr int KS = 4;                                    // K stages: scores run two tiles ahead
  static constexpr int VS = D == 128 ? 5 : 8;                     // stages of V's codes: copies take 2 us under load
  static constexpr int VB = 16 * D + 16;                          // V's codes of a block and the scales behind them: one copy
  static constexpr int SC = 4;                                    // stages of scales, [block] (K scale, e, 2^-e, -)
  static constexpr int KR = 0, V16 = KR + KS * TILE, VR = V16 + 4 * TILE;
  static constexpr int SCALES = VR + VS * 8 * VB, REF = SCALES + SC * 128, SUM = REF + 2 * 128 * 4, STRETCH = SUM + 2 * 128 * 4;
  static constexpr int TOP = STRETCH + 8 * 2 * 40;                // [row warp][turn]
  static constexpr int SWAP = TOP + 128 * 4, BARS = SWAP + 2 * 8 * 128 * 4;  // halves of rows that two lanes share
  static constexpr int LEN = BARS + 496, PRE = LEN + TQ_MAX_BATCH * 8;
  static constexpr int T_O = 256, T_Q = 384;                      // columns of O and of the queries' terms (S_i at 128 i)
  static constexpr int SMEM = PRE + (TQ_MAX_BATCH + 1) * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr int PART = 128 * (D + 2);                      // floats of a partial: M[128], l[128], O[D / 4][128][4]
  static constexpr int CARRY = 2 * 256;                           // and of a block's (M, l) between the stretches of a slab, by row thread
};
// (P_FULL: part h of group i at 2 i + h)
enum Bar { K_FULL = 0, K_EMPTY = 8, VR_FULL = 16, VR_EMPTY = 24, V_FULL = 32, V_EMPTY = 34, S_FULL = 36, O_DONE = 38, REF_SET = 40,
           P_FULL = 42, SC_EMPTY = 46, SC_READY = 50, Q_FULL = 54, SUM_SET = 55, OUT_READ = 56, SWAPPED = 57, BAR_COUNT = 61 };
static_assert(8 * BAR_COUNT + 4 <= 496, "barriers and the tensor-memory slot");

// Virtual tiles of a row group: what a range costs beside its tiles (4 / 6 / 8 / 12: a batch of 64 unlike lengths, 91 rows
// 36 / 35 / 36 / 40 us; of 32, 64 rows 39 / 36 / 36 / 36; 8 x 32768 tokens 98 / 97 / 97 / 97).
constexpr int kTreeGroupCost = 6;
__device__ __forceinline__ int tree_cost(int tiles) { return tiles > 0 ? tiles + kTreeGroupCost : 0; }

// The plan: all live row groups of an entry cover its whole sequence.  len[b]: (tokens, drafts).
template <int ROWS>
__device__ __forceinline__ int live_groups(const TcParams& p, int2 len) { return len.x > 0 ? (len.y * p.G + ROWS - 1) / ROWS : 0; }

// Costs before each entry (order: entry, row group, head), and the entries' lengths; written by warp 0.
template <int ROWS>
__device__ __forceinline__ void fill_tree_plan(const TcParams& p, int* pre, int2* len, int32_t* err) {
  const int lane = threadIdx.x & 31, most = p.a.pool.max_blocks * 16;
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.a.B; b0 += 32) {
      const int b = b0 + lane;
      int t = 0;
      if (b < p.a.B) {
        const int2 x = make_int2(clamped_len(p.a.seq_len, b, most, err), clamped_count(p.a.count, b, p.a.nq));
        len[b] = x;
        t = live_groups<ROWS>(p, x) * p.a.Hkv * tree_cost(tiles_of(x.x));
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

// A stretch of a slab's tiles [t0, t1), the first from cost `at` (< end) on that has a tile; t0 = t1: there is none.
// The tensor cores' sum O truncates at every product (16 tokens) that it takes in: over 100000 tokens of values with mean 1 it
// came out 4.1e-4 low (F = 2, where half of a lane's products are of zeros: 1.9e-4), twice fp16's rounding.  So a block's part
// of a slab is cut into stretches of at most kMostTiles, which join in fp32 in its place for a partial.  1024 products lose
// 2^-14 of an evenly growing sum at most; measured 4.1e-5 and 1.9e-5.  A cut costs the block a stretch's start and end (64 / 128 /
// 256 / none: 152 slabs of 49152 tokens, 64 rows 332 / 308 / 304 / 295 us, 128 rows 352 / 334 / 331 / 324; 8 x 32768 tokens with
// 64 rows, 108 tiles a block, 103 / 97 / 97 / 97).
constexpr int kMostTiles = 128;
struct Stretch {
  int b, h, rg, len, cnt;
  int t0, t1, tiles;
  int start, next;  // of the slab's group, of the stretch after this one
};
static_assert(sizeof(Stretch) <= 40, "its place in shared memory");
// The entry that holds cost `at` (< the total).
__device__ __forceinline__ int entry_at(const int* pre, int B, int at) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] <= at) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}
// b: the entry to look from.
__device__ __forceinline__ Stretch stretch_from(const TcParams& p, const int* pre, const int2* len, int b, int at, int end) {
  Stretch s = {};
  while (at < end) {
    while (pre[b + 1] <= at) ++b;
    const int2 n = len[b];
    const int tiles = tiles_of(n.x), span = tree_cost(tiles), x = at - pre[b], k = x / span, y = x - k * span;
    if (y < tiles) {
      const int rg = k / p.a.Hkv, left = min(tiles - y, end - at);
      int take = left, next = min(end, at + span - y);
      if (left > kMostTiles) {
        take = left < 2 * kMostTiles ? (left + 1) >> 1 : kMostTiles;
        next = at + take;
      }
      return Stretch{b, k - rg * p.a.Hkv, rg, n.x, n.y, y, y + take, tiles, at - y, next};
    }
    at += span - y;
  }
  s.next = end;
  return s;
}

// Swizzled K-major operand of rows of D codes: 128-byte swizzle in groups of 1024 bytes, 64-byte in 512.
template <int D>
__device__ __forceinline__ uint64_t sdesc_codes(uint32_t addr) {
  if constexpr (D == 128) return sdesc128(addr);
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (1ull << 16) | ((uint64_t)(512 >> 4) << 32) | (1ull << 46) | (4ull << 61);
}
__host__ __device__ constexpr uint32_t idesc(int n) { return (1u << 4) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24); }  // M = 128

// D = A B (+ D) on 8-bit floats with A in tensor memory (row i in lane i, four values to a column).
__device__ __forceinline__ void mma_f8_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n}\n"
      :: "r"(d_tmem), "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void st4_async(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}

// S of the tile in K buffer ST, for group ST % 2.
template <int D, int NT, int ST>
__device__ __forceinline__ void issue_scores(uint32_t sb) {
  using L = Plan<D>;
  constexpr int i = ST & 1;
  const uint64_t k = sdesc_codes<D>(sb + L::KR + ST * L::TILE);
  if (elected()) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < D / 32; ++j) mma_f8_ta(128 * i, L::T_Q + t * (D / 4) + 8 * j, k + 2 * j, idesc(kTok), t + j > 0);
    tqd::tc_commit(sb + L::BARS + 8 * (S_FULL + i));
    tqd::tc_commit(sb + L::BARS + 8 * (K_EMPTY + ST));
  }
  __syncwarp();
}
template <int D, int NT>
__device__ __forceinline__ void issue_scores(uint32_t sb, uint32_t n) {
  static_assert(Plan<D>::KS == 4, "one case a buffer");
  switch (n & 3) {
    case 0: return issue_scores<D, NT, 0>(sb);
    case 1: return issue_scores<D, NT, 1>(sb);
    case 2: return issue_scores<D, NT, 2>(sb);
    default: return issue_scores<D, NT, 3>(sb);
  }
}
// Part h of O += P_i V of the tile in V buffer i (accumulate: not the first tile of a stretch).  F = 1: blocks
// [0, FIRST), then the others; F = 2: all at once, a row's lanes end together.
template <int D, int F, int i, int h>
__device__ __forceinline__ void issue_readout(uint32_t sb, bool accumulate) {
  using L = Plan<D>;
  constexpr int k0 = h == 0 ? 0 : L::FIRST, k1 = h == 0 && F == 1 ? L::FIRST : 8;
  const uint64_t v = sdesc128(sb + L::V16 + i * 2 * L::TILE);
  if (elected()) {
#pragma unroll
    for (int k = k0; k < k1; ++k)
      tqd::tc_mma_f16_ta(L::T_O, 128 * i + 8 * k, v + (uint64_t)((k >> 2) * (L::TILE >> 4) + 2 * (k & 3)), idesc(D),
                         accumulate || k > 0);
    if (k1 == 8) {
      tqd::tc_commit(sb + L::BARS + 8 * (O_DONE + i));
      tqd::tc_commit(sb + L::BARS + 8 * (V_EMPTY + i));
    }
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t pack2(const __nv_bfloat16*, float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(const __half*, float a, float b) { return tqd::pack_half2(a, b); }
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack2(p, v.x, v.y), pack2(p, v.z, v.w));
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack2(p, v[0], v[1]), pack2(p, v[2], v[3]), pack2(p, v[4], v[5]), pack2(p, v[6], v[7]));
}

// 32 W scores from column t_s of this thread's lane to -infinity where the row (draft i of entry b) does not attend to
// the token; j0: the draft at the first (negative: a token before the drafts).  Their factors, a row's (2^-90 at least) times
// a block's scale (2^-30 at least), are positive normal numbers, so it hides them.
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

// A query row as NT e4m3 terms.  The code is kept small: what a block runs once a stretch waits for its instructions.
// The row is loaded ahead (request), so that it does not wait behind the next tiles' copies; its words are then put through
// D / 2 columns of tensor memory from t_raw on, so that a loop can take them 16 values at a time: put(t, c, w) takes codes
// 16 c .. of term t, for chunks c in [c0, c1).  Returned: the factor of the row's scores, log2(e) |scale| 2^e (the sign of
// `scale` goes into the terms), never so small that a scaled one of -infinity is not.  A row with an infinity is all NaN
// codes (a NaN is one by itself): what the row attends to makes it NaN, as the formula does, and where that is nothing it is zeros.
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
  const bool odd = !(amax <= 3.402823466e38f);  // an infinity
  const unsigned u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // amax <= 448 2^e
  e = min(120, max(-120, e));
  if (amax == 0.f || odd) e = 0;
  const float inv = odd ? __uint_as_float(0x7fc00000u) : scale < 0.f ? -exp2i(-e) : exp2i(-e);
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
  return fmaxf(fabsf(scale) * kLog2e * exp2i(e), 8.07793567e-28f);  // 2^-90
}

template <int D, int NT, int F, typename T>
__global__ void __launch_bounds__(kThreads, 1) tree_kernel(const TcParams p) {
  using L = Plan<D>;
  constexpr int ROWS = 128 / F;     // rows of a group: each has F lanes,
  constexpr int NB = 8 / F;         // each of which takes this many blocks of a tile
  extern __shared__ __align__(1024) unsigned char sm[];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const AttnArgs& A = p.a;
  const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t sb = (uint32_t)__cvta_generic_to_shared(sm);
  const uint32_t bars = sb + L::BARS;
  auto bar = [&](int kind, int i) { return bars + 8 * (kind + i); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + L::BARS + 8 * BAR_COUNT);
  int* pre = reinterpret_cast<int*>(sm + L::PRE);
  int2* lens = reinterpret_cast<int2*>(sm + L::LEN);
  if (sb & 1023u) {  // the swizzled operands need it (the plan gives it)
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    if (threadIdx.x == 0) {
      p.heads[blockIdx.x].last = -1;
      if (A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_SMEM_PLAN);
    }
    return;
  }
  if (warp == 13) tqd::tc_alloc((uint32_t)__cvta_generic_to_shared(slot), 512);
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      tqd::mbar_init(bar(V_FULL, i), 4);
      tqd::mbar_init(bar(V_EMPTY, i), 1);
      tqd::mbar_init(bar(S_FULL, i), 1);
      tqd::mbar_init(bar(P_FULL, 2 * i), 128);
      tqd::mbar_init(bar(P_FULL, 2 * i + 1), 128);
      tqd::mbar_init(bar(O_DONE, i), 1);
      tqd::mbar_init(bar(REF_SET, i), 128);
      tqd::mbar_init(bar(SWAPPED, 2 * i), 64);
      tqd::mbar_init(bar(SWAPPED, 2 * i + 1), 64);
    }
    for (int i = 0; i < L::KS; ++i) {
      tqd::mbar_init(bar(K_FULL, i), 1);
      tqd::mbar_init(bar(K_EMPTY, i), 1);
    }
    for (int i = 0; i < L::VS; ++i) {
      tqd::mbar_init(bar(VR_FULL, i), 1);
      tqd::mbar_init(bar(VR_EMPTY, i), 4);
    }
    for (int i = 0; i < L::SC; ++i) {
      tqd::mbar_init(bar(SC_EMPTY, i), 4);
      tqd::mbar_init(bar(SC_READY, i), 1);
    }
    tqd::mbar_init(bar(Q_FULL, 0), 256);
    tqd::mbar_init(bar(SUM_SET, 0), 256);
    tqd::mbar_init(bar(OUT_READ, 0), 256);
    tqd::fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;\n" ::: "memory");  // (what is above may run beside the kernel before this one)
  fill_tree_plan<ROWS>(p, pre, lens, blockIdx.x == 0 ? A.pool.err : nullptr);
  tqd::tc_fence_before();
  __syncthreads();
  tqd::tc_fence_after();
  // all 512 columns are this block's: they begin at column 0, lane 0
  const bool whole_tmem = *slot == 0;
  const int total = pre[A.B], per = range_of(total, p.grid);
  const int begin = min(total, (int)blockIdx.x * per), end = min(total, begin + per);
  const int b_first = entry_at(pre, A.B, begin);

  bool ok = whole_tmem;  // cleared by a wait that gave up: the role stops working and ends
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (ok && !poll(b, parity)) ok = false;
    return ok;
  };

  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRowRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
  if (warp < 8) {
    // ---- rows: group i takes the tiles n = i (mod 2) of the block's sequence
    const int i = warp >> 2, r = (warp & 3) * 32 + lane, rr = r % ROWS, part = r / ROWS;  // lane r: part `part` of row rr
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = lanes + 128 * i, t_o = lanes + L::T_O;
    const uint32_t t_mine = t_s + 16 * NB * part, t_p = t_s + 8 * NB * part;  // the lane's scores and its part of P
    float* refs = reinterpret_cast<float*>(sm + L::REF);  // [tile % 2][lane]: M from this tile on
    float* sums = reinterpret_cast<float*>(sm + L::SUM);  // [group][lane]
    float* tops = reinterpret_cast<float*>(sm + L::TOP);  // [lane]
    float* swap = reinterpret_cast<float*>(sm + L::SWAP) + i * 8 * 128;
    // groups without a live row: zeros, spread over the grid
    for (int k = blockIdx.x; k < A.B * p.groups; k += gridDim.x) {
      const int b = k / p.groups, rg = k - b * p.groups, row = rg * ROWS + rr;
      if (rg < live_groups<ROWS>(p, lens[b]) || row >= p.rows) continue;
      for (int h = part; h < A.Hkv; h += F) {
        uint4* o = reinterpret_cast<uint4*>(out_row<D, T>(p, b, h, row)) + i * (D / 16);
        for (int c = 0; c < D / 16; ++c) o[c] = make_uint4(0u, 0u, 0u, 0u);
      }
    }
    uint32_t n = 0, segs = 0, swaps = 0;  // tiles, stretches and phases of SWAPPED so far
    int t0 = 0, t1 = 0, qi = 0;
    bool headed = false, live = false, asks = false;
    QueryRow<D> q;
    // The stretches wait in shared memory (a row's scores leave few registers): each is looked for while the one before
    // it runs, and its queries are requested before that one's sums are written.
    auto stretch = [&](uint32_t k) { return reinterpret_cast<Stretch*>(sm + L::STRETCH + (warp * 2 + (k & 1)) * 40); };
    auto look = [&](uint32_t k, int b, int at) {
      const Stretch s = stretch_from(p, pre, lens, b, at, end);
      if (lane == 0) *stretch(k) = s;
      __syncwarp();
    };
    auto begin_stretch = [&](uint32_t k) {
      const Stretch& s = *stretch(k);
      t0 = s.t0;
      t1 = s.t1;
      const int row = s.rg * ROWS + rr;
      live = row < p.rows;
      qi = live ? row / p.G : 0;
      // (rows past the count are zero queries whose sums are dropped, so that they hide nothing)
      asks = live && qi < s.cnt;
      const int hd = s.h * p.G + (live ? row - qi * p.G : 0);
      q.request(reinterpret_cast<const T*>(A.q.p) + s.b * A.q.sb + qi * A.q.st + hd * A.q.sh, asks);
      return t0 < t1;
    };
    look(0, b_first, begin);
    bool more = begin_stretch(0);
    while (more && ok) {
      const bool idle = !__any_sync(kFull, asks);  // (uniform over the two groups' warps of the same rows)
      // (each group converts half of the coordinates)
      const float f = query_terms<D, NT, T>(q, A.scale, t_s, i * (D / 32), (i + 1) * (D / 32), [&](int t, int c, const uint32_t* w) {
        st4_async(lanes + L::T_Q + t * (D / 4) + 4 * c, w);
      });
      asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
      tqd::tc_fence_before();
      tqd::tc_mbar_arrive(bar(Q_FULL, 0));
      look(segs + 1, stretch(segs)->b, stretch(segs)->next);
      float M = -INFINITY, l = 0.f;  // l under the reference M
      const int t_first = t0 + (int)((n ^ (uint32_t)i) & 1u), drafts = stretch(segs)->len - stretch(segs)->cnt;  // drafts: the first one's position
      // one tile; false: a wait gave up
      auto tile = [&](int t) {
        const uint32_t g_tile = n + (uint32_t)(t - t0), turn = g_tile >> 1;
        float m_old = -INFINITY;
        const int ss = g_tile % L::SC;
        // (scales and the reference are waited for before the scores, and below the next keys before the readout: a wait that is
        // over takes time too.  Behind / before: 8 x 32768 tokens, 128 rows 110 / 103 us, fp16 123 / 121, 64 rows 97 / 97; d = 64, 64 rows 78 / 71.)
        if (!wait(bar(SC_READY, ss), (g_tile / L::SC) & 1)) return false;
        const float4* sc = reinterpret_cast<const float4*>(sm + L::SCALES + 128 * ss) + NB * part;
        float a[NB], e[NB], v[2][32];
#pragma unroll
        for (int g = 0; g < NB; ++g) {
          const float2 x = *reinterpret_cast<const float2*>(sc + g);
          a[g] = f * x.x;
          e[g] = x.y;
        }
        if (t > t0 && !idle) {
          if (!wait(bar(REF_SET, i ^ 1), ((g_tile - 1) >> 1) & 1)) return false;
          m_old = refs[128 * (i ^ 1) + r];
        }
        if (!wait(bar(S_FULL, i), turn & 1)) return false;
        if (idle) {
          tqd::tc_mbar_arrive(bar(REF_SET, i));
          tqd::tc_mbar_arrive(bar(P_FULL, 2 * i));
          if (F == 1) tqd::tc_mbar_arrive(bar(P_FULL, 2 * i + 1));
          if (lane == 0) tqd::tc_mbar_arrive(bar(SC_EMPTY, ss));
          return true;
        }
        tqd::tc_fence_after();
        const int j0 = kTok * t + 16 * NB * part - drafts;  // the draft at the lane's first score
        if (j0 + 16 * NB > 0) hide_scores<NB / 2>(t_mine, A.tree, stretch(segs)->b, qi, asks, stretch(segs)->cnt, j0);
        // A whole row's scores are read twice, 32 at a time, for the maximum and for P: held from one to the other they
        // left the warps too few registers (138 us for 8 x 32768 tokens and 64 rows).  P takes the first half of the columns:
        // block g's lie at 8 g, below the scores of block g that it comes from.
        ld32_async(t_mine, v[0]);
        if (F == 2) ld32_async(t_mine + 32, v[1]);
        float top = -INFINITY;
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
          ld_wait<32>(v[c & 1]);
          if (F == 1) ld32_async(t_mine + 32 * ((c + 1) & 3), v[(c + 1) & 1]);
          top = fmaxf(top, fmaxf(block_top<false>(v[c & 1], 0, a[2 * c], e[2 * c]), block_top<false>(v[c & 1] + 16, 0, a[2 * c + 1], e[2 * c + 1])));
        }
        if (F == 2) {  // the tokens of the row's other lane count for nothing here
          const uint32_t none[8] = {};
#pragma unroll
          for (int g = 0; g < NB; ++g) st8_async(t_s + 8 * (NB * (1 - part) + g), none);
        }
        const bool raise = top > m_old + kSlack;
        const float m_new = raise ? top - kTop : m_old;
        refs[128 * i + r] = m_new;
        tqd::tc_mbar_arrive(bar(REF_SET, i));
        if (M != m_new) {
          l *= ex2(M - m_new);
          M = m_new;
        }
        if (t > t0 && __any_sync(kFull, raise)) {
          const float cor = raise ? ex2(m_old - m_new) : 1.f;
          if (!wait(bar(O_DONE, i ^ 1), ((g_tile - 1) >> 1) & 1)) return false;
          tqd::tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            float o[16];
            uint32_t w[16];
            tqd::tc_ld16(t_o + 16 * c, o);
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * cor);
            tqd::tc_st16(t_o + 16 * c, w);
          }
        }
        const float mr = M == -INFINITY ? 0.f : M;
        float z[NB];
#pragma unroll
        for (int g = 0; g < NB; ++g) z[g] = sc[g].z;
#pragma unroll
        for (int c = 0; c < NB / 2; ++c) {
          if (F == 1) {
            ld_wait<32>(v[c & 1]);
            if (c < 3) ld32_async(t_mine + 32 * (c + 1), v[(c + 1) & 1]);
          }
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int g = 2 * c + h;
            uint32_t w[8];
            const float sum = block_p<false>(v[c & 1] + 16 * h, 0, a[g], e[g] - mr, w);
            l = fmaf(sum, z[g], l);
            st8_async(t_p + 8 * g, w);
          }
          if ((F == 1 && 2 * c + 2 == L::FIRST) || 2 * c + 2 == NB) {
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            tqd::tc_fence_before();
            tqd::tc_mbar_arrive(bar(P_FULL, 2 * i + (F == 1 && c == 3)));
          }
        }
        __syncwarp();
        if (lane == 0) tqd::tc_mbar_arrive(bar(SC_EMPTY, ss));
        return true;
      };
      for (int t = t_first; t < t1; t += 2) {
        if (!tile(t)) break;
      }
      if (!ok) break;
      // the next stretch's queries are requested before this one's last products are waited for
      const uint32_t tiles = (uint32_t)(t1 - t0);
      const bool was_live = live, asked = asks;
      more = begin_stretch(segs + 1);
      // Every product of the stretch is done with its last tile's.  (The tile before it is waited for first: a wait for a
      // phase tells nothing while the barrier is two phases behind.)
      const uint32_t last = n + tiles - 1;
      if (last > n && !wait(bar(O_DONE, (last - 1) & 1), ((last - 1) >> 1) & 1)) break;
      if (!wait(bar(O_DONE, last & 1), (last >> 1) & 1)) break;
      n = last + 1;
      tqd::tc_fence_after();
      const float top = idle ? -INFINITY : refs[128 * (last & 1) + r];
      if (M != top) l *= ex2(M - top);  // (the other group raised it last; a group without a tile has l = 0)
      sums[128 * i + r] = asked ? l : 0.f;
      if (i == 0) tops[r] = top;
      tqd::tc_mbar_arrive(bar(SUM_SET, 0));
      if (!wait(bar(SUM_SET, 0), segs & 1)) break;
      const Stretch now = *stretch(segs++);
      // each group takes half of the coordinates; a row's lanes join
      float sum = sums[r] + sums[128 + r], most = top, mine = 1.f;  // mine: the weight of this lane's sums
      if (F == 2) {
        const float other = tops[r ^ 64];
        most = fmaxf(top, other);
        const float ref = most == -INFINITY ? 0.f : most;
        mine = ex2(top - ref);
        sum = fmaf(sum, mine, (sums[r ^ 64] + sums[128 + (r ^ 64)]) * ex2(other - ref));
      }
      // the block's part of the slab: tiles [max(0, begin - start), stop)
      const int stop = min(now.tiles, end - now.start);
      const bool inside = now.start >= begin && stop == now.tiles, done = now.t1 == stop, whole = inside && done;
      // (a slab that lies inside the range uses the place of the last one, which comes after it)
      float* partial = p.part + (2ll * blockIdx.x + (now.start <= begin ? 0 : 1)) * L::PART;
      float2* carry = reinterpret_cast<float2*>(p.part + 2ll * p.grid * L::PART + (long long)blockIdx.x * L::CARRY) + threadIdx.x;
      // [4 coordinates][row]: a warp writes 512 bytes in a row (as rows of their own they took 6000 cycles)
      float4* to = reinterpret_cast<float4*>(partial + 256) + rr;
      if (now.t0 > max(0, begin - now.start) && !idle) {  // the sums of the stretches before
        const float2 x = *carry;
        const float all = fmaxf(most, x.x), ref = all == -INFINITY ? 0.f : all, w = ex2(most - ref), before = ex2(x.x - ref);
        sum = fmaf(sum, w, x.y * before);
        most = all;
        mine *= w;
#pragma unroll 1
        for (int c = i * (D / 8); c < (i + 1) * (D / 8); c += 4) {
          float o[16];
          uint32_t y[16];
          tqd::tc_ld16(t_o + 4 * c, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 z = part == 0 ? to[(c + k) * 128] : make_float4(0.f, 0.f, 0.f, 0.f);
            y[4 * k] = __float_as_uint(fmaf(z.x, before, o[4 * k] * mine));
            y[4 * k + 1] = __float_as_uint(fmaf(z.y, before, o[4 * k + 1] * mine));
            y[4 * k + 2] = __float_as_uint(fmaf(z.z, before, o[4 * k + 2] * mine));
            y[4 * k + 3] = __float_as_uint(fmaf(z.w, before, o[4 * k + 3] * mine));
          }
          tqd::tc_st16(t_o + 4 * c, y);
        }
        mine = 1.f;
      }
      if (!done) *carry = make_float2(most, sum);
      if (whole) mine *= sum > 0.f || sum != sum ? 1.f / sum : 0.f;
      T* out = out_row<D, T>(p, now.b, now.h, was_live ? now.rg * ROWS + rr : 0);
      if (!whole && i == 0 && part == 0) {
        partial[rr] = most;
        partial[128 + rr] = sum;
      }
      if (whole || !idle) {  // (a partial's rows without a sum are left out by the join)
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          const int col = i * (D / 2) + 16 * c;
          float v[16];
          tqd::tc_ld16(t_o + col, v);
          // (rows that do not ask may hold NaN: what lies behind the tokens is hidden from the others only)
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = asked ? v[k] * mine : 0.f;
          if constexpr (F == 1) {
            if (whole) {
              if (was_live) store16(out + col, v);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k) to[(col / 4 + k) * 128] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            }
          } else {  // lane 0 of a row finishes the first eight coordinates, lane 1 the others; the two warps meet
            const uint32_t met = bar(SWAPPED, 2 * i + (warp & 1));
            if (c > 0 && !wait(met, (swaps - 1) & 1)) break;  // (the last values were read)
#pragma unroll
            for (int k = 0; k < 8; ++k) swap[128 * k + r] = part ? v[k] : v[8 + k];
            tqd::tc_mbar_arrive(met);
            if (!wait(met, swaps++ & 1)) break;
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = (part ? v[8 + k] : v[k]) + swap[128 * k + (r ^ 64)];
            tqd::tc_mbar_arrive(met);
            ++swaps;
            if (whole) {
              if (was_live) store8(out + col + 8 * part, x);
            } else {
#pragma unroll
              for (int k = 0; k < 2; ++k) to[(col / 4 + 2 * part + k) * 128] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
            }
          }
        }
      }
      tqd::tc_fence_before();
      tqd::tc_mbar_arrive(bar(OUT_READ, 0));  // (the next stretch's first products overwrite the sums)
      if (threadIdx.x == 0 && done && !inside && now.start >= begin) {  // this range's last slab goes on past it
        p.heads[blockIdx.x] = JoinHead{(now.start + now.tiles - 1) / per, now.start == begin ? 0 : 1, now.b, now.h, now.rg};
        headed = true;
      }
    }
    if (threadIdx.x == 0 && !headed) p.heads[blockIdx.x].last = -1;
  } else if (warp < 12) {
    // ---- V codes to fp16, K-major [coordinate][token], 64 tokens per 128-byte row
    uint32_t n = 0;
    for (Stretch s = stretch_from(p, pre, lens, b_first, begin, end); s.t0 < s.t1 && ok; s = stretch_from(p, pre, lens, s.b, s.next, end)) {
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int st = n & 1, vs = n % L::VS, ss = n % L::SC;
        if (!wait(bar(VR_FULL, vs), (n / L::VS) & 1)) break;
        if (warp == 8) {
          if (n >= L::SC && !wait(bar(SC_EMPTY, ss), (n / L::SC - 1) & 1)) break;
          if (lane < 8) {
            float2 x = *reinterpret_cast<const float2*>(sm + L::VR + (vs * 8 + lane) * L::VB + 16 * D);
            // Within an append's range, 2^-30 to 2^30, whatever stands there: a block behind the tokens, or of hidden drafts that were
            // never appended, may hold anything (in a zeroed pool 0, and 0 times a hidden score of -infinity is NaN).
            x.x = fminf(fmaxf(x.x, 9.31322575e-10f), 1073741824.f);
            x.y = fminf(fmaxf(x.y, 9.31322575e-10f), 1073741824.f);
            const int e = log2i(x.y);
            *reinterpret_cast<float4*>(sm + L::SCALES + 128 * ss + 16 * lane) =
                make_float4(x.x, (float)e, exp2i(max(-126, min(126, -e))), 0.f);
          }
          __syncwarp();
          if (lane == 0) tqd::tc_mbar_arrive(bar(SC_READY, ss));
        }
        if (n >= 2 && !wait(bar(V_EMPTY, st), ((n >> 1) - 1) & 1)) break;
        uint4 raw[2][D / 32];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int m = 0; m < D / 32; ++m)
            raw[k][m] = *reinterpret_cast<const uint4*>(sm + L::VR + (vs * 8 + (warp - 8) + 4 * k) * L::VB + 16 * (lane + 32 * m));
        if (kTok * (t + 1) > s.len - s.cnt) {  // tokens behind the last become zeros, and NaN codes (of hidden drafts never appended)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int have = s.len - kTok * t - 16 * ((warp - 8) + 4 * k);
            uint32_t keep[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              keep[u] = (2 * u < have ? 0xffu : 0u) | (2 * u + 1 < have ? 0xff00u : 0u) | (2 * u + 8 < have ? 0xff0000u : 0u) |
                        (2 * u + 9 < have ? 0xff000000u : 0u);
#pragma unroll
            for (int m = 0; m < D / 32; ++m) {
              raw[k][m].x = without_nans(raw[k][m].x & keep[0]);
              raw[k][m].y = without_nans(raw[k][m].y & keep[1]);
              raw[k][m].z = without_nans(raw[k][m].z & keep[2]);
              raw[k][m].w = without_nans(raw[k][m].w & keep[3]);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          unsigned char* dst = sm + L::V16 + st * 2 * L::TILE + k * L::TILE;
#pragma unroll
          for (int m = 0; m < D / 32; ++m) {
            const int d = lane + 32 * m, c = 2 * (warp - 8);
            uint32_t w[8];
            codes_half4(raw[k][m].x, w[0], w[1]);
            codes_half4(raw[k][m].y, w[2], w[3]);
            codes_half4(raw[k][m].z, w[4], w[5]);
            codes_half4(raw[k][m].w, w[6], w[7]);
            *reinterpret_cast<uint4*>(dst + d * 128 + ((c ^ (d & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + d * 128 + (((c + 1) ^ (d & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        tqd::tc_fence_smem();
        __syncwarp();
        if (lane == 0) {
          tqd::tc_mbar_arrive(bar(VR_EMPTY, vs));
          tqd::tc_mbar_arrive(bar(V_FULL, st));
        }
      }
    }
  } else if (warp != 13) {
    // ---- copies: warp 12 the K codes, 14 the V codes and scales.  (A warp takes some 80 cycles a copy: one for
    // both, and copies of the scales beside them, took 2000 cycles a tile and bounded the kernel.)
    const bool keys = warp == 12;
    uint32_t n = 0;
    for (Stretch s = stretch_from(p, pre, lens, 0, warp == 15 ? end : begin, end); s.t0 < s.t1 && ok;
         s = stretch_from(p, pre, lens, s.b, s.next, end)) {
      const int blocks = (s.len + 15) >> 4;
      auto entries = [&](int t) { return 8 * t + lane < blocks ? page_entry(A.pool, s.b, 8 * t + lane) : 0; };
      int ahead = entries(s.t0), page = 0;  // of four tiles, requested four tiles before their use
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int u = (t - s.t0) & 3, j = lane & 7, nb = min(8, blocks - 8 * t);
        if (u == 0) {
          page = checked_page(A.pool, ahead);
          ahead = entries(t + 4);
        }
        const int pg = __shfl_sync(kFull, page, 8 * u + j);
        const unsigned char* blk = A.pool.base + pool_block(A.pool, pg, s.h) * L::BLK;
        if (keys) {
          const int st = n % L::KS;
          if (n >= L::KS && !wait(bar(K_EMPTY, st), (n / L::KS - 1) & 1)) break;
          if (lane == 0) tqd::mbar_arrive_expect_tx(bar(K_FULL, st), nb * 16 * D);
          __syncwarp();
          if (lane < nb) tqd::bulk_g2s(sb + L::KR + st * L::TILE + j * 16 * D, blk, 16 * D, bar(K_FULL, st));
        } else {
          const int st = n % L::VS;
          if (n >= L::VS && !wait(bar(VR_EMPTY, st), (n / L::VS - 1) & 1)) break;
          if (lane == 0) tqd::mbar_arrive_expect_tx(bar(VR_FULL, st), nb * L::VB);
          __syncwarp();
          if (lane < nb) tqd::bulk_g2s(sb + L::VR + (st * 8 + j) * L::VB, blk + 16 * D, L::VB, bar(VR_FULL, st));
        }
        __syncwarp();
      }
    }
    // every copy has landed before the block gives up its shared memory
    if (keys)
      for (uint32_t k = n > L::KS ? n - L::KS : 0; k < n; ++k) poll(bar(K_FULL, k % L::KS), (k / L::KS) & 1);
    else
      for (uint32_t k = n > L::VS ? n - L::VS : 0; k < n; ++k) poll(bar(VR_FULL, k % L::VS), (k / L::VS) & 1);
  } else if (warp == 13) {
    // ---- MMA issue, from operands that are constants of the stage
    uint32_t n = 0, segs = 0;
    for (Stretch s = stretch_from(p, pre, lens, b_first, begin, end); s.t0 < s.t1 && ok; s = stretch_from(p, pre, lens, s.b, s.next, end)) {
      const uint32_t tiles = (uint32_t)(s.t1 - s.t0);
      if (!wait(bar(Q_FULL, 0), segs & 1)) break;
      for (uint32_t k = 0; k < min(2u, tiles); ++k) {
        if (!wait(bar(K_FULL, (n + k) % L::KS), ((n + k) / L::KS) & 1)) break;
        tqd::tc_fence_after();
        issue_scores<D, NT>(sb, n + k);
      }
      if (segs && !wait(bar(OUT_READ, 0), (segs - 1) & 1)) break;
      ++segs;
      for (uint32_t k = 0; k < tiles && ok; ++k) {
        const uint32_t g = n + k;
        if (k + 2 < tiles && !wait(bar(K_FULL, (g + 2) % L::KS), ((g + 2) / L::KS) & 1)) break;
        if (!wait(bar(V_FULL, g & 1), (g >> 1) & 1)) break;
        if (!wait(bar(P_FULL, 2 * (g & 1)), (g >> 1) & 1)) break;
        tqd::tc_fence_after();
        if (g & 1) issue_readout<D, F, 1, 0>(sb, k > 0);
        else issue_readout<D, F, 0, 0>(sb, k > 0);
        if constexpr (F == 1) {
          if (!wait(bar(P_FULL, 2 * (g & 1) + 1), (g >> 1) & 1)) break;
          tqd::tc_fence_after();
          if (g & 1) issue_readout<D, F, 1, 1>(sb, true);
          else issue_readout<D, F, 0, 1>(sb, true);
        }
        if (k + 2 < tiles) issue_scores<D, NT>(sb, g + 2);
      }
      n += tiles;
    }
  }
  if (!ok && lane == 0 && A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_WAIT_TIMEOUT);
  tqd::tc_fence_before();
  __syncthreads();  // (the rows waited for every readout, so every MMA has completed)
  if (warp == 13) {
    tqd::tc_fence_after();
    tqd::tc_dealloc(*slot, 512);
  }
}

// join_kernel for the partials of tree_kernel: a thread takes four coordinates of a row, rows beside each other in a
// warp, as the partials hold them.  Rows that did not ask have no sum, and whatever lies in their place is left out.
constexpr int kJoinThreads = 256;
template <int D, int F, typename T>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const JoinParams p) {
  constexpr int ROWS = kJoinThreads / (D / 4);
  constexpr long long PART = Plan<D>::PART;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const JoinHead H = p.heads[blockIdx.x];
  const int rr = blockIdx.y * ROWS + threadIdx.x % ROWS, c = threadIdx.x / ROWS, row = H.group * (128 / F) + rr;
  if (H.last < 0 || rr >= 128 / F || row >= p.rows) return;
  const int n = H.last - (int)blockIdx.x + 1;
  const float* first = p.part + (2ll * blockIdx.x + H.place) * PART;
  const float* rest = p.part + 2ll * blockIdx.x * PART;  // part i >= 1 at rest + 2 i PART
  auto at = [&](int i) { return i ? rest + 2ll * i * PART : first; };
  float top = -INFINITY;
#pragma unroll 8
  for (int i = 0; i < n; ++i) top = fmaxf(top, at(i)[rr]);
  const float ref = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const float* x = at(i);
    const float w = ex2(x[rr] - ref);
    const float4 v = reinterpret_cast<const float4*>(x + 256)[c * 128 + rr];
    l = fmaf(x[128 + rr], w, l);
    o.x = fmaf(v.x, w, o.x);
    o.y = fmaf(v.y, w, o.y);
    o.z = fmaf(v.z, w, o.z);
    o.w = fmaf(v.w, w, o.w);
  }
  const bool some = l > 0.f || l != l;
  const float il = 1.f / l;
  const int qi = row / p.G, hd = H.h * p.G + row - qi * p.G;
  T* out = reinterpret_cast<T*>(p.out) + (((long long)H.b * p.nq + qi) * p.Hq + hd) * D + 4 * c;
  store4(out, some ? make_float4(o.x * il, o.y * il, o.z * il, o.w * il) : make_float4(0.f, 0.f, 0.f, 0.f));
}

template <int D, int NT, int F, typename T>
cudaError_t tree_go(TcParams p, int sms, int device, cudaStream_t s) {
  using L = Plan<D>;
  constexpr int ROWS = 128 / F;
  static std::atomic<uint64_t> done{0};
  p.groups = (p.rows + ROWS - 1) / ROWS;
  p.grid = sms;
  cudaError_t e = allow_smem((const void*)tree_kernel<D, NT, F, T>, L::SMEM, device, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(p.grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = L::SMEM;
  if ((e = cudaLaunchKernelEx(&cfg, tree_kernel<D, NT, F, T>, p)) != cudaSuccess || p.grid == 1) return e;
  cfg.dynamicSmemBytes = 0;
  const int rows = p.rows < ROWS ? p.rows : ROWS;
  constexpr int join_rows = kJoinThreads / (D / 4);
  cfg.gridDim = dim3(p.grid - 1, (rows + join_rows - 1) / join_rows);
  cfg.blockDim = dim3(kJoinThreads);
  return cudaLaunchKernelEx(&cfg, tree_join_kernel<D, F, T>, JoinParams{p.heads, p.part, p.a.out, p.a.nq, p.a.Hq, p.G, p.rows});
}

// Rows above which the tensor cores take a call.  Both sides (us, 8 entries, 8 KV heads, bf16; split / here), of 32768
// tokens: d = 128 8 rows 99 / 94, 12 rows 109 / 94; d = 64 8 rows 54 / 69, 12 rows 84 / 69.  Of 1024: d = 128 8 rows 14.9 / 14.9, 12
// rows 17.0 / 14.9; d = 64 8 rows 11.3 / 12.7, 12 rows 13.4 / 12.8.
constexpr int kTreeMinRows = 8;

}  // namespace

bool tree_tc_takes(const AttnArgs& a) {
  const int rows = a.Hq / a.Hkv * a.nq;
  if ((a.d != 64 && a.d != 128) || a.dtype == TQ_F32 || rows <= kTreeMinRows) return false;
  // the plan counts tiles in 32 bits
  const long long groups = (rows + 63) / 64, tiles = (a.pool.max_blocks + 7) / 8 + kTreeGroupCost;
  return (long long)a.B * a.Hkv * groups * tiles < (1ll << 31) - (1ll << 20);
}

size_t tree_tc_workspace(int d, int rows, tq_dtype dtype) {
  if ((d != 64 && d != 128) || dtype == TQ_F32 || rows <= kTreeMinRows) return 0;
  return kJoinHeadBytes + (size_t)kMaxSms * (2 * 128 * (d + 2) + 2 * 256) * sizeof(float);
}

template <typename T, int NT>
static cudaError_t tree_type(const TcParams& p, int sms, int dev, cudaStream_t s) {
  if (p.a.d == 64) return p.rows <= 64 ? tree_go<64, NT, 2, T>(p, sms, dev, s) : tree_go<64, NT, 1, T>(p, sms, dev, s);
  return p.rows <= 64 ? tree_go<128, NT, 2, T>(p, sms, dev, s) : tree_go<128, NT, 1, T>(p, sms, dev, s);
}

cudaError_t launch_tree_tc(const AttnArgs& a, cudaStream_t s) {
  TcParams p;
  int dev;
  const int sms = tc_params(a, &p, &dev);
  return a.dtype == TQ_BF16 ? tree_type<__nv_bfloat16, 2>(p, sms, dev, s) : tree_type<__half, 3>(p, sms, dev, s);
}

}  // namespace tqb
