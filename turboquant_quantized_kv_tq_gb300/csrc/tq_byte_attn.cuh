// The tile step shared by the byte cache's mma.sync attention kernels: 16 tokens of one KV head
// against 8 NR query rows held by one warp.
//
// Mathematics, per row: o = sum_j p_j 2^(e_j) c_j / sum_j p_j, with c_j token j's V codes, 2^(e_j) its
// block's V scale and p_j = 2^(s_j), s_j = log2(e) scale q . k_j.  The running reference is
//   M = max_j (s_j + e_j) - 14,   P_j = 2^(s_j + e_j - M) in (0, 2^14],
// so that the matrix product sum_j P_j c_j takes P as fp16 whatever the scales are: its largest
// contribution sits at the top of fp16's range, and what underflows is 2^-38 of it.  The softmax
// sum l = sum_j P_j 2^(-e_j) stays in fp32 (|e_j| <= 30 keeps it in range).  The scale of a block
// costs nothing this way: e_j is added to the exponent's constant.
//
// Products are mma.sync with the tokens (scores) or the coordinates (readout) as M and the query rows as
// N, so 8 rows fill an instruction:
//   S^T[16 tok x 8 rows] += K[16 x d] Q^T[d x 8],  O^T[16 d x 8 rows] += V^T[16 d x 16 tok] P^T.
// Both are m16n8k16 on fp16; codes are exact in fp16.  (Scores as m16n8k32 on the stored e4m3 codes, the
// queries as e4m3 terms, need no conversion of keys but measured slower: 103 us instead of 98 for
// 8 x 32768 tokens, 138 instead of 116 for 16 rows.)  Thread (g, u) of the warp (g = lane / 4, u = lane % 4)
// holds tokens g, g + 8 and rows 2u, 2u + 1 of the scores; coordinates within a product are permuted so
// that its K operand is 16 contiguous codes per shared-memory load, and V's stored token order is that
// of the P operand.
#pragma once

#include <atomic>

#include "tq_byte.cuh"

namespace tqb {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kShift = 14.f;            // M is this far below the largest s + e
constexpr int kQueryTop = 14;             // exponent of a query row's largest magnitude as an fp16 operand
constexpr uint32_t kWaitLimit = 1u << 20; // polls of an mbarrier before giving up

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// fp16 terms of the queries and of the probabilities.
template <typename T>
constexpr int kTermsOf = sizeof(T) == 4 ? 2 : 1;

template <int D, int NR, typename T>
struct QFrag {
  uint32_t v[kTermsOf<T>][NR][D / 16][2];  // B operand of k-step s: coordinates 4 s' .. of the thread's chunks
  float f[NR][2];                          // rows 2u, 2u + 1: log2(e) * scale * the row's power-of-two scale
};

template <int D, int NR>
struct State {
  float o[NR][D / 16][4];  // O^T: coordinates 16 m + g, + 8; rows 2u, 2u + 1
  float m[NR][2], l[NR][2];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[r][i][k] = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[r][k] = -INFINITY;
        l[r][k] = 0.f;
      }
    }
  }
};

// First coordinate of the 16 codes of load i (0 .. D/64 - 1) of thread u of a quad, and its chunk.
template <int D>
__device__ __forceinline__ int frag_chunk(int u, int i) {
  if constexpr (D == 64) return u;
  return (i >> 1) * 8 + 2 * u + (i & 1);
}

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <> __device__ __forceinline__ float to_float(float x) { return x; }
template <> __device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
template <> __device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 consecutive elements as loaded.
template <typename T>
struct Raw16 {
  uint4 v[sizeof(T)];
};
__device__ __forceinline__ void unpack16(const Raw16<float>& r, float (&x)[16], const float*) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[4 * i] = __uint_as_float(r.v[i].x); x[4 * i + 1] = __uint_as_float(r.v[i].y);
    x[4 * i + 2] = __uint_as_float(r.v[i].z); x[4 * i + 3] = __uint_as_float(r.v[i].w);
  }
}
__device__ __forceinline__ void unpack16(const Raw16<__nv_bfloat16>& r, float (&x)[16], const __nv_bfloat16*) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack16(const Raw16<__half>& r, float (&x)[16], const __half*) {
  const uint32_t w[8] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w, r.v[1].x, r.v[1].y, r.v[1].z, r.v[1].w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// The thread's part of query rows row0 + 8 r + g (head h G + row % G of query row / G), as loaded: the
// load is issued before the copies of the slab's tiles, behind which it would wait for microseconds.
template <int D, int NR, typename T>
struct QRaw {
  Raw16<T> x[NR][D / 64];
};
template <int D, int NR, typename T>
__device__ __forceinline__ void request_q(QRaw<D, NR, T>& q, const Rows& X, int b, int h, int G, int row0, int rows, int lane) {
  const int g = lane >> 2, u = lane & 3;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int row = row0 + 8 * r + g;
    const bool live = row < rows;
    const int i = live ? row / G : 0, hd = h * G + (live ? row - i * G : 0);
    const T* src = reinterpret_cast<const T*>(X.p) + b * X.sb + i * X.st + hd * X.sh;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int k = 0; k < (int)sizeof(T); ++k) {
        q.x[r][c].v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (live) q.x[r][c].v[k] = __ldg(reinterpret_cast<const uint4*>(src + 16 * frag_chunk<D>(u, c)) + k);
      }
  }
}

// Query rows as fp16 operands.  Each row is scaled by the power of two that brings its largest magnitude
// into [2^14, 2^15), the top of fp16's range: what its smallest step, 2^-24, rounds away is then 2^-39 of the
// row's largest value at most (at [1, 2) it was 2^-25, so that beside a channel 2^12 times the others fp32 results
// were off by 1e-4).  bf16 and fp16 values are exact above that; fp32 rows take a second fp16 term of what the first
// leaves, together off by at most 2^-23 of a value or by 2^-39 of the largest.  Scores stay below
// 2^15 * 2 * 448 * 256 times the scales, far inside fp32.
template <int D, int NR, typename T>
__device__ __forceinline__ void convert_q(QFrag<D, NR, T>& q, const QRaw<D, NR, T>& raw, float score_scale, int lane) {
  const int u = lane & 3;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float amax = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float x[16];
      unpack16(raw.x[r][c], x, (const T*)nullptr);
#pragma unroll
      for (int k = 0; k < 16; ++k) amax = fmaxf(amax, fabsf(x[k]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 2));
    // exponent of amax less 14, held where 2^-e is a normal number (rows below 2^-112 keep fewer bits)
    const int e = max(log2i(amax), -112) - kQueryTop;
    const float inv = exp2i(-e);
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      float x[16];
      unpack16(raw.x[r][c], x, (const T*)nullptr);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const float a = x[4 * k + 2 * w] * inv, bb = x[4 * k + 2 * w + 1] * inv;
          const uint32_t hi = tqd::pack_half2(a, bb);
          q.v[0][r][4 * c + k][w] = hi;
          if constexpr (kTermsOf<T> == 2) {
            const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
            q.v[1][r][4 * c + k][w] = tqd::pack_half2(a - back.x, bb - back.y);
          }
        }
    }
    // (an infinity makes the row NaN: scores of -inf alone would look like a row that attends to nothing)
    const float f = amax <= 3.402823466e38f ? exp2i(e) * score_scale * kLog2e : __uint_as_float(0x7fc00000u);
    // (of row g: the threads that hold rows 2u, 2u + 1 need it)
    q.f[r][0] = __shfl_sync(kFull, f, 8 * u);
    q.f[r][1] = __shfl_sync(kFull, f, 8 * u + 4);
  }
}

// Bits j .. j + 31 of a draft's mask m, j counted from the entry's first draft: tokens before it are seen, those
// past the count are not.
__device__ __forceinline__ uint32_t tree_word(const uint32_t* m, int words, int cnt, int j) {
  if (j <= -32) return 0xffffffffu;
  if (j >= cnt) return 0u;
  const int w = j >> 5;  // (floor: -1 for the word that reaches back over the first draft)
  const uint32_t lo = w < 0 ? 0xffffffffu : __ldg(m + w), hi = w + 1 < words ? __ldg(m + w + 1) : 0u;
  const uint32_t v = __funnelshift_r(lo, hi, j & 31);
  return cnt - j >= 32 ? v : v & ((1u << (cnt - j)) - 1u);
}

// Which tokens rows 2u + k of group r do not attend to: those from the row's limit on.
template <int NR>
struct Limits {
  static constexpr bool kTree = false;
  const int (&lim)[NR][2];
  __device__ __forceinline__ bool operator()(int r, int k, int tok) const { return tok >= lim[r][k]; }
};
// The same of a tree: drafts whose bit is clear, and every draft for rows past the count.
struct TreeLimits {
  static constexpr bool kTree = true;
  const TreeMasks& M;
  int b, row0, G, drafts, cnt;  // row0: of the thread's row (0, 0); drafts: the first draft's position
  __device__ __forceinline__ bool operator()(int r, int k, int tok) const {
    const int i = (row0 + 8 * r + k) / G, j = tok - drafts;
    return j >= 0 && (i >= cnt || j >= cnt || !(__ldg(M.row(b, i) + (j >> 5)) >> (j & 31) & 1u));
  }
};

// One tile: `blk` is the block in shared memory, tok0 its first token, hide(r, k, tok) the tokens that row
// 2u + k of group r does not attend to, edge: some row of the warp does not attend to all 16 tokens, len:
// the sequence's length (codes of tokens behind it may be anything).
template <int D, int NR, bool EDGE, bool ADD, typename H, typename T>
__device__ __forceinline__ void tile_step_edge(const unsigned char* blk, const QFrag<D, NR, T>& q, State<D, NR>& st, int tok0,
                                               H hide, int len, int lane) {
  constexpr int TERMS = kTermsOf<T>;
  const int g = lane >> 2, u = lane & 3;
  float s[NR][4];
#pragma unroll
  for (int r = 0; r < NR; ++r)
#pragma unroll
    for (int k = 0; k < 4; ++k) s[r][k] = 0.f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    const int ch = frag_chunk<D>(u, c);
    const uint4 lo = *reinterpret_cast<const uint4*>(blk + k_chunk<D>(g, ch));
    const uint4 hi = *reinterpret_cast<const uint4*>(blk + k_chunk<D>(g + 8, ch));
    const uint32_t wl[4] = {lo.x, lo.y, lo.z, lo.w}, wh[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t a0, a1, a2, a3;
      codes_half4(wl[k], a0, a2);
      codes_half4(wh[k], a1, a3);
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
          tqd::mma16816(s[r], a0, a1, a2, a3, q.v[t][r][4 * c + k][0], q.v[t][r][4 * c + k][1]);
    }
  }
  const float2 scales = *reinterpret_cast<const float2*>(blk + 32 * D);
  const int ev = log2i(scales.y);
  const float e = (float)ev, inv_e = exp2i(max(-126, min(126, -ev)));
  bool up = false;
  float fk[NR][2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    fk[r][0] = q.f[r][0] * scales.x;
    fk[r][1] = q.f[r][1] * scales.x;
#pragma unroll
    for (int k = 0; k < 4; ++k) s[r][k] *= fk[r][k & 1];
    if (EDGE) {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (hide(r, k & 1, tok0 + g + 8 * (k >> 1))) s[r][k] = -INFINITY;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) up |= fmaxf(s[r][k], s[r][k + 2]) + (e - kShift) > st.m[r][k];
  }
  if (__any_sync(kFull, up)) {  // some row's reference rises
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float c = fmaxf(s[r][k], s[r][k + 2]) + (e - kShift);
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) c = fmaxf(c, __shfl_xor_sync(kFull, c, m));
        const float mn = fmaxf(st.m[r][k], c);
        const float cor = ex2(st.m[r][k] - (mn == -INFINITY ? 0.f : mn));
        st.m[r][k] = mn;
        st.l[r][k] *= cor;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          st.o[r][i][k] *= cor;
          st.o[r][i][k + 2] *= cor;
        }
      }
  }
  uint32_t p[TERMS][NR][2];
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float m = st.m[r][k & 1];
      v[k] = ex2(s[r][k] + (e - (m == -INFINITY ? 0.f : m)));
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) st.l[r][k] = fmaf(v[k] + v[k + 2], inv_e, st.l[r][k]);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint32_t hi = tqd::pack_half2(v[2 * w], v[2 * w + 1]);
      p[0][r][w] = tqd::movmatrix_trans(hi);
      if constexpr (TERMS == 2) {
        const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        p[1][r][w] = tqd::movmatrix_trans(tqd::pack_half2(v[2 * w] - back.x, v[2 * w + 1] - back.y));
      }
    }
  }
  // codes behind the sequence's end, and of hidden drafts that were never appended, may be NaN: zero them (their
  // probabilities are zero already)
  uint32_t keep = 0xffffffffu;
  if (EDGE && tok0 + 16 > len) {
    const int t = len - tok0;
    keep = (2 * u < t ? 0xffu : 0u) | (2 * u + 1 < t ? 0xff00u : 0u) | (2 * u + 8 < t ? 0xff0000u : 0u) |
           (2 * u + 9 < t ? 0xff000000u : 0u);
  }
  const unsigned char* vb = blk + 16 * D + 16 * g + 4 * u;
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t w0 = *reinterpret_cast<const uint32_t*>(vb + 256 * i), w1 = *reinterpret_cast<const uint32_t*>(vb + 256 * i + 128);
    if (EDGE) {
      w0 &= keep;
      w1 &= keep;
      if constexpr (H::kTree) {
        w0 = without_nans(w0);
        w1 = without_nans(w1);
      }
    }
    uint32_t a0, a1, a2, a3;
    codes_half4(w0, a0, a2);
    codes_half4(w1, a1, a3);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if constexpr (ADD) {
        float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int t = 0; t < TERMS; ++t) tqd::mma16816(o, a0, a1, a2, a3, p[t][r][0], p[t][r][1]);
#pragma unroll
        for (int k = 0; k < 4; ++k) st.o[r][i][k] += o[k];
      } else {
#pragma unroll
        for (int t = 0; t < TERMS; ++t) tqd::mma16816(st.o[r][i], a0, a1, a2, a3, p[t][r][0], p[t][r][1]);
      }
    }
  }
}

// ADD: the tile's readout is a product from zero that is then added in fp32.  The tensor cores' own
// accumulation truncates: chained over the 7600 tiles of a long sequence it was off by 2.8e-4 of the result.
// fp32 takes it always, 16-bit types where one warp walks a whole sequence.
template <int D, int NR, bool ADD, typename H, typename T>
__device__ __forceinline__ void tile_step(const unsigned char* blk, const QFrag<D, NR, T>& q, State<D, NR>& st, int tok0,
                                          H hide, bool edge, int len, int lane) {
  if (edge) tile_step_edge<D, NR, true, ADD>(blk, q, st, tok0, hide, len, lane);
  else tile_step_edge<D, NR, false, ADD>(blk, q, st, tok0, hide, len, lane);
}

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <> __device__ __forceinline__ float from_float<float>(float x) { return x; }
template <> __device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }
template <> __device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Host side (tq_byte_attn.cu): SMs of the current device and its index; a kernel's permission for its
// shared memory, once per kernel and device.
int sm_count(int* device);
cudaError_t allow_smem(const void* kernel, int bytes, int device, std::atomic<uint64_t>& done);
// The tensor-memory kernel (tq_byte_tc.cu): whether it takes a call, its workspace, its launch.
// It takes more than kTcMinRows rows: one pass over the pool, where the split makes one per 16 rows.  Both sides (us, 32 / 8
// heads, bf16, split / tensor memory), 16 x 16384 tokens: 16 rows 110 / 175, 32 rows 204 / 176, 64 rows 388 / 177, 80 rows
// 484 / 179; one sequence of 131072: 65 / 95, 107 / 95, 192 / 95, 235 / 96.  So above 16 rows it is the faster one already;
// the split, which it would replace there, keeps more bits of the queries (2^-39 instead of 2^-18 of a row's largest).
constexpr int kMaxSms = 160;
constexpr int kTcMinRows = 64;
bool tc_takes(const AttnArgs& a);
size_t tc_workspace(int rows);
cudaError_t launch_tc(const AttnArgs& a, cudaStream_t s);
// A tree's calls on the tensor memory (tq_byte_tree.cu): whether it takes a call, its workspace (0: it never takes
// such calls), its launch.
bool tree_tc_takes(const AttnArgs& a);
size_t tree_tc_workspace(int d, int rows, tq_dtype dtype);
cudaError_t launch_tree_tc(const AttnArgs& a, cudaStream_t s);

// Length and count of sequence b as the kernels use them.
__device__ __forceinline__ int clamped_len(const int32_t* seq_len, int b, int most, int32_t* err) {
  const int v = __ldg(seq_len + b);
  const int c = min(max(v, 0), most);
  if (c != v && err) atomicExch(err, TQ_DEVERR_BAD_LENGTH);
  return c;
}
__device__ __forceinline__ int clamped_count(const int32_t* count, int b, int nq) {
  return count ? min(max(__ldg(count + b), 0), nq) : nq;
}
// Tokens that a row of query i attends to.
__device__ __forceinline__ int row_limit(int i, int len, int cnt) { return i < cnt ? max(0, len - cnt + 1 + i) : 0; }

// ---- The join of ranges that share a slab's rows.  A range (one block of the main kernel) covers a
// contiguous stretch of slabs; where a slab goes on past its range's end, that range's head names the
// slab and the last range that holds a part of it.  In every later range the part is the first
// stretch (place 0), in the first one at place `place`.
struct JoinHead {
  int last;   // -1: no slab goes on past this range's end
  int place;
  int b, h, group;
};
constexpr int kJoinRows = 8;
constexpr int kMaxRanges = 512;
constexpr size_t kJoinHeadBytes = 16384;  // heads of the ranges, at the workspace's start
static_assert(kJoinHeadBytes >= kMaxRanges * sizeof(JoinHead), "heads");

struct JoinParams {
  const JoinHead* heads;
  const float* part;  // [range][2](M[ROWS], l[ROWS], O[ROWS][D]); of tree_join_kernel as tree_kernel's Plan says
  void* out;
  int nq, Hq, G, rows;
};

// Joins rows of the slab that goes on past range blockIdx.x: weights 2^(M_i - max M).  WARPS = 1: a block
// of kJoinRows warps takes as many rows; otherwise a block's WARPS warps share one row's parts.
constexpr int kJoinWarps = 4;
template <int D, int ROWS, int WARPS, typename T>
__global__ void __launch_bounds__(32 * (WARPS == 1 ? kJoinRows : WARPS)) join_kernel(const JoinParams p) {
  constexpr long long PART = (long long)ROWS * (D + 2);
  __shared__ float sum[WARPS][D + 1];
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rr = WARPS == 1 ? blockIdx.y * kJoinRows + warp : blockIdx.y, part0 = WARPS == 1 ? 0 : warp;
  const JoinHead H = p.heads[blockIdx.x];
  const int row = H.group * ROWS + rr;
  if (H.last < 0 || rr >= ROWS || row >= p.rows) return;  // (uniform over the warps that share a row)
  const int n = H.last - (int)blockIdx.x + 1;
  const float* first = p.part + (2ll * blockIdx.x + H.place) * PART;
  const float* rest = p.part + 2ll * blockIdx.x * PART;  // part i >= 1 at rest + 2 i PART
  auto at = [&](int i) { return i ? rest + 2ll * i * PART : first; };
  float mt = -INFINITY;
  for (int i = lane; i < n; i += 32) mt = fmaxf(mt, at(i)[rr]);
  mt = tqd::warp_max(mt);
  const float mr = mt == -INFINITY ? 0.f : mt;
  float l = 0.f, o[D / 32] = {};
  // lane i takes the statistics of the warp's parts i, i + 32, ...; their values are then read eight at a time
  for (int base = part0; base < n; base += 32 * WARPS) {
    const int mine = base + WARPS * lane;
    float w = 0.f;
    if (mine < n) {
      const float* x = at(mine);
      w = ex2(x[rr] - mr);
      l = fmaf(x[ROWS + rr], w, l);
    }
    const int m = min(32, (n - base + WARPS - 1) / WARPS);
#pragma unroll 8
    for (int i = 0; i < m; ++i) {
      const float wi = __shfl_sync(kFull, w, i);
      const float* v = at(base + WARPS * i) + 2 * ROWS + rr * D + lane * (D / 32);
#pragma unroll
      for (int k = 0; k < D / 32; k += 2) {
        const float2 f = *reinterpret_cast<const float2*>(v + k);
        o[k] = fmaf(f.x, wi, o[k]);
        o[k + 1] = fmaf(f.y, wi, o[k + 1]);
      }
    }
  }
  l = tqd::warp_sum(l);
  if constexpr (WARPS > 1) {
#pragma unroll
    for (int k = 0; k < D / 32; ++k) sum[warp][lane * (D / 32) + k] = o[k];
    if (lane == 0) sum[warp][D] = l;
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
      l += sum[w][D];
#pragma unroll
      for (int k = 0; k < D / 32; ++k) o[k] += sum[w][lane * (D / 32) + k];
    }
  }
  const float il = l > 0.f || l != l ? 1.f / l : 0.f;
  const int qi = row / p.G, hd = H.h * p.G + row - qi * p.G;
  T* out = reinterpret_cast<T*>(p.out) + (((long long)H.b * p.nq + qi) * p.Hq + hd) * D + lane * (D / 32);
#pragma unroll
  for (int k = 0; k < D / 32; ++k) out[k] = from_float<T>(o[k] * il);
}

}  // namespace tqb
