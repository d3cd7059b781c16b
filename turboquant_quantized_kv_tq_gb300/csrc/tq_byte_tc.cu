// Attention over the byte cache for chunks of queries (head dim 128, bf16 and fp16 queries), on the
// 5th-generation tensor cores.
//
// The rows of a slab (batch entry, KV head) are the chunk's (query, head) pairs, r = i G + g.  A block
// takes up to 256 of them, two tiles of 128, and walks the tokens 128 at a time:
//   S_i[128 x 128 tok] = Q_i K^T     kind::f8f6f4 on the codes as they are stored: K blocks are bulk-
//     copied from the pool straight into a 128-byte-swizzled operand.  The queries enter as e4m3
//     terms of 4 significant bits each: two hold a bf16 value exactly, three an fp16 value (two fp8
//     products cost what one fp16 product does, and no key is unpacked).  A row is scaled by the power
//     of two that puts its largest magnitude into (224, 448]; what lies below e4m3's smallest step
//     there, 2^-18 of the row's largest value, is rounded away.
//   O_i[128 x 128]    += P_i V       kind::f16, P from tensor memory, V's codes turned to fp16 (exact)
//     in shared memory by four warps, once for both row tiles.
// S_0, S_1, O_0, O_1 fill the tensor memory; P_i (fp16) takes the first half of S_i's columns.  While
// warps 0-3 work on S_0 the tensor cores work on tile 1, and the other way round.  A thread of
// warps 0-7 owns one row.  Softmax as in tq_byte_attn.cuh: block scales are exponents, so the value
// scale costs nothing and P keeps fp16's precision whatever the scales are, down to 2^-21 of the row's
// largest; below that it is off by up to 2^-32 of the largest.  The reference M is raised only when a
// row's maximum passes it by 15 (P <= 2^15), so O is rescaled rarely.
//
// The (row group, token tile) pairs of all slabs form one sequence cut into equal ranges, one per
// SM; ranges that share a row group leave partials that join_kernel joins.
//
// Warps: 0-7 rows, 8-11 V to fp16, 12 copies, 13 MMA issue (14, 15 only complete the warpgroup that
// gives registers to the rows: 192 a thread there, so that a row's 128 scores stay in registers from
// the maximum to the probabilities, and 64 in the other warps).
//
// Measured: 512 queries of 32 heads over 4 x 32768 tokens (8 KV heads, bf16) 787 us, 1386 TFLOP/s, 0.72 of
// the measured bf16 burst rate (0.81 of the sustained one: the run is at the power cap); fp16 (three
// query terms) 841 us; the last 64 positions 120 us; a prompt of
// 4096 tokens (one sequence) 203 us, of 32768 6.9 ms, 1270 TFLOP/s.  A tile takes about 2850 cycles, 2048 of them MMA.
// What bounds it is the chain of a row tile -- 128 scores to P, P V, the next scores -- beside the other
// tile's, and shared memory: an fp8 product of N = 128 reads 8 KB in its 64 cycles, all that it delivers.
// Tiles of 80 tokens, whose P has columns of its own so that scores run ahead, were slower (1480 us): at
// N = 80 a product still reads the 4 KB of Q and takes 55 cycles.
#include <atomic>
#include <string>
#include <type_traits>

#include "tq_byte_tc.cuh"

namespace tqb {
namespace {

using tqd::mbar_wait;

constexpr int kD = 128;
constexpr int kGroupCost = 8;      // virtual tiles of a row group: what a range costs beside its tiles (4: 125 us for
                                   // the last 64 positions, 8: 122, 14: 124)
constexpr int kBlk = 32 * kD + 32;

template <int NT, int NQ>
struct Plan {
  static constexpr int ROWS = 128 * NQ;
  // blocks of a tile in the first of the two parts in which P is handed over: with two query terms the
  // products keep up and one late hand-over costs least (4 / 6 / 7 blocks: 815 / 805 / 788 us for 512 queries
  // x 4 x 32768 tokens), with three they start early (4 / 6 / 7: 841 / 866 / 958 us)
  static constexpr int FIRST = NT == 2 ? 7 : 4;
  static constexpr int SC = 4;                                    // scale stages of 8 x 16 bytes
  static constexpr int Q = 0, KR = Q + NQ * NT * 16384, VR = KR + 2 * 16384, V16 = VR + 2 * 16384;
  // [stage][block]: as copied (K scale, V scale, -, -), then in place (K scale, e, 2^-e, -)
  static constexpr int SCALES = V16 + 2 * 32768, BARS = SCALES + SC * 128, PRE = BARS + 320;
  static constexpr int SMEM = PRE + (TQ_MAX_BATCH + 1) * 4;
  static_assert(SMEM <= 227 * 1024, "shared memory");
  static constexpr int PART = ROWS * (kD + 2);                    // floats of a partial
};
// (P_FULL: half h of row tile i at 2 i + h)
enum Bar { K_FULL = 0, K_EMPTY = 2, VR_FULL = 4, VR_EMPTY = 6, V_FULL = 8, V_EMPTY = 10, S_FULL = 12, O_DONE = 14,
           Q_FULL = 16, P_FULL = 18, SC_FULL = 22, SC_EMPTY = 26, SC_READY = 30, BAR_COUNT = 34 };
static_assert(8 * BAR_COUNT + 4 <= 320, "barriers and the tensor-memory slot");

__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// Products of one elected lane of a converged warp, from constant operands.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);  // M = N = 128, fp32 D
static_assert(kTok == 128 && kD == 128, "one instruction shape for both products");

// S_i of the tile in K buffer ST.
template <int NT, int NQ, int ST>
__device__ __forceinline__ void issue_scores(uint32_t sb, int i) {
  using L = Plan<NT, NQ>;
  const uint64_t q = sdesc128(sb + L::Q + i * NT * 16384), k = sdesc128(sb + L::KR + ST * 16384);
  if (elected()) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int j = 0; j < 4; ++j) mma_f8(128 * i, q + (uint64_t)(t * (16384 >> 4) + 2 * j), k + 2 * j, kIdesc, t + j > 0);
    tqd::tc_commit(sb + L::BARS + 8 * (S_FULL + i));
    if (i == NQ - 1) tqd::tc_commit(sb + L::BARS + 8 * (K_EMPTY + ST));
  }
  __syncwarp();
}
// Part h (blocks [0, FIRST), [FIRST, 8)) of O_i += P_i V of the tile in V buffer ST (accumulate: not the
// range's first tile).
template <int NT, int NQ, int ST>
__device__ __forceinline__ void issue_readout(uint32_t sb, int i, int h, bool accumulate) {
  using L = Plan<NT, NQ>;
  const uint64_t v = sdesc128(sb + L::V16 + ST * 32768);
  if (elected()) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if ((k >= L::FIRST) == (h == 1))
        tqd::tc_mma_f16_ta(256 + 128 * i, 128 * i + 8 * k, v + (uint64_t)((k >> 2) * (16384 >> 4) + 2 * (k & 3)), kIdesc,
                           accumulate || k > 0);
    if (h == 1) {
      tqd::tc_commit(sb + L::BARS + 8 * (O_DONE + i));
      if (i == NQ - 1) tqd::tc_commit(sb + L::BARS + 8 * (V_EMPTY + ST));
    }
  }
  __syncwarp();
}

// Tokens that the rows of group rg of an entry attend to at most, and tiles.
__device__ __forceinline__ int group_limit(const TcParams& p, int rows_per, int rg, int len, int cnt) {
  const int last = min((rg + 1) * rows_per, p.rows) - 1;
  const int i = min(cnt - 1, last / p.G);
  return i * p.G + p.G - 1 < rg * rows_per ? 0 : row_limit(i, len, cnt);
}
__device__ __forceinline__ int cost_of(int tiles) { return tiles > 0 ? tiles + kGroupCost : 0; }

// Costs before each entry (order: entry, row group, head); written by warp 0.
__device__ __forceinline__ void fill_plan(const TcParams& p, int rows_per, int* pre, int32_t* err) {
  const int lane = threadIdx.x & 31, most = p.a.pool.max_blocks * 16;
  if (threadIdx.x < 32) {
    int run = 0;
    for (int b0 = 0; b0 < p.a.B; b0 += 32) {
      const int b = b0 + lane;
      int t = 0;
      if (b < p.a.B) {
        const int len = clamped_len(p.a.seq_len, b, most, err), cnt = clamped_count(p.a.count, b, p.a.nq);
        for (int rg = 0; rg < p.groups; ++rg) t += cost_of(tiles_of(group_limit(p, rows_per, rg, len, cnt)));
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
    s.limit = group_limit(p, rows_per, s.rg, s.len, s.cnt);
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

// One query row as NT e4m3 terms in the swizzled operand tiles at q (term t at q + 16384 t); returns
// the factor of its scores, log2(e) |scale| 2^e (the sign of `scale` goes into the terms).
template <typename T, int NT>
__device__ __forceinline__ float query_row(const T* src, bool live, float scale, unsigned char* q, int r) {
  uint4 raw[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) raw[c] = live ? __ldg(reinterpret_cast<const uint4*>(src) + c) : make_uint4(0u, 0u, 0u, 0u);
  float amax = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) {
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
  for (int c = 0; c < 8; ++c) {
    float x[16];
    unpack16(Raw16<T>{{raw[2 * c], raw[2 * c + 1]}}, x, src);
    const int at = r * 128 + ((c ^ (r & 7)) << 4);
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
      *reinterpret_cast<uint4*>(q + 16384 * t + at) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  return odd ? __uint_as_float(0x7fc00000u) : fabsf(scale) * kLog2e * exp2i(e);
}

template <typename T, int NT, int NQ>
__global__ void __launch_bounds__(kThreads, 1) tc_kernel(const TcParams p) {
  using L = Plan<NT, NQ>;
  extern __shared__ __align__(1024) unsigned char sm[];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const AttnArgs& A = p.a;
  const int warp = __shfl_sync(kFull, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t sb = (uint32_t)__cvta_generic_to_shared(sm);
  const uint32_t bars = sb + L::BARS;
  auto bar = [&](int kind, int i) { return bars + 8 * (kind + i); };
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + L::BARS + 8 * BAR_COUNT);
  int* pre = reinterpret_cast<int*>(sm + L::PRE);
  if (sb & 1023u) {  // the swizzled operands need it (the plan gives it)
    if (threadIdx.x == 0) {
      p.heads[blockIdx.x].last = -1;
      if (A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_SMEM_PLAN);
    }
    return;
  }
  if (warp == 13) tqd::tc_alloc((uint32_t)__cvta_generic_to_shared(slot), 512);
  if (threadIdx.x == 32) {
    for (int i = 0; i < 2; ++i) {
      tqd::mbar_init(bar(K_FULL, i), 1);
      tqd::mbar_init(bar(K_EMPTY, i), 1);
      tqd::mbar_init(bar(VR_FULL, i), 1);
      tqd::mbar_init(bar(VR_EMPTY, i), 4);
      tqd::mbar_init(bar(V_FULL, i), 4);
      tqd::mbar_init(bar(V_EMPTY, i), 1);
      tqd::mbar_init(bar(S_FULL, i), 1);
      tqd::mbar_init(bar(P_FULL, 2 * i), 128);
      tqd::mbar_init(bar(P_FULL, 2 * i + 1), 128);
      tqd::mbar_init(bar(O_DONE, i), 1);
      tqd::mbar_init(bar(Q_FULL, i), 128);
    }
    for (int i = 0; i < L::SC; ++i) {
      tqd::mbar_init(bar(SC_FULL, i), 1);
      tqd::mbar_init(bar(SC_EMPTY, i), 4 * NQ);
      tqd::mbar_init(bar(SC_READY, i), 1);
    }
    tqd::fence_mbar_init();
  }
  fill_plan(p, L::ROWS, pre, blockIdx.x == 0 ? A.pool.err : nullptr);
  tqd::tc_fence_before();
  __syncthreads();
  tqd::tc_fence_after();
  // all 512 columns are this block's: they begin at column 0, lane 0
  const bool whole_tmem = *slot == 0;
  constexpr uint32_t tmem = 0;
  const int total = pre[A.B], per = range_of(total, p.grid);
  const int begin = min(total, (int)blockIdx.x * per), end = min(total, begin + per);

  bool ok = whole_tmem;  // cleared by a wait that gave up: the role stops working and ends
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (ok && !mbar_wait(b, parity, kWaitLimit)) ok = false;
    return ok;
  };

  if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kRowRegs));
  else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kOtherRegs));
  if (warp < 4 * NQ) {
    // ---- rows
    const int i = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + 128 * i, t_o = tmem + lanes + 256 + 128 * i;
    uint32_t n = 0;       // tiles so far
    // groups without a live row: zeros, spread over the grid
    {
      const int slabs = A.B * p.groups * A.Hkv, most = A.pool.max_blocks * 16;
      for (int s = blockIdx.x; s < slabs; s += gridDim.x) {
        const int h = s % A.Hkv, rg = s / A.Hkv % p.groups, b = s / A.Hkv / p.groups;
        const int len = clamped_len(A.seq_len, b, most, nullptr), cnt = clamped_count(A.count, b, A.nq);
        if (group_limit(p, L::ROWS, rg, len, cnt) > 0) continue;
        const int row = rg * L::ROWS + i * 128 + r;
        if (row < p.rows) {
          T* o = out_row<kD, T>(p, b, h, row);
          for (int c = 0; c < 16; ++c) reinterpret_cast<uint4*>(o)[c] = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    }
    int at = begin;
    bool headed = false;
    while (at < end && ok) {
      const Seg s = seg_at(p, L::ROWS, pre, at, end);
      const bool first = at == begin;
      at = s.next;
      if (s.t0 == s.t1) continue;
      const int row = s.rg * L::ROWS + i * 128 + r;
      const bool live = row < p.rows;
      const int qi = live ? row / p.G : 0, hd = s.h * p.G + (live ? row - qi * p.G : 0);
      const int lim = live ? row_limit(qi, s.len, s.cnt) : 0;
      const int least = __reduce_min_sync(kFull, live ? lim : 0x7fffffff);
      const float f = query_row<T, NT>(reinterpret_cast<const T*>(A.q.p) + s.b * A.q.sb + qi * A.q.st + hd * A.q.sh, live,
                                       A.scale, sm + L::Q + i * NT * 16384, r);
      tqd::tc_fence_smem();
      tqd::tc_mbar_arrive(bar(Q_FULL, i));
      float M = -INFINITY, l = 0.f;
      // one tile; false: a wait gave up
      auto tile = [&](auto edge_tag, int t) {
        constexpr bool EDGE = decltype(edge_tag)::value;
        if (!wait(bar(S_FULL, i), n & 1)) return false;
        const int ss = n % L::SC;
        if (!wait(bar(SC_READY, ss), (n / L::SC) & 1)) return false;
        tqd::tc_fence_after();
        const float4* sc = reinterpret_cast<const float4*>(sm + L::SCALES + 128 * ss);
        const int left = lim - kTok * t;  // tokens of this tile that the row attends to
        float v[128];
        ld32_async(t_s, v);
        ld32_async(t_s + 32, v + 32);
        float a[8], e[8];
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float4 x = sc[g];
          a[g] = f * x.x;
          e[g] = x.y;
        }
        ld_wait<64>(v);
        ld32_async(t_s + 64, v + 64);
        ld32_async(t_s + 96, v + 96);
        float top = block_top<EDGE>(v, left, a[0], e[0]);
#pragma unroll
        for (int g = 1; g < 4; ++g) top = fmaxf(top, block_top<EDGE>(v + 16 * g, left - 16 * g, a[g], e[g]));
        ld_wait<64>(v + 64);
#pragma unroll
        for (int g = 4; g < 8; ++g) top = fmaxf(top, block_top<EDGE>(v + 16 * g, left - 16 * g, a[g], e[g]));
        const bool raise = top > M + kSlack;
        if (__any_sync(kFull, raise)) {
          const float m_new = raise ? top - kTop : M;
          const float cor = raise ? ex2(M - m_new) : 1.f;
          M = m_new;
          if (t > s.t0) {
            l *= cor;
            if (!wait(bar(O_DONE, i), (n - 1) & 1)) return false;
            tqd::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < 8; ++c) {
              float o[16];
              uint32_t w[16];
              tqd::tc_ld16(t_o + 16 * c, o);
#pragma unroll
              for (int k = 0; k < 16; ++k) w[k] = __float_as_uint(o[k] * cor);
              tqd::tc_st16(t_o + 16 * c, w);
            }
          }
        }
        const float mr = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          uint32_t w[8];
          const float sum = block_p<EDGE>(v + 16 * g, left - 16 * g, a[g], e[g] - mr, w);
          l = fmaf(sum, sc[g].z, l);
          st8_async(t_s + 8 * g, w);
          if (g == L::FIRST - 1 || g == 7) {
            asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory");
            tqd::tc_fence_before();
            tqd::tc_mbar_arrive(bar(P_FULL, 2 * i + (g == 7)));
          }
        }
        __syncwarp();
        if (lane == 0) tqd::tc_mbar_arrive(bar(SC_EMPTY, ss));
        ++n;
        return true;
      };
      for (int t = s.t0; t < s.t1; ++t) {
        if (kTok * (t + 1) > least ? !tile(std::true_type{}, t) : !tile(std::false_type{}, t)) break;
      }
      if (!ok || !wait(bar(O_DONE, i), (n - 1) & 1)) break;
      tqd::tc_fence_after();
      const bool whole = s.t0 == 0 && s.t1 == s.tiles;
      if (whole) {
        const float il = l > 0.f || l != l ? 1.f / l : 0.f;
        T* o = out_row<kD, T>(p, s.b, s.h, live ? row : 0);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tqd::tc_ld32(t_o + 32 * c, v);
          if (live) {
#pragma unroll
            for (int k = 0; k < 32; ++k) v[k] *= il;
            store16(o + 32 * c, v);
            store16(o + 32 * c + 16, v + 16);
          }
        }
      } else {
        float* part = p.part + (2ll * blockIdx.x + (first ? 0 : 1)) * L::PART;
        const int rr = i * 128 + r;
        part[rr] = M;
        part[L::ROWS + rr] = l;
        float* o = part + 2 * L::ROWS + (long long)rr * kD;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tqd::tc_ld32(t_o + 32 * c, v);
#pragma unroll
          for (int k = 0; k < 8; ++k)
            reinterpret_cast<float4*>(o + 32 * c)[k] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
      }
      tqd::tc_fence_before();  // (the next range's first product overwrites O after its P arrives)
      if (threadIdx.x == 0 && s.t0 == 0 && s.t1 < s.tiles) {  // this range's last stretch begins a group that goes on
        p.heads[blockIdx.x] = JoinHead{(s.start + s.tiles - 1) / per, first ? 0 : 1, s.b, s.h, s.rg};
        headed = true;
      }
    }
    if (threadIdx.x == 0 && !headed) p.heads[blockIdx.x].last = -1;
  } else if (warp >= 8 && warp < 12) {
    // ---- V codes to fp16, K-major [coordinate][token], 64 tokens per 128-byte row
    uint32_t n = 0;
    int at = begin;
    while (at < end && ok) {
      const Seg s = seg_at(p, L::ROWS, pre, at, end);
      at = s.next;
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int st = n & 1, ss = n % L::SC;
        if (warp == 8) {
          if (!wait(bar(SC_FULL, ss), (n / L::SC) & 1)) break;
          if (lane < 8) {
            float4* x = reinterpret_cast<float4*>(sm + L::SCALES + 128 * ss + 16 * lane);
            const int e = log2i(x->y);  // (of a block behind the tokens: any exponent; 2^-e stays finite)
            x->y = (float)e;
            x->z = exp2i(max(-126, min(126, -e)));
          }
          __syncwarp();
          if (lane == 0) tqd::tc_mbar_arrive(bar(SC_READY, ss));
        }
        if (!wait(bar(VR_FULL, st), (n >> 1) & 1)) break;
        if (n >= 2 && !wait(bar(V_EMPTY, st), ((n >> 1) - 1) & 1)) break;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int j = (warp - 8) + 4 * k;
          const int have = s.limit - kTok * t - 16 * j;  // tokens of the block in use; the rest become zeros
          uint32_t keep[4];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            keep[u] = have >= 16 ? 0xffffffffu
                                 : (2 * u < have ? 0xffu : 0u) | (2 * u + 1 < have ? 0xff00u : 0u) |
                                       (2 * u + 8 < have ? 0xff0000u : 0u) | (2 * u + 9 < have ? 0xff000000u : 0u);
          const unsigned char* src = sm + L::VR + st * 16384 + j * 2048;
          unsigned char* dst = sm + L::V16 + st * 32768 + (j >> 2) * 16384;
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int d = lane + 32 * m;
            const uint4 v = *reinterpret_cast<const uint4*>(src + 16 * d);
            uint32_t w[8];
            codes_half4(v.x & keep[0], w[0], w[1]);
            codes_half4(v.y & keep[1], w[2], w[3]);
            codes_half4(v.z & keep[2], w[4], w[5]);
            codes_half4(v.w & keep[3], w[6], w[7]);
            const int c = 2 * (j & 3);
            *reinterpret_cast<uint4*>(dst + d * 128 + ((c ^ (d & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(dst + d * 128 + (((c + 1) ^ (d & 7)) << 4)) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
        tqd::tc_fence_smem();
        __syncwarp();
        if (lane == 0) {
          tqd::tc_mbar_arrive(bar(VR_EMPTY, st));
          tqd::tc_mbar_arrive(bar(V_FULL, st));
        }
      }
    }
  } else if (warp == 12) {
    // ---- copies: lanes 0-7 the K codes of a block each, 8-15 the V codes, 16-23 the scales
    uint32_t n = 0;
    int at = begin;
    while (at < end && ok) {
      const Seg s = seg_at(p, L::ROWS, pre, at, end);
      at = s.next;
      const int blocks = (s.limit + 15) >> 4;
      int page = 0;
      for (int t = s.t0; t < s.t1; ++t, ++n) {
        const int u = (t - s.t0) & 3;
        if (u == 0) page = 8 * t + lane < blocks ? page_of(A.pool, s.b, 8 * t + lane) : 0;
        const int pg = __shfl_sync(kFull, page, 8 * u + (lane & 7));
        const int nb = min(8, blocks - 8 * t), st = n & 1, ss = n % L::SC;
        if (n >= 2) {
          if (!wait(bar(K_EMPTY, st), ((n >> 1) - 1) & 1)) break;
          if (!wait(bar(VR_EMPTY, st), ((n >> 1) - 1) & 1)) break;
        }
        if (n >= L::SC && !wait(bar(SC_EMPTY, ss), (n / L::SC - 1) & 1)) break;
        if (lane == 0) {
          tqd::mbar_arrive_expect_tx(bar(K_FULL, st), nb * 2048);
          tqd::mbar_arrive_expect_tx(bar(VR_FULL, st), nb * 2048);
          tqd::mbar_arrive_expect_tx(bar(SC_FULL, ss), nb * 16);
        }
        __syncwarp();
        const int j = lane & 7;
        if (j < nb && lane < 24) {
          const unsigned char* blk = A.pool.base + pool_block(A.pool, pg, s.h) * kBlk;
          if (lane < 8) tqd::bulk_g2s(sb + L::KR + st * 16384 + j * 2048, blk, 2048, bar(K_FULL, st));
          else if (lane < 16) tqd::bulk_g2s(sb + L::VR + st * 16384 + j * 2048, blk + 2048, 2048, bar(VR_FULL, st));
          else tqd::bulk_g2s(sb + L::SCALES + ss * 128 + j * 16, blk + 4096, 16, bar(SC_FULL, ss));
        }
        __syncwarp();
      }
    }
    // every copy has landed before the block gives up its shared memory
    for (uint32_t k = n > 2 ? n - 2 : 0; k < n; ++k) {
      mbar_wait(bar(K_FULL, k & 1), (k >> 1) & 1, kWaitLimit);
      mbar_wait(bar(VR_FULL, k & 1), (k >> 1) & 1, kWaitLimit);
      mbar_wait(bar(SC_FULL, k % L::SC), (k / L::SC) & 1, kWaitLimit);
    }
  } else if (warp == 13) {
    // ---- MMA issue.  Every operand is a constant of the stage (the buffers' parity is a template
    // argument, the tensor memory begins at column 0), so the descriptors sit in uniform registers;
    // with operands computed per tile the issue took 60-100 cycles an instruction and bounded the kernel.
    uint32_t n = 0, segs = 0;
    int at = begin;
    while (at < end && ok) {
      const Seg s = seg_at(p, L::ROWS, pre, at, end);
      at = s.next;
      if (s.t0 == s.t1) continue;
      if (!wait(bar(K_FULL, n & 1), (n >> 1) & 1)) break;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        if (!wait(bar(Q_FULL, i), segs & 1)) break;
        tqd::tc_fence_after();
        if (n & 1) issue_scores<NT, NQ, 1>(sb, i);
        else issue_scores<NT, NQ, 0>(sb, i);
      }
      ++segs;
      for (int t = s.t0; t < s.t1 && ok; ++t, ++n) {
        const bool more = t + 1 < s.t1;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
          if (i == 0 && !wait(bar(V_FULL, n & 1), (n >> 1) & 1)) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!wait(bar(P_FULL, 2 * i + h), n & 1)) break;
            tqd::tc_fence_after();
            if (n & 1) issue_readout<NT, NQ, 1>(sb, i, h, t > s.t0);
            else issue_readout<NT, NQ, 0>(sb, i, h, t > s.t0);
          }
          if (!ok) break;
          if (more) {
            if (i == 0 && !wait(bar(K_FULL, (n + 1) & 1), ((n + 1) >> 1) & 1)) break;
            if (n & 1) issue_scores<NT, NQ, 0>(sb, i);
            else issue_scores<NT, NQ, 1>(sb, i);
          }
        }
      }
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

template <typename T, int NT, int NQ>
cudaError_t tc_go(TcParams p, int sms, int device, cudaStream_t s) {
  using L = Plan<NT, NQ>;
  static std::atomic<uint64_t> done{0};
  p.groups = (p.rows + L::ROWS - 1) / L::ROWS;
  p.grid = sms;
  cudaError_t e = allow_smem((const void*)tc_kernel<T, NT, NQ>, L::SMEM, device, done);
  if (e != cudaSuccess) return e;
  tc_kernel<T, NT, NQ><<<p.grid, kThreads, L::SMEM, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  const int rows = p.rows < L::ROWS ? p.rows : L::ROWS;
  cfg.gridDim = dim3(p.grid - 1, (rows + kJoinRows - 1) / kJoinRows);
  cfg.blockDim = dim3(32 * kJoinRows);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<kD, L::ROWS, 1, T>, JoinParams{p.heads, p.part, p.a.out, p.a.nq, p.a.Hq, p.G, p.rows});
}

}  // namespace

bool tc_takes(const AttnArgs& a) {
  const int rows = a.Hq / a.Hkv * a.nq;
  if (a.d != kD || a.dtype == TQ_F32 || rows <= kTcMinRows) return false;
  // the plan counts tiles in 32 bits
  const long long groups = (rows + 127) / 128, tiles = (a.pool.max_blocks + 7) / 8 + kGroupCost;
  return (long long)a.B * a.Hkv * groups * tiles < (1ll << 31) - (1ll << 20);
}

size_t tc_workspace(int rows) {
  return kJoinHeadBytes + (size_t)2 * kMaxSms * (rows > 128 ? Plan<2, 2>::PART : Plan<2, 1>::PART) * sizeof(float);
}

int tc_params(const AttnArgs& a, TcParams* p, int* dev) {
  p->a = a;
  p->G = a.Hq / a.Hkv;
  p->rows = p->G * a.nq;
  p->groups = p->grid = 0;
  p->heads = (JoinHead*)a.ws;
  p->part = (float*)((unsigned char*)a.ws + kJoinHeadBytes);
  const int sms = sm_count(dev);
  return sms > kMaxSms ? kMaxSms : sms;
}

cudaError_t launch_tc(const AttnArgs& a, cudaStream_t s) {
  TcParams p;
  int dev;
  const int sms = tc_params(a, &p, &dev);
  if (a.dtype == TQ_BF16)
    return p.rows > 128 ? tc_go<__nv_bfloat16, 2, 2>(p, sms, dev, s) : tc_go<__nv_bfloat16, 2, 1>(p, sms, dev, s);
  return p.rows > 128 ? tc_go<__half, 3, 2>(p, sms, dev, s) : tc_go<__half, 3, 1>(p, sms, dev, s);
}

}  // namespace tqb
