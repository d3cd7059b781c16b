// Attention over the byte cache for few query rows per KV head (single tokens, drafts), and the
// mma.sync kernel for chunks where the tensor-memory kernel is not built.
//
// split_kernel: bound by HBM -- every code is read once, 4 d flops per byte and row.  The tiles
// (16-token blocks) of all slabs (batch entry, KV head, group of 8 NR rows), each slab followed by
// kSlabCost virtual tiles for the work it costs a block beside its tiles (queries, the join of the
// warps), form one sequence that is cut into equal contiguous ranges, one per resident block, so the
// load is even whatever the lengths are.  Each warp streams its own tiles through its own ring of bulk
// copies: a block of the pool is contiguous, codes and scales in one copy.  Warps meet only at the end of
// a slab's range.  Ranges that cover part of a slab leave (M, l, O) in the workspace for join_kernel,
// which is launched early and waits for this grid.
// Measured: 8 x 32768 tokens, 32 / 8 heads, bf16, 98 us, 5.51 TB/s (0.81 of the measured copy rate); fp32
// queries 97 us; 131072 tokens of 64 / 8 heads 56 us; 16 x 16384 tokens with 16 rows 110 us; 1024 tokens
// 10 us.  Of the first's 18 us above its floor some 5 pass before the tiles flow (lengths, plan, page
// table, first copies), 3 in the join, and the rest at the end: SMs differ by up to a fifth in what they
// stream (groups of 10 to 20 neighbours), and the fast ones idle.
// rows_kernel: 8 warps of 8 NR rows share one ring; each tile is read once per 64 NR rows.  Bound by the
// mma.sync rate and the conversions, which every warp repeats: 107 TFLOP/s (fp32, d = 64), 148 (16 bits, d = 64),
// 193 (d = 256).  It does not split the tokens: with few slabs it leaves SMs idle (see use_rows).
#include <atomic>
#include <string>

#include "tq_byte_attn.cuh"

namespace tqb {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxGrid = kMaxRanges;  // resident blocks of the split, at most (the workspace is sized for it)
constexpr int kMinTiles = 8;   // tiles of a range, at least: one per warp
constexpr int kSlabCost = 32;  // virtual tiles of a slab (4-5 us of a block; 8 / 16 / 24 / 40: a batch of 64 unlike
                               // lengths 45 / 32 / 27 / 26 us)

struct AttnParams {
  AttnArgs a;
  int G, rows, groups;   // query heads per KV head, rows per KV head, row groups of 8 NR
  float* part;           // partials: [block][first stretch, last](M[8 NR], l[8 NR], O[8 NR][D])
  JoinHead* heads;
  int grid;              // blocks of the split
};

// a / b, in 32 bits where a fits (a 64-bit division costs hundreds of cycles).
__device__ __forceinline__ long long div_small(long long a, int b) {
  return (a >> 31) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}

// Tiles (virtual ones included) before each batch entry, in the order entry, head, row group; the
// split's range length.
struct Plan {
  long long total, per;
};
__device__ __forceinline__ Plan make_plan(const AttnParams& p, long long* pre) {
  // one warp: inclusive scan over the entries, 32 at a time
  const int lane = threadIdx.x & 31;
  const int most = p.a.pool.max_blocks * 16;
  const long long per_tile = (long long)p.a.Hkv * p.groups;
  if (threadIdx.x < 32) {
    long long run = 0;
    for (int b0 = 0; b0 < p.a.B; b0 += 32) {
      const int b = b0 + lane;
      long long t = 0;
      if (b < p.a.B && clamped_count(p.a.count, b, p.a.nq) > 0) {
        const int len = clamped_len(p.a.seq_len, b, most, blockIdx.x == 0 ? p.a.pool.err : nullptr);
        if (len > 0) t = (((len + 15) >> 4) + kSlabCost) * per_tile;
      }
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const long long o = __shfl_up_sync(kFull, t, m);
        if (lane >= m) t += o;
      }
      if (b < p.a.B) pre[b + 1] = run + t;
      run += __shfl_sync(kFull, t, 31);
    }
    if (lane == 0) pre[0] = 0;
  }
  __syncthreads();
  Plan P;
  P.total = pre[p.a.B];
  P.per = (div_small(P.total + p.grid - 1, p.grid) + kMinTiles - 1) / kMinTiles * kMinTiles;
  return P;
}

// A stretch of one slab: tiles [t0, t1) of its `tiles`; next: where the following stretch begins;
// start: where the slab does.
struct Seg {
  int b, h, rg;
  int t0, t1, tiles;
  long long start, next;
};
// The stretch that begins at tile `at` (< end) of the sequence, empty where only virtual tiles are
// left; b: the entry to look from.
__device__ __forceinline__ Seg seg_at(const AttnParams& p, const long long* pre, long long at, long long end, int b) {
  while (pre[b + 1] <= at) ++b;
  Seg s;
  s.b = b;
  const int slabs = p.a.Hkv * p.groups;
  const int span = (int)div_small(pre[b + 1] - pre[b], slabs);
  s.tiles = span - kSlabCost;
  const long long off = at - pre[b];
  const int k = (int)div_small(off, span), x = (int)(off - (long long)k * span);
  s.t0 = min(x, s.tiles);
  s.t1 = (int)min((long long)s.tiles, x + (end - at));
  s.start = at - x;
  s.next = min(end, at + (span - x));
  s.h = k / p.groups;
  s.rg = k - s.h * p.groups;
  return s;
}
// Entry that holds tile `at`.
__device__ __forceinline__ int find_entry(const long long* pre, int B, long long at) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] <= at) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

template <int D, int NR, int TERMS>
struct Cfg {
  static constexpr int BLK = 32 * D + 32;
  // warps: fp32 at d = 128 12 of 168 registers (8 x 32768 tokens: 97 us, 8 warps 109 us)
  static constexpr int NW = NR == 1 && D == 128 && TERMS == 2 ? 12 : 8;
  static constexpr bool TWO = NR == 1 && D <= 128 && TERMS * D <= 128;      // two blocks per SM
  static constexpr int ROOM = (TWO ? 115200 : 231424) - 4160 - 512;         // less the plan and barriers
  static constexpr int RED = NW * 8 * NR * (D / 4 + 4) * 4;             // a quarter of O per round
  static constexpr int ST0 = (ROOM - RED) / (NW * BLK);
  static constexpr int STAGES = ST0 > 8 ? 8 : ST0;
  static constexpr int RING = NW * STAGES * BLK;
  // ring, reduction, barriers, (m, l) of the warps, plan
  static constexpr int O_RED = RING, O_BAR = O_RED + RED, O_ML = O_BAR + NW * STAGES * 8;
  static constexpr int O_PRE = (O_ML + NW * 8 * NR * 8 + 15) / 16 * 16;
  static int smem(int B) { return O_PRE + (B + 1) * 8; }
  static constexpr int PART = 8 * NR * (D + 2);                             // floats of a partial
};

template <int D, int NR, int TERMS, bool TREE, typename T>
__global__ void __launch_bounds__(Cfg<D, NR, TERMS>::NW * 32, (Cfg<D, NR, TERMS>::TWO ? 2 : 1)) split_kernel(const AttnParams p) {
  using C = Cfg<D, NR, TERMS>;
  extern __shared__ __align__(128) unsigned char sm[];
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const AttnArgs& A = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, u = lane & 3;
  long long* pre = reinterpret_cast<long long*>(sm + C::O_PRE);
  const uint32_t bar0 = (uint32_t)__cvta_generic_to_shared(sm + C::O_BAR) + warp * C::STAGES * 8;
  unsigned char* ring = sm + warp * C::STAGES * C::BLK;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  if (lane == 0) {
    for (int i = 0; i < C::STAGES; ++i) tqd::mbar_init(bar0 + 8 * i, 1);
    tqd::fence_mbar_init();
  }
  const Plan P = make_plan(p, pre);  // (its barrier also publishes the mbarriers)
  const int most = A.pool.max_blocks * 16;
  // rows that attend to nothing because their sequence is empty: zeros, spread over the grid
  {
    T* out = reinterpret_cast<T*>(A.out);
    for (int b = blockIdx.x; b < A.B; b += gridDim.x)
      if (pre[b + 1] == pre[b])
        for (long long i = threadIdx.x; i < (long long)A.nq * A.Hq * D; i += C::NW * 32)
          out[(long long)b * A.nq * A.Hq * D + i] = from_float<T>(0.f);
  }
  const long long begin = blockIdx.x * P.per, end = min(P.total, begin + P.per);
  bool headed = false;
  if (begin >= end) {
    if (threadIdx.x == 0) p.heads[blockIdx.x].last = -1;
    return;
  }

  // the warp's cursor of copies: runs ahead of the computation, across stretches
  long long c_at = begin;
  Seg c = seg_at(p, pre, c_at, end, find_entry(pre, A.B, begin));
  int c_t = c.t0 + warp, c_base = c_t, c_page = 0;
  bool c_more = true;
  auto pages = [&](int from) {
    const int t = from + C::NW * lane;
    return t < c.t1 ? page_of(A.pool, c.b, t) : 0;
  };
  c_page = pages(c_base);
  QRaw<D, NR, T> raw;  // of the next stretch
  // Rows of entry b that ask.  (A tree's rows past the count are zero queries whose sums are dropped, so that they
  // hide nothing; without a tree their limit of 0 does it.)
  auto asking = [&](int b) { return TREE ? min(p.rows, clamped_count(A.count, b, A.nq) * p.G) : p.rows; };
  request_q<D, NR, T>(raw, A.q, c.b, c.h, p.G, c.rg * 8 * NR, asking(c.b), lane);
  int raw_b = c.b, raw_h = c.h, raw_rg = c.rg;
  uint32_t issued = 0;
  auto issue = [&]() {  // the warp's next tile into the next stage, if there is one
    while (c_more && c_t >= c.t1) {
      c_at = c.next;
      if (c_at >= end) {
        c_more = false;
      } else {
        c = seg_at(p, pre, c_at, end, c.b);
        c_t = c_base = c.t0 + warp;
        c_page = pages(c_base);
      }
    }
    if (!c_more) return;
    if (c_t - c_base >= 32 * C::NW) {
      c_base = c_t;
      c_page = pages(c_base);
    }
    const int page = __shfl_sync(kFull, c_page, (c_t - c_base) / C::NW);
    if (lane == 0) {
      const uint32_t st = issued % C::STAGES;
      tqd::mbar_arrive_expect_tx(bar0 + 8 * st, C::BLK);
      tqd::bulk_g2s(ring_s + st * C::BLK, A.pool.base + pool_block(A.pool, page, c.h) * C::BLK, C::BLK, bar0 + 8 * st);
    }
    ++issued;
    c_t += C::NW;
  };
#pragma unroll 1
  for (int i = 0; i < C::STAGES; ++i) issue();

  uint32_t used = 0, landed = 0;  // (landed: stages whose copy was seen to complete)
  bool alive = true;
  long long at = begin;
  int b_from = find_entry(pre, A.B, begin);
  while (at < end) {
    const Seg s = seg_at(p, pre, at, end, b_from);
    b_from = s.b;
    const int place = at == begin ? 0 : 1;  // (a stretch that is neither the first nor the last covers its slab)
    at = s.next;
    if (s.t0 == s.t1) continue;
    const int len = min(max(__ldg(A.seq_len + s.b), 0), most), cnt = clamped_count(A.count, s.b, A.nq);
    const int row0 = s.rg * 8 * NR, asks = asking(s.b), drafts = len - cnt;  // drafts: the first one's position (TREE)
    QFrag<D, NR, T> q;
    if (raw_b != s.b || raw_h != s.h || raw_rg != s.rg) request_q<D, NR, T>(raw, A.q, s.b, s.h, p.G, row0, asks, lane);
    convert_q<D, NR, T>(q, raw, A.scale, lane);
    int lim[NR][2], least = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = row0 + 8 * r + 2 * u + k;
        lim[r][k] = row >= asks ? 0 : TREE ? max(0, drafts) : row_limit(row / p.G, len, cnt);
        least = min(least, row < asks ? lim[r][k] : 0x7fffffff);
      }
    least = __reduce_min_sync(kFull, least);
    least = min(least, TREE ? max(0, drafts) : len);  // (a tree's drafts are hidden from a group without a row that asks, too)
    auto hide = [&] {
      if constexpr (TREE) return TreeLimits{A.tree, s.b, row0 + 2 * u, p.G, drafts, cnt};
      else return Limits<NR>{lim};
    }();
    State<D, NR> st;
    st.clear();
#pragma unroll 1
    for (int t = s.t0 + warp; t < s.t1; t += C::NW) {
      const uint32_t slot = used % C::STAGES;
      if (alive && !tqd::mbar_wait(bar0 + 8 * slot, (used / C::STAGES) & 1, kWaitLimit)) {
        alive = false;
        if (A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_WAIT_TIMEOUT);
      }
      if (alive)
        tile_step<D, NR, TERMS == 2>(ring + slot * C::BLK, q, st, 16 * t, hide, 16 * t + 16 > least, len, lane);
      __syncwarp();
      ++used;
      if (alive) {
        landed = used;
        issue();
      }
    }
    if (at < end) {  // the next stretch's queries, while the warps meet
      const Seg nx = seg_at(p, pre, at, end, b_from);
      request_q<D, NR, T>(raw, A.q, nx.b, nx.h, p.G, nx.rg * 8 * NR, asking(nx.b), lane);
      raw_b = nx.b, raw_h = nx.h, raw_rg = nx.rg;
    }
    // the warps' states of this stretch into one
    float* ml = reinterpret_cast<float*>(sm + C::O_ML);
    float* red = reinterpret_cast<float*>(sm + C::O_RED);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) st.l[r][k] += __shfl_xor_sync(kFull, st.l[r][k], m);
        if (TREE && row0 + 8 * r + 2 * u + k >= asks) st.l[r][k] = 0.f;
        if (g == 0) {
          ml[2 * (warp * 8 * NR + 8 * r + 2 * u + k)] = st.m[r][k];
          ml[2 * (warp * 8 * NR + 8 * r + 2 * u + k) + 1] = st.l[r][k];
        }
      }
    __syncthreads();
    float f[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mt = -INFINITY;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) mt = fmaxf(mt, ml[2 * (w * 8 * NR + 8 * r + 2 * u + k)]);
        f[r][k] = ex2(st.m[r][k] - (mt == -INFINITY ? 0.f : mt));
      }
    const bool whole = s.t0 == 0 && s.t1 == s.tiles;
    float* part = p.part + (2ll * blockIdx.x + place) * C::PART;
    constexpr int QD = D / 4, PITCH = QD + 4;
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int i = 0; i < QD / 16; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            red[(warp * 8 * NR + 8 * r + 2 * u + (k & 1)) * PITCH + 16 * i + g + 8 * (k >> 1)] =
                st.o[r][qd * (QD / 16) + i][k] * f[r][k & 1];
      __syncthreads();
      for (int i = threadIdx.x; i < 8 * NR * QD; i += C::NW * 32) {
        const int row = i / QD, x = i - row * QD;
        float mt = -INFINITY, lt = 0.f, o = 0.f;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) mt = fmaxf(mt, ml[2 * (w * 8 * NR + row)]);
        const float mr = mt == -INFINITY ? 0.f : mt;
#pragma unroll
        for (int w = 0; w < C::NW; ++w) {
          lt = fmaf(ml[2 * (w * 8 * NR + row) + 1], ex2(ml[2 * (w * 8 * NR + row)] - mr), lt);
          o += red[(w * 8 * NR + row) * PITCH + x];
        }
        const int d = qd * QD + x, rr = row0 + row;
        if (whole) {
          if (rr < p.rows) {
            const int qi = rr / p.G, hd = s.h * p.G + rr - qi * p.G;
            reinterpret_cast<T*>(A.out)[(((long long)s.b * A.nq + qi) * A.Hq + hd) * D + d] =
                from_float<T>(lt > 0.f || lt != lt ? o / lt : 0.f);
          }
        } else {
          part[16 * NR + row * D + d] = o;
          if (d == 0) {
            part[row] = mt;
            part[8 * NR + row] = lt;
          }
        }
      }
      __syncthreads();
    }
    if (threadIdx.x == 0 && s.t0 == 0 && s.t1 < s.tiles) {  // this range's last stretch begins a slab that goes on
      p.heads[blockIdx.x] = JoinHead{(int)((s.start + s.tiles - 1) / P.per), place, s.b, s.h, s.rg};
      headed = true;
    }
  }
  if (threadIdx.x == 0 && !headed) p.heads[blockIdx.x].last = -1;
  if (!alive)  // copies still in flight must land before the block's shared memory is given up
    for (uint32_t i = landed; i < issued; ++i) tqd::mbar_wait(bar0 + 8 * (i % C::STAGES), (i / C::STAGES) & 1, kWaitLimit);
}

template <int D, int NR, int TERMS>
struct RowsCfg {
  static constexpr int BLK = 32 * D + 32;
  static constexpr int ST0 = 200 * 1024 / BLK;
  static constexpr int STAGES = ST0 > 24 ? 24 : ST0;
  static constexpr int O_BAR = STAGES * BLK, SMEM = O_BAR + STAGES * 16;
};

template <int D, int NR, int TERMS, typename T>
__global__ void __launch_bounds__((kWarps + 1) * 32, 1) rows_kernel(const AttnParams p) {
  using C = RowsCfg<D, NR, TERMS>;
  extern __shared__ __align__(128) unsigned char sm[];
  const AttnArgs& A = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, u = lane & 3;
  const int h = blockIdx.y, b = blockIdx.z;
  const int first = (gridDim.x - 1 - blockIdx.x) * kWarps * 8 * NR;  // the longest rows first
  const uint32_t full = (uint32_t)__cvta_generic_to_shared(sm + C::O_BAR), empty = full + 8 * C::STAGES;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      tqd::mbar_init(full + 8 * i, 1);
      tqd::mbar_init(empty + 8 * i, kWarps);
    }
    tqd::fence_mbar_init();
  }
  __syncthreads();
  const int most = A.pool.max_blocks * 16;
  const int len = clamped_len(A.seq_len, b, most, blockIdx.x == 0 && threadIdx.x == 0 && h == 0 ? A.pool.err : nullptr);
  const int cnt = clamped_count(A.count, b, A.nq);
  auto limit_of = [&](int row) { return row < p.rows ? row_limit(row / p.G, len, cnt) : 0; };
  // limits grow with the row up to the count: the largest of rows [r0, r1) is that of the last live row
  auto largest = [&](int r0, int r1) {
    const int last = min(min(r1, p.rows), cnt * p.G) - 1;
    return last < r0 ? 0 : limit_of(last);
  };
  const int tiles = (largest(first, first + kWarps * 8 * NR) + 15) >> 4;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(sm);
  if (warp == kWarps) {
    int page = 0, issued = 0;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      if ((t & 31) == 0) page = t + lane < tiles ? page_of(A.pool, b, t + lane) : 0;
      const int pg = __shfl_sync(kFull, page, t & 31);
      const int st = t % C::STAGES;
      if (t >= C::STAGES) ok = tqd::mbar_wait(empty + 8 * st, ((t / C::STAGES) - 1) & 1, kWaitLimit);
      if (!ok) break;
      if (lane == 0) {
        tqd::mbar_arrive_expect_tx(full + 8 * st, C::BLK);
        tqd::bulk_g2s(ring_s + st * C::BLK, A.pool.base + pool_block(A.pool, pg, h) * C::BLK, C::BLK, full + 8 * st);
      }
      __syncwarp();
      issued = t + 1;
    }
    if (!ok && A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_WAIT_TIMEOUT);
    // every copy issued has landed before the block's shared memory is given up
    for (int t = max(0, issued - C::STAGES); t < issued; ++t)
      tqd::mbar_wait(full + 8 * (t % C::STAGES), (t / C::STAGES) & 1, kWaitLimit);
  } else {
    const int row0 = first + warp * 8 * NR;
    QFrag<D, NR, T> q;
    QRaw<D, NR, T> raw;
    request_q<D, NR, T>(raw, A.q, b, h, p.G, row0, p.rows, lane);
    convert_q<D, NR, T>(q, raw, A.scale, lane);
    int lim[NR][2], least = 0x7fffffff;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        lim[r][k] = limit_of(row0 + 8 * r + 2 * u + k);
        least = min(least, lim[r][k]);
      }
    least = min(__reduce_min_sync(kFull, least), len);
    const int mine = (largest(row0, row0 + 8 * NR) + 15) >> 4;
    State<D, NR> st;
    st.clear();
    bool alive = true;
#pragma unroll 1
    for (int t = 0; t < tiles; ++t) {
      const int slot = t % C::STAGES;
      if (alive && !tqd::mbar_wait(full + 8 * slot, (t / C::STAGES) & 1, kWaitLimit)) {
        alive = false;
        if (A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_WAIT_TIMEOUT);
      }
      if (!alive) break;
      if (t < mine)
        tile_step<D, NR, true>(sm + slot * C::BLK, q, st, 16 * t, Limits<NR>{lim}, 16 * t + 16 > least, len, lane);
      __syncwarp();
      if (lane == 0) asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];\n" ::"r"(empty + 8 * slot) : "memory");
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float l = st.l[r][k];
#pragma unroll
        for (int m = 4; m <= 16; m <<= 1) l += __shfl_xor_sync(kFull, l, m);
        const int row = row0 + 8 * r + 2 * u + k;
        if (row < p.rows) {
          const int qi = row / p.G, hd = h * p.G + row - qi * p.G;
          T* out = reinterpret_cast<T*>(A.out) + (((long long)b * A.nq + qi) * A.Hq + hd) * D;
          const float il = l > 0.f || l != l ? 1.f / l : 0.f;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            out[16 * i + g] = from_float<T>(st.o[r][i][k] * il);
            out[16 * i + g + 8] = from_float<T>(st.o[r][i][k + 2] * il);
          }
        }
      }
  }
  __syncthreads();
}

// Rows per warp: 16 where the registers hold them and there are more than 8.
int row_groups_of(int d, int terms, int rows) { return rows > 8 && d <= 128 ? 2 : 1; }

// A tree's rows per warp: more drafts than 8 rows are the rule, and one pass for 16 is worth the spilled registers of
// 16 bits at d = 256 (64 rows of 4 x 16384 tokens 197 us, 226 with 8 rows).
int tree_row_groups(int d, int terms, int rows) { return rows > 8 && d * terms <= 256 ? 2 : 1; }

template <int D, int NR, int TERMS, bool TREE, typename T>
cudaError_t split_go(AttnParams p, cudaStream_t s) {
  using C = Cfg<D, NR, TERMS>;
  static_assert(C::STAGES >= 2, "ring");
  p.groups = (p.rows + 8 * NR - 1) / (8 * NR);
  const long long most = (long long)p.a.B * p.a.Hkv * p.groups * p.a.pool.max_blocks;
  static std::atomic<uint64_t> done{0};
  int dev;
  long long grid = (long long)sm_count(&dev) * (C::TWO ? 2 : 1);
  if (grid > kMaxGrid) grid = kMaxGrid;
  const long long need = (most + (long long)p.a.B * p.a.Hkv * p.groups * kSlabCost + kMinTiles - 1) / kMinTiles;
  if (grid > need) grid = need;
  p.grid = (int)grid;
  const int smem = C::smem(p.a.B);
  cudaError_t e = allow_smem((const void*)split_kernel<D, NR, TERMS, TREE, T>, C::smem(TQ_MAX_BATCH), dev, done);
  if (e != cudaSuccess) return e;
  split_kernel<D, NR, TERMS, TREE, T><<<p.grid, C::NW * 32, smem, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.grid == 1) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  const int rows = p.rows < 8 * NR ? p.rows : 8 * NR;
  cfg.gridDim = dim3(p.grid - 1, rows);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D, 8 * NR, kJoinWarps, T>, JoinParams{p.heads, p.part, p.a.out, p.a.nq, p.a.Hq, p.G, p.rows});
}

template <int D, int NR, int TERMS, typename T>
cudaError_t rows_go(AttnParams p, cudaStream_t s) {
  using C = RowsCfg<D, NR, TERMS>;
  static std::atomic<uint64_t> done{0};
  int dev;
  sm_count(&dev);
  cudaError_t e = allow_smem((const void*)rows_kernel<D, NR, TERMS, T>, C::SMEM, dev, done);
  if (e != cudaSuccess) return e;
  const dim3 grid((p.rows + kWarps * 8 * NR - 1) / (kWarps * 8 * NR), p.a.Hkv, p.a.B);
  rows_kernel<D, NR, TERMS, T><<<grid, (kWarps + 1) * 32, C::SMEM, s>>>(p);
  return cudaGetLastError();
}

// From five row groups on the rows kernel takes a call, because the split reads the pool once per group.  That is
// right for grids that fill the GPU and many rows (32 / 8 heads, fp32, d = 128, 8 x 16384 tokens: 256 rows, split 1238 us,
// rows kernel 1120), and wrong below: 80 rows of the same 399 and 1119 us; one sequence of 131072 tokens 380 and 8821 us;
// at d = 256 40 rows of one such sequence 404 and 5701 us.  The rule does not look at the grid.
bool use_rows(int groups) { return groups > 4; }

template <int D, int TERMS, typename T>
cudaError_t attention_d(const AttnParams& p, cudaStream_t s) {
  constexpr bool wide = D <= 128;
  const int nr = row_groups_of(D, TERMS, p.rows);
  const bool rows = use_rows((p.rows + 8 * nr - 1) / (8 * nr));
  if constexpr (wide) {
    if (nr == 2) return rows ? rows_go<D, 2, TERMS, T>(p, s) : split_go<D, 2, TERMS, false, T>(p, s);
  }
  return rows ? rows_go<D, 1, TERMS, T>(p, s) : split_go<D, 1, TERMS, false, T>(p, s);
}

template <int D, int TERMS, typename T>
cudaError_t tree_d(const AttnParams& p, cudaStream_t s) {
  if constexpr (D * TERMS <= 256) {
    if (tree_row_groups(D, TERMS, p.rows) == 2) return split_go<D, 2, TERMS, true, T>(p, s);
  }
  return split_go<D, 1, TERMS, true, T>(p, s);
}

template <int D>
cudaError_t attention_type(const AttnParams& p, cudaStream_t s) {
  if (p.a.tree.bits) {
    if (p.a.dtype == TQ_F32) return tree_d<D, 2, float>(p, s);
    return p.a.dtype == TQ_BF16 ? tree_d<D, 1, __nv_bfloat16>(p, s) : tree_d<D, 1, __half>(p, s);
  }
  if (p.a.dtype == TQ_F32) return attention_d<D, 2, float>(p, s);
  if (p.a.dtype == TQ_BF16) return attention_d<D, 1, __nv_bfloat16>(p, s);
  return attention_d<D, 1, __half>(p, s);
}

cudaError_t by_head_dim(const AttnArgs& a, cudaStream_t s) {
  AttnParams p;
  p.a = a;
  p.G = a.Hq / a.Hkv;
  p.rows = p.G * a.nq;
  p.groups = 0;
  p.grid = 0;
  p.heads = (JoinHead*)a.ws;
  p.part = (float*)((unsigned char*)a.ws + kJoinHeadBytes);
  switch (a.d) {
    case 64: return attention_type<64>(p, s);
    case 128: return attention_type<128>(p, s);
    case 256: return attention_type<256>(p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// SMs of the current device, and its index (looked up once per device).
int sm_count(int* device) {
  static std::atomic<int> known[64];
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) dev = -1;
  *device = dev;
  if (dev >= 0 && dev < 64 && (n = known[dev].load(std::memory_order_relaxed)) > 0) return n;
  if (dev < 0 || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 152;
  if (dev < 64) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Lets a kernel use `bytes` of shared memory on the device, once per kernel and device (`done`:
// the kernel's own bit set; `bytes` is then its largest).
cudaError_t allow_smem(const void* kernel, int bytes, int device, std::atomic<uint64_t>& done) {
  const uint64_t bit = device >= 0 && device < 64 ? 1ull << device : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

size_t byte_attention_workspace(int d, int B, int nq, int Hq, int Hkv, tq_dtype dtype) {
  const int rows = Hq / Hkv * nq, nr = row_groups_of(d, dtype == TQ_F32 ? 2 : 1, rows);
  const int groups = (rows + 8 * nr - 1) / (8 * nr);
  size_t need = use_rows(groups) ? 256 : kJoinHeadBytes + (size_t)2 * kMaxGrid * 8 * nr * (d + 2) * sizeof(float);
  if (d == 128 && dtype != TQ_F32 && rows > kTcMinRows && tc_workspace(rows) > need) need = tc_workspace(rows);
  return need;
}

size_t tree_attention_workspace(int d, int B, int nq, int Hq, int Hkv, tq_dtype dtype) {
  (void)B;
  const int rows = Hq / Hkv * nq, nr = tree_row_groups(d, dtype == TQ_F32 ? 2 : 1, rows);
  const size_t split = kJoinHeadBytes + (size_t)2 * kMaxGrid * 8 * nr * (d + 2) * sizeof(float);
  const size_t tc = tree_tc_workspace(d, rows, dtype);
  return tc > split ? tc : split;
}

tq_status launch_byte_attention(const AttnArgs& a, Stream s) {
  return cuda_error("byte attention", tc_takes(a) ? launch_tc(a, (cudaStream_t)s) : by_head_dim(a, (cudaStream_t)s));
}

tq_status launch_tree_attention(const AttnArgs& a, Stream s) {
  return cuda_error("tree attention", tree_tc_takes(a) ? launch_tree_tc(a, (cudaStream_t)s) : by_head_dim(a, (cudaStream_t)s));
}

}  // namespace tqb
