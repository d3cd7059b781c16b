// Head norms with the position rotation (norm_rotate), and the append of keys and values into the
// byte cache with that norm and rotation on the way (byte_append).
//
// norm_rotate reads every row once and writes it once: bound by HBM for chunks, by the launch and
// the chain position -> angle -> row for single tokens.  A block of 256 threads takes a few tokens
// and all their heads, so a token's sines are computed once for its 2 * heads rows; three blocks an SM
// with three rows in flight per thread carry the latency.  Measured: 4096 tokens of 64 + 8 heads, d = 128,
// bf16, 31 us, 4.9 TB/s of the 6.8 of a copy (a copy of this size: 24 us); 57 % of issue slots, so the
// arithmetic (packed fp32) is the next bound; one token of 8 sequences 2.6 us.
//
// byte_append gives each warp one side of one 16-token block of one KV head: it reads the block's
// new rows, rotates keys, finds the block's scale with a warp maximum, and writes the codes; held
// codes are rounded to a raised scale by the same warp, so a block has one writer.  The queries of
// the step ride along as further blocks of the grid.  Measured: 4096 tokens of 64 + 8 heads 37 us (17 us
// without the queries: a chain of dependent loads in 514 blocks; a copy of all bytes takes 25 us; warps also
// wait for instructions, the code of both kinds of block being live at once); one token of 8 sequences 5.8 us.
#include <string>

#include "tq_byte_attn.cuh"
#include "tq_rotate.cuh"

namespace tqb {
namespace {

constexpr int kThreads = 256;

// Cosines and sines of tokens [0, count) at pos(token, axis) into cs ([token][r floats], pair_slot order).
template <typename F>
__device__ __forceinline__ void fill_angles(float* cs, const Rotary& R, int count, F pos) {
  const int half = R.r / 2;
  for (int i = threadIdx.x; i < count * half; i += blockDim.x) {
    const int tk = i / half, p = i - tk * half;
    const uint64_t entry = __ldg(reinterpret_cast<const unsigned long long*>(R.table) + p);
    float* at = cs + 2 * tk * half + pair_slot(p, R.r, R.interleaved);
    const float2 v = pair_angle(entry, [&](int axis) { return pos(tk, axis); });
    at[0] = v.x;
    at[2] = v.y;
  }
}

template <typename T>
__device__ __forceinline__ void load_weight(const void* w, int ca, int cb, float (&wa)[8], float (&wb)[8]) {
  if (w) {
    unpack8(load8(reinterpret_cast<const T*>(w) + 8 * ca), wa);
    unpack8(load8(reinterpret_cast<const T*>(w) + 8 * cb), wb);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.f;
  }
}

// Where the rows of a block's tokens begin: source, and destination of keys ([B][heads][n][D]).
struct TokenAt {
  long long src, dst;
};
constexpr int kMaxTokens = 16;  // of a block

template <bool KEYS>
__device__ __forceinline__ void fill_tokens(TokenAt* tok, const Rows& X, int t0, int nt, int n, int D) {
  if ((int)threadIdx.x < nt) {
    const int g = t0 + threadIdx.x, b = g / n, j = g - b * n;
    tok[threadIdx.x].src = b * X.sb + j * X.st;
    tok[threadIdx.x].dst = KEYS ? ((long long)b * X.heads * n + j) * D : (long long)g * X.heads * D;
  }
}

// Rows of heads [h0, h0 + nh) of a block's nt tokens: normed, rotated and stored at out + tok.dst +
// h * out_head.  Loads of kU rows are in flight per thread; `angles` (which writes the tokens' cosines)
// runs once, behind the first loads.  Rows are walked without divisions: those and the address
// arithmetic were half of the pass's instructions.
template <int D, typename T, typename O, int kU, typename A>
__device__ __forceinline__ void rows_pass(const Rows& X, const TokenAt* tok, const void* w, float eps, const Rotary& R,
                                          const float4* cs, int nt, int h0, int nh, O* out, long long out_head, bool& filled,
                                          A angles) {
  constexpr int TPR = D / 16, RPP = kThreads / TPR;
  const int l = threadIdx.x % TPR, row0 = threadIdx.x / TPR;
  const int ca = chunk_a(l, R.r), cb = chunk_b(l, R.r);
  const int total = nt * nh, step_t = RPP / nh, step_h = RPP - step_t * nh;
  int tk = row0 / nh, h = row0 - tk * nh;  // of the next row to load
  float wa[8], wb[8];
  load_weight<T>(w, ca, cb, wa, wb);
  for (int base = 0; base < total; base += RPP * kU) {
    Raw8<T> ra[kU], rb[kU];
    int tks[kU], hs[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      tks[u] = tk;
      hs[u] = h0 + h;
      if (tk < nt) {
        const T* src = reinterpret_cast<const T*>(X.p) + tok[tk].src + hs[u] * X.sh;
        ra[u] = load8_rw(src + 8 * ca);
        rb[u] = load8_rw(src + 8 * cb);
      } else {
        ra[u] = Raw8<T>{};
        rb[u] = Raw8<T>{};
      }
      tk += step_t;
      h += step_h;
      if (h >= nh) {
        h -= nh;
        ++tk;
      }
    }
    if (!filled) {
      angles();
      __syncthreads();
      filled = true;
    }
    uint32_t again = 0;  // rows whose squares leave fp32's range
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (base + u * RPP >= total) break;  // (uniform over the block)
      float a[8], b[8];
      unpack8(ra[u], a);
      unpack8(rb[u], b);
      const bool live = tks[u] < nt;
      const bool far = norm_rotate_row<TPR, kNear>(a, b, l, w != nullptr, wa, wb, D, eps, cs + (live ? tks[u] : 0) * (R.r / 4), R.r,
                                                   R.interleaved);
      if (live && !far) {
        O* dst = out + tok[tks[u]].dst + hs[u] * out_head;
        store8(dst + 8 * ca, a);
        store8(dst + 8 * cb, b);
      }
      if (far) again |= 1u << u;
    }
    if (__any_sync(kFull, again)) {  // (indexes and weights once more: nothing of this is held through the loop)
      float va[8], vb[8];
      load_weight<T>(w, ca, cb, va, vb);
#pragma unroll 1
      for (int u = 0; u < kU; ++u) {
        const int row = base + u * RPP + row0;
        const bool mine = (again >> u & 1) && row < total;
        const int tk1 = mine ? row / nh : 0, h1 = h0 + row - row / nh * nh;
        Raw8<T> xa = {}, xb = {};
        if (mine) {  // (not stored yet, also where the output is the input's buffer)
          const T* src = reinterpret_cast<const T*>(X.p) + tok[tk1].src + h1 * X.sh;
          xa = load8_rw(src + 8 * ca);
          xb = load8_rw(src + 8 * cb);
        }
        float a[8], b[8];
        unpack8(xa, a);
        unpack8(xb, b);
        norm_rotate_row<TPR, kFar>(a, b, l, true, va, vb, D, eps, cs + tk1 * (R.r / 4), R.r, R.interleaved);
        if (mine) {
          O* dst = out + tok[tk1].dst + h1 * out_head;
          store8(dst + 8 * ca, a);
          store8(dst + 8 * cb, b);
        }
      }
    }
  }
}

struct RotateParams {
  RotateArgs a;
  int tokens;      // B n
  int per;         // tokens per block
  int q_split;     // blocks over the heads: blockIdx.y takes heads [y * q_split, ...) of q then k
};

template <int D, typename T, typename O>
__global__ void __launch_bounds__(kThreads, 3) norm_rotate_kernel(const RotateParams p) {
  extern __shared__ __align__(16) float cs[];
  __shared__ TokenAt tok[2][kMaxTokens];
  const RotateArgs& A = p.a;
  const int t0 = blockIdx.x * p.per, nt = min(p.per, p.tokens - t0);
  auto angles = [&] {
    if (A.rot.r)
      fill_angles(cs, A.rot, nt, [&](int tk, int axis) {
        const int g = t0 + tk, b = g / A.n;
        return token_position(A.pos, axis, b, g - b * A.n, A.B, A.n);
      });
  };
  // heads of q and k in one range [0, Hq + Hk)
  const int lo = blockIdx.y * p.q_split, hi = min(lo + p.q_split, A.q.heads + A.k.heads);
  const int q0 = min(lo, A.q.heads), q1 = min(hi, A.q.heads);
  const int k0 = max(lo, A.q.heads) - A.q.heads, k1 = max(hi, A.q.heads) - A.q.heads;
  fill_tokens<false>(tok[0], A.q, t0, nt, A.n, D);
  fill_tokens<true>(tok[1], A.k, t0, nt, A.n, D);
  __syncthreads();
  bool filled = false;
  constexpr int kU = sizeof(T) == 2 ? 3 : 2;
  const float4* c4 = reinterpret_cast<const float4*>(cs);
  if (q1 > q0)
    rows_pass<D, T, O, kU>(A.q, tok[0], A.wq, A.eps, A.rot, c4, nt, q0, q1 - q0, reinterpret_cast<O*>(A.q_out), D, filled, angles);
  if (k1 > k0)
    rows_pass<D, T, O, kU>(A.k, tok[1], A.wk, A.eps, A.rot, c4, nt, k0, k1 - k0, reinterpret_cast<O*>(A.k_out),
                           (long long)A.n * D, filled, angles);
}

struct AppendParams {
  AppendArgs a;
  int blocks;      // 16-token blocks a batch entry's tokens can touch
  int groups;      // head groups of 4
  int kv_blocks;   // B * blocks * groups; the other grid blocks take queries
  int every;       // grid block i * every is kv block i: the append's blocks wait on memory in long
                   // chains, so they are spread among the queries' (4096 tokens of 64 + 8 heads: 17 us
                   // and 26 us each kind alone, 37 us so)
  int per, tokens, q_split, q_groups;
};

// E = 2, 4 or 8 consecutive elements as loaded, and as fp32.
template <typename T, int E>
struct RawE {
  static constexpr int W = E * (int)sizeof(T) / 4;  // 32-bit words
  uint32_t w[W];
};
template <typename T, int E>
__device__ __forceinline__ RawE<T, E> load_some(const T* p) {
  RawE<T, E> r;
  constexpr int W = RawE<T, E>::W;
  if constexpr (W == 1) {
    r.w[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  } else if constexpr (W == 2) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x; r.w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < W / 4; ++i) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
      r.w[4 * i] = v.x; r.w[4 * i + 1] = v.y; r.w[4 * i + 2] = v.z; r.w[4 * i + 3] = v.w;
    }
  }
  return r;
}
template <int E>
__device__ __forceinline__ void unpack_some(const RawE<float, E>& r, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E; ++i) x[i] = __uint_as_float(r.w[i]);
}
template <int E>
__device__ __forceinline__ void unpack_some(const RawE<__nv_bfloat16, E>& r, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    x[2 * i] = __uint_as_float(r.w[i] << 16);
    x[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
template <int E>
__device__ __forceinline__ void unpack_some(const RawE<__half, E>& r, float (&x)[E]) {
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r.w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

// Element i of those.
template <int E>
__device__ __forceinline__ float element(const RawE<float, E>& r, int i) { return __uint_as_float(r.w[i]); }
template <int E>
__device__ __forceinline__ float element(const RawE<__nv_bfloat16, E>& r, int i) {
  return __uint_as_float(i & 1 ? r.w[i >> 1] & 0xffff0000u : r.w[i >> 1] << 16);
}
template <int E>
__device__ __forceinline__ float element(const RawE<__half, E>& r, int i) {
  return __half2float(__ushort_as_half((unsigned short)(i & 1 ? r.w[i >> 1] >> 16 : r.w[i >> 1])));
}

// The block's scale exponent from its new tokens' largest magnitude and, where it holds tokens, its
// old one; the scale is stored and the old exponent returned in e_old.
__device__ __forceinline__ int block_scale(float amax, int held, float old_scale, float* scale, int lane, int& e_old) {
  int e = scale_exponent(tqd::warp_max(amax));
  e_old = e;
  if (held > 0) {
    e_old = min(kEMax, max(kEMin, log2i(old_scale)));
    e = max(e, e_old);
  }
  if (lane == 0) *scale = exp2i(e);
  return e;
}

// Running largest magnitude, and 0 * x summed: NaN as soon as one x is infinite or NaN.
struct Magnitude {
  float top = 0.f;
  uint64_t zero = 0;
  __device__ __forceinline__ void add(float a, float b) {
    top = fmaxf(top, fmaxf(fabsf(a), fabsf(b)));
    zero = fma2(pair(a, b), 0, zero);
  }
  __device__ __forceinline__ bool odd() const {
    float x, y;
    unpair(zero, x, y);
    return x + y != 0.f;
  }
};

// The warp's rows [lo, hi) of one block of keys.  rot: the warp's shared memory for its rotated rows
// (fp32, 16 D of them): a thread reads back what it wrote, so that it need not hold 64 values (d = 128)
// from the maximum to the codes, which would cost the occupancy that the loads need.
template <int D, typename T, typename B, typename F>
__device__ __forceinline__ bool append_keys(const AppendArgs& A, B block, const float4* cs, float4* rot, int b, int h,
                                            long long j0, int lo, int hi, int held, int lane, F angles) {
  constexpr int TPR = D / 16, RPW = 32 / TPR, NP = 16 / RPW;
  const int l = lane % TPR, r0 = lane / TPR;
  const int ca = chunk_a(l, A.rot.r), cb = chunk_b(l, A.rot.r);
  const T* src = reinterpret_cast<const T*>(A.k.p) + b * A.k.sb + h * A.k.sh;
  Raw8<T> ra[NP], rc[NP];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int s = p * RPW + r0;
    ra[p] = rc[p] = Raw8<T>{};
    if (s >= lo && s < hi) {
      const T* row = src + (j0 + s) * A.k.st;
      ra[p] = load8(row + 8 * ca);
      rc[p] = load8(row + 8 * cb);
    }
  }
  float wa[8], wb[8];
  load_weight<T>(A.wk, ca, cb, wa, wb);
  angles();
  __syncthreads();
  unsigned char* blk = block();
  float* scale = reinterpret_cast<float*>(blk + 32 * D);
  const float old_scale = held > 0 ? *scale : 1.f;
  rot += lane;
  Magnitude mag;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    if (p * RPW + RPW <= lo || p * RPW >= hi) continue;  // (uniform over the warp)
    const int s = p * RPW + r0;
    float a[8], c[8];
    unpack8(ra[p], a);
    unpack8(rc[p], c);
    // (slots without a new token go along as zeros, with the cosines of an existing slot, and count for nothing)
    const bool live = s >= lo && s < hi;
    norm_rotate_row<TPR, kAll>(a, c, l, A.wk != nullptr, wa, wb, D, A.eps, cs + (live ? s : lo) * (A.rot.r / 4), A.rot.r,
                         A.rot.interleaved);
    if (live) {
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        mag.add(a[i], a[i + 1]);
        mag.add(c[i], c[i + 1]);
      }
      rot[(4 * p + 0) * 32] = make_float4(a[0], a[1], a[2], a[3]);
      rot[(4 * p + 1) * 32] = make_float4(a[4], a[5], a[6], a[7]);
      rot[(4 * p + 2) * 32] = make_float4(c[0], c[1], c[2], c[3]);
      rot[(4 * p + 3) * 32] = make_float4(c[4], c[5], c[6], c[7]);
    }
  }
  const bool odd = __any_sync(kFull, mag.odd());
  if (odd) {  // infinities and NaN do not count for the scale
    mag.top = 0.f;
    for (int i = 0; i < 4 * NP; ++i) {
      const int s = (i >> 2) * RPW + r0;
      if (s < lo || s >= hi) continue;
      const float4 v = rot[i * 32];
      mag.top = fmaxf(mag.top, fmaxf(fmaxf(finite_abs(v.x), finite_abs(v.y)), fmaxf(finite_abs(v.z), finite_abs(v.w))));
    }
  }
  int e_old;
  const int e = block_scale(mag.top, held, old_scale, scale, lane, e_old);
  const float inv = exp2i(-e);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int s = p * RPW + r0;
    if (s < lo || s >= hi) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 v = rot[(4 * p + 2 * k) * 32], u = rot[(4 * p + 2 * k + 1) * 32];
      const float x[8] = {v.x * inv, v.y * inv, v.z * inv, v.w * inv, u.x * inv, u.y * inv, u.z * inv, u.w * inv};
      const uint2 w = odd ? make_uint2(encode4(x), encode4(x + 4)) : make_uint2(encode4_finite(x), encode4_finite(x + 4));
      const int ch = k ? cb : ca;
      *reinterpret_cast<uint2*>(blk + k_chunk<D>(s, ch >> 1) + 8 * (ch & 1)) = w;
    }
  }
  if (e > e_old && held > 0) {  // held rows to the raised scale, 16 codes at a time
    const float f = exp2i(e_old - e);
    for (int i = lane; i < held * (D / 16); i += 32) {
      uint4* at = reinterpret_cast<uint4*>(blk + k_chunk<D>(i / (D / 16), i % (D / 16)));
      uint4 v = *at;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float x[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) x[m] = decode1((unsigned char)(w[u] >> (8 * m))) * f;
        w[u] = encode4(x);
      }
      *at = v;
    }
  }
  return odd;
}

template <int D, typename T, typename B, typename F>
__device__ __forceinline__ bool append_values(const AppendArgs& A, B block, int b, int h, long long j0, int lo, int hi,
                                              int held, int lane, F angles) {
  constexpr int E = D / 32;  // coordinates E * lane .. of all 16 tokens
  const T* src = reinterpret_cast<const T*>(A.v.p) + b * A.v.sb + h * A.v.sh + E * lane;
  RawE<T, E> raw[16];
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    raw[s] = RawE<T, E>{};
    if (s >= lo && s < hi) raw[s] = load_some<T, E>(src + (j0 + s) * A.v.st);
  }
  angles();
  __syncthreads();  // (the block's barrier for the key warps' cosines)
  unsigned char* blk = block();
  float* scale = reinterpret_cast<float*>(blk + 32 * D + 4);
  const float old_scale = held > 0 ? *scale : 1.f;
  Magnitude mag;
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    float x[E];
    unpack_some<E>(raw[s], x);
#pragma unroll
    for (int i = 0; i < E; i += 2) mag.add(x[i], x[i + 1]);
  }
  const bool odd = __any_sync(kFull, mag.odd());
  if (odd) {  // infinities and NaN do not count for the scale
    mag.top = 0.f;
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      float x[E];
      unpack_some<E>(raw[s], x);
#pragma unroll
      for (int i = 0; i < E; ++i) mag.top = fmaxf(mag.top, finite_abs(x[i]));
    }
  }
  int e_old;
  const int e = block_scale(mag.top, held, old_scale, scale, lane, e_old);
  const float inv = exp2i(-e);
  const bool raise = held > 0 && e > e_old;
  const float f = exp2i(e_old - e);
  unsigned char* vb = blk + 16 * D + 16 * E * lane;
#pragma unroll
  for (int i = 0; i < E; ++i) {
    uint32_t w[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {  // tokens 2u, 2u + 1, 2u + 8, 2u + 9
      const float four[4] = {element<E>(raw[2 * u], i) * inv, element<E>(raw[2 * u + 1], i) * inv,
                             element<E>(raw[2 * u + 8], i) * inv, element<E>(raw[2 * u + 9], i) * inv};
      w[u] = odd ? encode4(four) : encode4_finite(four);
    }
    if (lo == 0 && hi == 16) {
      *reinterpret_cast<uint4*>(vb + 16 * i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        unsigned char* at = vb + 16 * i + v_slot(s);
        if (s >= lo && s < hi)
          *at = (unsigned char)(w[v_slot(s) >> 2] >> (8 * (v_slot(s) & 3)));
        else if (raise && s < held)
          *at = (unsigned char)encode2(decode1(*at) * f, 0.f);
      }
    }
  }
  return odd;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, (D * sizeof(T) <= 256 ? 3 : 1)) byte_append_kernel(const AppendParams p) {
  extern __shared__ __align__(16) float cs[];
  const AppendArgs& A = p.a;
  const int turn = (int)blockIdx.x / p.every;
  if (turn >= p.kv_blocks || (int)blockIdx.x != turn * p.every) {  // queries
    const int i = blockIdx.x - min(p.kv_blocks, turn + 1), part = i % p.q_groups, t0 = i / p.q_groups * p.per;
    const int nt = min(p.per, p.tokens - t0), h0 = part * p.q_split, nh = min(p.q_split, A.Hq - h0);
    __shared__ TokenAt tok[kMaxTokens];
    fill_tokens<false>(tok, A.q, t0, nt, A.n, D);
    __syncthreads();
    bool filled = false;
    auto angles = [&] {
      if (A.rot.r)
        fill_angles(cs, A.rot, nt, [&](int tk, int axis) {
          const int g = t0 + tk, b = g / A.n;
          return token_position(A.pos, axis, b, g - b * A.n, A.B, A.n);
        });
    };
    rows_pass<D, T, T, (sizeof(T) == 2 ? 3 : 2)>(A.q, tok, A.wq, A.eps, A.rot, reinterpret_cast<const float4*>(cs), nt, h0, nh,
                                                 reinterpret_cast<T*>(A.q_out), D, filled, angles);
    return;
  }
  const int hg = turn % p.groups, rest = turn / p.groups;
  const int i = rest % p.blocks, b = rest / p.blocks;
  const int start = __ldg(A.start + b);
  const int count = A.count ? min(A.n, __ldg(A.count + b)) : A.n;
  const int first = start >> 4;                            // (floor, also of a negative start)
  const long long tile = (long long)first + i;
  const long long j0 = tile * 16 - start;                  // the token at the block's slot 0
  const int lo = (int)max(0ll, -j0), hi = (int)min(16ll, (long long)count - j0);
  if (hi <= lo) return;                                    // (uniform over the block)
  const int held = i == 0 ? (start & 15) : 0;              // = lo in the first block
  auto angles = [&] {
    if (A.rot.r) {
      const int half = A.rot.r / 2;
      for (int u = threadIdx.x; u < (hi - lo) * half; u += kThreads) {
        const int s = lo + u / half, pr = u % half;
        const uint64_t entry = __ldg(reinterpret_cast<const unsigned long long*>(A.rot.table) + pr);
        float* at = cs + 2 * s * half + pair_slot(pr, A.rot.r, A.rot.interleaved);
        const float2 v = pair_angle(entry, [&](int axis) { return token_position(A.pos, axis, b, (int)(j0 + s), A.B, A.n); });
        at[0] = v.x;
        at[2] = v.y;
      }
    }
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = hg * 4 + (warp >> 1);
  if (h >= A.pool.heads) {
    angles();
    __syncthreads();
    return;
  }
  // the table's entry is requested here and looked at behind the rows' loads
  const int entry = tile >= 0 && tile < A.pool.max_blocks ? __ldg(A.pool.table + (long long)b * A.pool.max_blocks + tile) : -1;
  auto block = [&] {
    int page = entry;
    if ((unsigned)page >= (unsigned)A.pool.num_pages) {
      if (A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_BAD_PAGE);
      page = A.pool.num_pages;
    }
    return A.pool.base + pool_block(A.pool, page, h) * block_bytes(D);
  };
  const bool bad = (warp & 1) ? append_values<D, T>(A, block, b, h, j0, lo, hi, held, lane, angles)
                              : append_keys<D, T>(A, block, reinterpret_cast<const float4*>(cs),
                                                    reinterpret_cast<float4*>(cs + 16 * A.rot.r) + (warp >> 1) * 4 * D, b, h, j0, lo, hi, held, lane, angles);
  if (bad && A.pool.err) atomicExch(A.pool.err, TQ_DEVERR_NONFINITE);
}

template <int D>
__global__ void __launch_bounds__(256) byte_dequantize_kernel(const Pool P, int b, int h, int t0, int t1, float* k, float* v) {
  const long long total = (long long)(t1 - t0) * D;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    const int t = t0 + (int)(i / D), x = (int)(i % D);
    const unsigned char* blk = P.base + pool_block(P, page_of(P, b, t >> 4), h) * block_bytes(D);
    const float* s = reinterpret_cast<const float*>(blk + 32 * D);
    k[i] = decode1(blk[k_chunk<D>(t & 15, x >> 4) + (x & 15)]) * s[0];
    v[i] = decode1(blk[16 * D + 16 * x + v_slot(t & 15)]) * s[1];
  }
}

// Tokens per block and heads per block of a rows pass: enough rows for a few passes of the block's
// threads per set of cosines, unless that leaves SMs without a block; single tokens spread their
// heads over blocks instead, one pass each.
void rows_split(int d, int tokens, int heads, int* per, int* split) {
  const int rpp = kThreads / (d / 16);
  *split = heads;
  *per = (6 * rpp + heads - 1) / heads;
  const int fill = (tokens + 455) / 456;  // three blocks on each of 152 SMs
  if (*per > fill) *per = fill;
  if (*per > kMaxTokens) *per = kMaxTokens;
  if (*per < 1) *per = 1;
  if (tokens <= 304 && heads > rpp) *split = rpp;
}

template <int D, typename T, typename O>
cudaError_t rotate_go(const RotateArgs& a, cudaStream_t s) {
  RotateParams p;
  p.a = a;
  p.tokens = a.B * a.n;
  const int heads = a.q.heads + a.k.heads;
  rows_split(D, p.tokens, heads, &p.per, &p.q_split);
  const dim3 grid((p.tokens + p.per - 1) / p.per, (heads + p.q_split - 1) / p.q_split);
  norm_rotate_kernel<D, T, O><<<grid, kThreads, (size_t)p.per * a.rot.r * sizeof(float), s>>>(p);
  return cudaGetLastError();
}
template <int D, typename T>
cudaError_t rotate_out(const RotateArgs& a, cudaStream_t s) {
  return a.out_dtype == TQ_F32 ? rotate_go<D, T, float>(a, s) : rotate_go<D, T, T>(a, s);
}
template <int D>
cudaError_t rotate_type(const RotateArgs& a, cudaStream_t s) {
  if (a.dtype == TQ_F32) return rotate_go<D, float, float>(a, s);
  if (a.dtype == TQ_BF16) return rotate_out<D, __nv_bfloat16>(a, s);
  return rotate_out<D, __half>(a, s);
}

template <int D, typename T>
cudaError_t append_go(const AppendArgs& a, cudaStream_t s) {
  AppendParams p;
  p.a = a;
  p.blocks = (15 + a.n + 15) / 16;
  p.groups = (a.pool.heads + 3) / 4;
  p.kv_blocks = a.B * p.blocks * p.groups;
  p.tokens = a.B * a.n;
  p.per = 1;
  p.q_split = p.q_groups = 1;
  int q_blocks = 0;
  if (a.q.heads) {
    rows_split(D, p.tokens, a.Hq, &p.per, &p.q_split);
    p.q_groups = (a.Hq + p.q_split - 1) / p.q_split;
    q_blocks = (p.tokens + p.per - 1) / p.per * p.q_groups;
  }
  p.every = (p.kv_blocks + q_blocks) / p.kv_blocks;
  const int tk = p.per > 16 ? p.per : 16;
  // the cosines of a block's tokens, and its four key warps' rotated rows
  const size_t smem = (size_t)tk * a.rot.r * sizeof(float) + 4 * 16 * D * sizeof(float);
  static std::atomic<uint64_t> done{0};
  int dev;
  sm_count(&dev);
  const cudaError_t e = allow_smem((const void*)byte_append_kernel<D, T>, 2 * 4 * 16 * D * sizeof(float), dev, done);
  if (e != cudaSuccess) return e;
  byte_append_kernel<D, T><<<p.kv_blocks + q_blocks, kThreads, smem, s>>>(p);
  return cudaGetLastError();
}
template <int D>
cudaError_t append_type(const AppendArgs& a, cudaStream_t s) {
  if (a.dtype == TQ_F32) return append_go<D, float>(a, s);
  if (a.dtype == TQ_BF16) return append_go<D, __nv_bfloat16>(a, s);
  return append_go<D, __half>(a, s);
}

}  // namespace

tq_status cuda_error(const char* what, int e) {
  if (e == 0) return TQ_OK;
  tqi::set_error(std::string(what) + ": " + cudaGetErrorString((cudaError_t)e));
  return TQ_ERR_CUDA;
}

tq_status launch_norm_rotate(const RotateArgs& a, Stream s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.d) {
    case 64: e = rotate_type<64>(a, (cudaStream_t)s); break;
    case 128: e = rotate_type<128>(a, (cudaStream_t)s); break;
    case 256: e = rotate_type<256>(a, (cudaStream_t)s); break;
    case 512: e = rotate_type<512>(a, (cudaStream_t)s); break;
  }
  return cuda_error("norm_rotate", e);
}

tq_status launch_byte_append(const AppendArgs& a, Stream s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.d) {
    case 64: e = append_type<64>(a, (cudaStream_t)s); break;
    case 128: e = append_type<128>(a, (cudaStream_t)s); break;
    case 256: e = append_type<256>(a, (cudaStream_t)s); break;
  }
  return cuda_error("byte append", e);
}

tq_status launch_byte_dequantize(const Pool& pool, int d, int b, int h, int t0, int t1, float* k, float* v, Stream s) {
  const long long total = (long long)(t1 - t0) * d;
  const int grid = (int)(total / 256 + 1 < 1216 ? total / 256 + 1 : 1216);
  switch (d) {
    case 64: byte_dequantize_kernel<64><<<grid, 256, 0, (cudaStream_t)s>>>(pool, b, h, t0, t1, k, v); break;
    case 128: byte_dequantize_kernel<128><<<grid, 256, 0, (cudaStream_t)s>>>(pool, b, h, t0, t1, k, v); break;
    case 256: byte_dequantize_kernel<256><<<grid, 256, 0, (cudaStream_t)s>>>(pool, b, h, t0, t1, k, v); break;
  }
  return cuda_error("byte dequantize", cudaGetLastError());
}

}  // namespace tqb
