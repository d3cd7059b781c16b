// What a step of drafted trees does beside its attention, and reading a cache back:
//
// draft_tree: a thread per draft, rows of bits in shared memory.  Each round a row takes in the row of the ancestor that
// it points at and points where that one does, so a tree of depth h takes log2(h) rounds.  (Threads that walked to the
// root took 140 ns a step: 16 us for 256 trees of 250 drafts and depth 100, 398 us for a chain of 1024; here 5.6 and 30.)
//
// byte_keep: the accepted path's tokens to where a plain decode would have put them.  A warp per (entry, KV head,
// side) takes the blocks that receive tokens in order: every token comes from its own place or a later one, so what
// a block takes is still there when its turn comes, and nobody else writes these blocks.  Bound by the launch and
// the chain path -> table -> scales and codes -> store, once per 16 kept tokens: 5 of 16 drafts of 8 sequences, 8 KV heads,
// d = 128 3.6 us, 20 of 64 of 256 sequences 13.4 us.  (V bytes one by one, all in flight; whole 16-byte words of each block
// that tokens come from, one block after the other, 4.0 and 15.5 us.)
//
// byte_read: values of a batch, both sides, code * 2^e.  A warp per (entry, KV head, block).  Bound by HBM: a byte
// read and an element written per value: 8 x 32768 tokens of 8 KV heads, bf16, 240 us, 6.7 TB/s (0.99 of the measured copy
// rate).
#include <atomic>
#include <string>

#include "tq_byte_attn.cuh"

namespace tqb {
namespace {

__device__ __forceinline__ int clamped(const int32_t* count, int b, int n) { return count ? min(max(__ldg(count + b), 0), n) : n; }

__global__ void __launch_bounds__(TQ_MAX_DRAFTS) draft_tree_kernel(const TreeArgs a) {
  constexpr int kRoot = -1, kDead = -2, kAtOnce = 8;  // words read before any is written
  extern __shared__ uint32_t bits[];                  // [word][draft], the rows one word apart
  __shared__ int up[TQ_MAX_DRAFTS];
  const int i = threadIdx.x, b = blockIdx.x, cnt = clamped(a.count, b, a.n), words = (a.n + 31) / 32, pitch = a.n | 1;
  const int start = a.start ? __ldg(a.start + b) : 0;
  int p = kRoot;
  if (i < a.n) {
    const int x = __ldg(a.parents + (long long)b * a.n + i);
    p = i < cnt && x >= kRoot && x < i ? x : kDead;
    up[i] = p;
    for (int w = 0; w < words; ++w) bits[w * pitch + i] = w == i >> 5 ? 1u << (i & 31) : 0u;
  }
  // a draft's row holds itself and its ancestors before p; p's row and what p points at double the way
  while (__syncthreads_or(p >= 0)) {
    const int q = p >= 0 ? up[p] : p;
    for (int w0 = 0; w0 < words; w0 += kAtOnce) {
      uint32_t x[kAtOnce];
#pragma unroll
      for (int w = 0; w < kAtOnce; ++w) x[w] = p >= 0 && w0 + w < words ? bits[(w0 + w) * pitch + p] : 0u;
      __syncthreads();
      if (p >= 0)
#pragma unroll
        for (int w = 0; w < kAtOnce; ++w)
          if (w0 + w < words) bits[(w0 + w) * pitch + i] |= x[w];
      __syncthreads();
    }
    p = q;
    if (i < a.n) up[i] = p;
  }
  if (i < a.n) {
    int above = -1;
    for (int w = 0; w < words; ++w) {
      if (p == kDead) bits[w * pitch + i] = 0;
      above += __popc(bits[w * pitch + i]);
    }
    a.positions[(long long)b * a.n + i] = (int32_t)((uint32_t)start + (uint32_t)max(above, 0));
  }
  __syncthreads();
  int32_t* out = a.masks + (long long)b * a.n * words;
  for (int k = i; k < a.n * words; k += blockDim.x) {
    const int d = k / words;
    out[k] = (int32_t)bits[(k - d * words) * pitch + d];
  }
}

// One code at a scale 2^-f times its own.
__device__ __forceinline__ unsigned char rescaled(unsigned char c, float f) { return (unsigned char)encode2(decode1(c) * f, 0.f); }
__device__ __forceinline__ uint32_t rescaled4(uint32_t w, float f) {
  float x[4];
#pragma unroll
  for (int m = 0; m < 4; ++m) x[m] = decode1((unsigned char)(w >> (8 * m))) * f;
  return encode4(x);
}

constexpr int kKeepWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kKeepWarps, D == 256 ? 2 : 4) byte_keep_kernel(const KeepArgs a) {
  const int lane = threadIdx.x & 31;
  const int unit = blockIdx.x * kKeepWarps + (threadIdx.x >> 5);
  const int side = unit & 1, h = (unit >> 1) % a.pool.heads, b = (unit >> 1) / a.pool.heads;
  if (b >= a.B) return;
  const int start = __ldg(a.start + b), cnt = clamped(a.count, b, a.n);
  const int32_t* path = a.path + (long long)b * a.n;
  bool bad = cnt > 0 && start < 0;
  for (int j = lane; j < cnt; j += 32) bad |= __ldg(path + j) <= (j ? __ldg(path + j - 1) : -1);
  bad = __any_sync(kFull, bad);
  if (lane == 0 && h == 0 && side == 0) {
    if (a.seq_len) a.seq_len[b] = (int32_t)((uint32_t)start + (bad ? 0u : (uint32_t)cnt));
    if (bad && a.pool.err) atomicExch(a.pool.err, TQ_DEVERR_BAD_PATH);
  }
  if (bad || cnt == 0) return;
  const long long first = start >> 4, last = ((long long)start + cnt - 1) >> 4;
  // Two blocks at a time: lane l looks up where slot l % 16 of block l / 16 takes its token from.  (One after the
  // other the lookups were a third of the time.)
  long long src2 = 0;
  const unsigned char *dst2 = nullptr, *from2 = nullptr;
  for (long long tile = first; tile <= last; ++tile) {
    const int half = (int)(tile - first) & 1;
    if (half == 0) {
      const long long t = tile + (lane >> 4), pos = t * 16 + (lane & 15), j = pos - start;
      src2 = t <= last && j >= 0 && j < cnt ? (long long)start + __ldg(path + j) : pos;
      if (t <= last) {
        dst2 = a.pool.base + pool_block(a.pool, page_of(a.pool, b, t), h) * block_bytes(D);
        from2 = src2 >> 4 == t ? dst2 : a.pool.base + pool_block(a.pool, page_of(a.pool, b, src2 >> 4), h) * block_bytes(D);
      }
    }
    // (of this block, on both halves of the warp)
    const int at = 16 * half + (lane & 15);
    const long long src = __shfl_sync(kFull, src2, at);
    const uint32_t moved = __ballot_sync(kFull, src != tile * 16 + (lane & 15)) & 0xffffu;
    if (moved == 0) continue;
    unsigned char* dst = reinterpret_cast<unsigned char*>(__shfl_sync(kFull, (unsigned long long)dst2, at));
    const unsigned char* from = reinterpret_cast<const unsigned char*>(__shfl_sync(kFull, (unsigned long long)from2, at));
    const float own_scale = *reinterpret_cast<const float*>(dst + 32 * D + 4 * side);
    const float from_scale = *reinterpret_cast<const float*>(from + 32 * D + 4 * side);
    // (looked at once the codes are on their way)
    int own, top;
    float f;
    bool round;
    auto scales = [&] {
      own = min(kEMax, max(kEMin, log2i(own_scale)));
      const int e = min(kEMax, max(kEMin, log2i(from_scale)));
      top = __reduce_max_sync(kFull, e);
      f = exp2i(e - top);
      round = __any_sync(kFull, e != top);
    };
    if (side == 0) {
      constexpr int C = D / 16, PER = D / 32;  // chunks of a row, of a lane
      uint4 v[PER];
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = lane + 32 * i, s = k / C, c = k % C;
        const unsigned char* blk = reinterpret_cast<const unsigned char*>(__shfl_sync(kFull, (unsigned long long)from, s));
        v[i] = *reinterpret_cast<const uint4*>(blk + k_chunk<D>((int)(__shfl_sync(kFull, src, s) & 15), c));
      }
      scales();
      __syncwarp();
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int k = lane + 32 * i, s = k / C, c = k % C;
        const float fs = __shfl_sync(kFull, f, s);
        if (round && fs != 1.f) {
          v[i].x = rescaled4(v[i].x, fs);
          v[i].y = rescaled4(v[i].y, fs);
          v[i].z = rescaled4(v[i].z, fs);
          v[i].w = rescaled4(v[i].w, fs);
        }
        if (fs != 1.f || (moved >> s & 1)) *reinterpret_cast<uint4*>(dst + k_chunk<D>(s, c)) = v[i];
      }
    } else {
#pragma unroll 1
      for (int x0 = lane; x0 < D; x0 += 128) {
        constexpr int E = D < 128 ? D / 32 : 4;  // coordinates at a time: x0, x0 + 32, ...
        uint4 v[E];
        unsigned char take[16][E];
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = *reinterpret_cast<const uint4*>(dst + 16 * D + 16 * (x0 + 32 * i));
#pragma unroll
        for (int s = 0; s < 16; ++s) {
          const unsigned char* blk = reinterpret_cast<const unsigned char*>(__shfl_sync(kFull, (unsigned long long)from, s));
          const int at = v_slot((int)(__shfl_sync(kFull, src, s) & 15));
#pragma unroll
          for (int i = 0; i < E; ++i) {
            take[s][i] = 0;
            if (moved >> s & 1) take[s][i] = blk[16 * D + 16 * (x0 + 32 * i) + at];
          }
        }
        scales();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < E; ++i) {
          uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
          for (int s = 0; s < 16; ++s) {
            const int k = v_slot(s) >> 2, sh = 8 * (v_slot(s) & 3);
            if (moved >> s & 1) w[k] = (w[k] & ~(0xffu << sh)) | ((uint32_t)take[s][i] << sh);
          }
          if (round) {
#pragma unroll
            for (int s = 0; s < 16; ++s) {
              const float fs = __shfl_sync(kFull, f, s);
              const int k = v_slot(s) >> 2, sh = 8 * (v_slot(s) & 3);
              if (fs != 1.f) w[k] = (w[k] & ~(0xffu << sh)) | ((uint32_t)rescaled((unsigned char)(w[k] >> sh), fs) << sh);
            }
          }
          *reinterpret_cast<uint4*>(dst + 16 * D + 16 * (x0 + 32 * i)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0 && top != own) *reinterpret_cast<float*>(dst + 32 * D + 4 * side) = exp2i(top);
  }
}

// N codes (2 or 4 to a 32-bit word's low end) times a power of two, as T.
template <int N>
__device__ __forceinline__ void decode_some(const uint32_t* w, float scale, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const uint32_t h = codes_half2(w[i >> 1] >> (16 * (i & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}
template <int N>
__device__ __forceinline__ void store_some(float* p, const float (&x)[N]) {
  if constexpr (N == 2) {
    *reinterpret_cast<float2*>(p) = make_float2(x[0], x[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __half*) { return tqd::pack_half2(a, b); }
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16*) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <int N, typename T>
__device__ __forceinline__ void store_some(T* p, const float (&x)[N]) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], p);
  if constexpr (N == 2) *reinterpret_cast<uint32_t*>(p) = w[0];
  else if constexpr (N == 4) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  else *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr int kReadWarps = 8;

template <int D, typename T>
__global__ void __launch_bounds__(32 * kReadWarps) byte_read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31, h = blockIdx.y, b = blockIdx.z;
  const int start = __ldg(a.start + b), cnt = clamped(a.count, b, a.n);
  const long long tile = (long long)(start >> 4) + blockIdx.x * kReadWarps + (threadIdx.x >> 5);
  const long long j0 = tile * 16 - start;  // the token at the block's slot 0
  if (j0 >= a.n) return;
  const long long row0 = ((long long)b * a.pool.heads + h) * a.n + j0;
  T* k = reinterpret_cast<T*>(a.k) + row0 * D;
  T* v = reinterpret_cast<T*>(a.v) + row0 * D;
  const int lo = (int)max(0ll, -j0), hi = (int)min(16ll, a.n - j0);   // slots written,
  const int live = (int)min((long long)hi, max(0ll, cnt - j0));       // and those of them below that are read
  constexpr int E = D / 32;                                           // V: coordinates E lane ..
  constexpr int KE = sizeof(T) == 4 ? 4 : 8, LPR = D / KE;           // K: codes of a lane, lanes of a row
  constexpr int KI = 16 * LPR / 32;                                   // K: pieces of a lane
  uint32_t kw[KI][KE / 4];
  uint4 vw[E];
  float2 scale = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < KI; ++i)
#pragma unroll
    for (int m = 0; m < KE / 4; ++m) kw[i][m] = 0;
#pragma unroll
  for (int i = 0; i < E; ++i) vw[i] = make_uint4(0u, 0u, 0u, 0u);
  if (live > lo) {
    const unsigned char* blk = a.pool.base + pool_block(a.pool, page_of(a.pool, b, tile), h) * block_bytes(D);
    scale = __ldg(reinterpret_cast<const float2*>(blk + 32 * D));
#pragma unroll
    for (int i = 0; i < KI; ++i) {
      const int at = lane + 32 * i, t = at / LPR, x = at % LPR * KE;
      const unsigned char* p = blk + k_chunk<D>(t, x >> 4) + (x & 15);
      if constexpr (KE == 8) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
        kw[i][0] = w.x, kw[i][1] = w.y;
      } else {
        kw[i][0] = __ldg(reinterpret_cast<const uint32_t*>(p));
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) vw[i] = __ldg(reinterpret_cast<const uint4*>(blk + 16 * D + 16 * (E * lane + i)));
  }
#pragma unroll
  for (int i = 0; i < KI; ++i) {
    const int at = lane + 32 * i, t = at / LPR, x = at % LPR * KE;
    float y[KE];
    decode_some<KE>(kw[i], scale.x, y);
    if (t >= live)
#pragma unroll
      for (int m = 0; m < KE; ++m) y[m] = 0.f;
    if (t >= lo && t < hi) store_some<KE>(k + (long long)t * D + x, y);
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    // byte v_slot(t) of each of the lane's coordinates
    uint32_t w[(E + 3) / 4] = {};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t q[4] = {vw[i].x, vw[i].y, vw[i].z, vw[i].w};
      w[i >> 2] |= (q[v_slot(t) >> 2] >> (8 * (v_slot(t) & 3)) & 0xffu) << (8 * (i & 3));
    }
    float y[E];
    decode_some<E>(w, scale.y, y);
    if (t >= live)
#pragma unroll
      for (int m = 0; m < E; ++m) y[m] = 0.f;
    if (t >= lo && t < hi) store_some<E>(v + (long long)t * D + E * lane, y);
  }
}

template <int D>
cudaError_t keep_go(const KeepArgs& a, cudaStream_t s) {
  const long long units = 2ll * a.B * a.pool.heads;
  byte_keep_kernel<D><<<(unsigned)((units + kKeepWarps - 1) / kKeepWarps), 32 * kKeepWarps, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D>
cudaError_t read_go(const ReadArgs& a, cudaStream_t s) {
  const int blocks = (int)(((long long)a.n + 15 + 15) / 16);  // that the tokens touch, at most
  const dim3 grid((blocks + kReadWarps - 1) / kReadWarps, a.pool.heads, a.B);
  if (a.dtype == TQ_F32) byte_read_kernel<D, float><<<grid, 32 * kReadWarps, 0, s>>>(a);
  else if (a.dtype == TQ_BF16) byte_read_kernel<D, __nv_bfloat16><<<grid, 32 * kReadWarps, 0, s>>>(a);
  else byte_read_kernel<D, __half><<<grid, 32 * kReadWarps, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

tq_status launch_draft_tree(const TreeArgs& a, Stream s) {
  static std::atomic<uint64_t> done{0};
  int dev;
  sm_count(&dev);
  constexpr int most = TQ_MAX_DRAFTS / 32 * (TQ_MAX_DRAFTS + 1) * 4;
  const cudaError_t e = allow_smem((const void*)draft_tree_kernel, most, dev, done);
  if (e != cudaSuccess) return cuda_error("draft tree", e);
  const int words = (a.n + 31) / 32;
  draft_tree_kernel<<<a.B, 32 * words, words * (a.n | 1) * 4, (cudaStream_t)s>>>(a);
  return cuda_error("draft tree", cudaGetLastError());
}

tq_status launch_byte_keep(const KeepArgs& a, Stream s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.d) {
    case 64: e = keep_go<64>(a, (cudaStream_t)s); break;
    case 128: e = keep_go<128>(a, (cudaStream_t)s); break;
    case 256: e = keep_go<256>(a, (cudaStream_t)s); break;
  }
  return cuda_error("byte keep", e);
}

tq_status launch_byte_read(const ReadArgs& a, Stream s) {
  cudaError_t e = cudaErrorInvalidValue;
  switch (a.d) {
    case 64: e = read_go<64>(a, (cudaStream_t)s); break;
    case 128: e = read_go<128>(a, (cudaStream_t)s); break;
    case 256: e = read_go<256>(a, (cudaStream_t)s); break;
  }
  return cuda_error("byte read", e);
}

}  // namespace tqb
