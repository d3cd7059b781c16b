// Internal declarations of the head norms / position rotation and of the byte cache: what the host
// checks hand to the launchers.
#pragma once

#include <cstddef>
#include <cstdint>

#include "tq_internal.h"

namespace tqb {

using tqi::Stream;

constexpr int kEMin = -30, kEMax = 30;  // scale exponents of a block
constexpr int kMaxAxes = 4;

#ifdef __CUDACC__
#define TQB_HD __host__ __device__
#else
#define TQB_HD
#endif
TQB_HD constexpr int block_bytes(int d) { return 32 * d + 32; }

// Rows of head_dim elements (strides in elements); heads = 0: absent.
struct Rows {
  const void* p;
  long long sb, st, sh;
  int heads;
};

struct Rotary {
  const uint64_t* table;  // [r / 2] or nullptr
  int r, interleaved, axes;
};

struct Positions {
  const int32_t* pos;    // [axes][B][n], or nullptr: start[b] + j
  const int32_t* start;  // [B] or nullptr: 0
};

// A paged pool of byte blocks.
struct Pool {
  unsigned char* base;
  const int32_t* table;
  int max_blocks, num_pages, heads;
  int32_t* err;
};

struct RotateArgs {
  int d, B, n;
  tq_dtype dtype, out_dtype;
  Rows q, k;
  const void *wq, *wk;
  void *q_out, *k_out;
  float eps;
  Rotary rot;
  Positions pos;
};

struct AppendArgs {
  int d, B, n, Hq;
  tq_dtype dtype;
  Pool pool;
  Rows k, v, q;
  const void *wk, *wq;
  void* q_out;
  const int32_t *start, *count;
  float eps;
  Rotary rot;
  Positions pos;
};

struct AttnArgs {
  int d, B, nq, Hq, Hkv;
  tq_dtype dtype;
  Pool pool;
  Rows q;
  const int32_t *seq_len, *count;
  float scale;
  void* out;
  void* ws;
};

tq_status cuda_error(const char* what, int e);
tq_status launch_norm_rotate(const RotateArgs& a, Stream s);
tq_status launch_byte_append(const AppendArgs& a, Stream s);
tq_status launch_byte_attention(const AttnArgs& a, Stream s);
tq_status launch_byte_dequantize(const Pool& pool, int d, int b, int h, int t0, int t1, float* k, float* v, Stream s);
// Bytes of attention workspace of a call (0 is never returned).
size_t byte_attention_workspace(int d, int B, int nq, int Hq, int Hkv, tq_dtype dtype);

}  // namespace tqb
