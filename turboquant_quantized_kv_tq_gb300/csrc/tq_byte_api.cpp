// C ABI entry points of the head norms / position rotation and of the byte cache: checks, then the
// launchers.
#include <cmath>
#include <string>

#include "tq_byte.h"

using namespace tqb;

namespace {

tq_status fail(tq_status s, const std::string& msg) {
  tqi::set_error(msg);
  return s;
}

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p % a) == 0; }

int dtype_bytes(tq_dtype t) { return t == TQ_F32 ? 4 : 2; }

tq_status check_dtype(tq_dtype t, const char* what) {
  if (t != TQ_F32 && t != TQ_BF16 && t != TQ_F16) return fail(TQ_ERR_INVALID_ARG, std::string("bad ") + what);
  return TQ_OK;
}

tq_status check_rows(const tq_heads* x, const char* what, int heads, int batch, int n, int bytes, Rows* out) {
  const std::string w(what);
  if (!x->data) return fail(TQ_ERR_INVALID_ARG, w + ": null data");
  if (x->heads < 1 || (heads > 0 && x->heads != heads)) return fail(TQ_ERR_INVALID_ARG, w + ": wrong number of heads");
  if (!aligned(x->data, 16)) return fail(TQ_ERR_INVALID_ARG, w + " must be 16-byte aligned");
  const int64_t lim = (int64_t)1 << 40;
  const int64_t s[3] = {x->batch_stride, x->token_stride, x->head_stride};
  const int len[3] = {batch, n, x->heads};
  int64_t use[3];
  for (int i = 0; i < 3; ++i) {
    use[i] = len[i] > 1 ? s[i] : 0;
    if (use[i] < 0 || use[i] > lim) return fail(TQ_ERR_INVALID_ARG, w + ": strides must be in [0, 2^40]");
    if ((use[i] * bytes) % 16) return fail(TQ_ERR_INVALID_ARG, w + ": strides must be multiples of 16 bytes");
  }
  *out = Rows{x->data, use[0], use[1], use[2], x->heads};
  return TQ_OK;
}

// Bytes [lo, hi) that rows cover.
struct Span {
  uintptr_t lo, hi;
};
Span span_of(const Rows& x, int batch, int n, int d, int bytes) {
  if (!x.heads || batch < 1 || n < 1) return {0, 0};
  const long long last = (batch - 1) * x.sb + (n - 1) * x.st + (x.heads - 1) * x.sh + d;
  return {(uintptr_t)x.p, (uintptr_t)x.p + (uintptr_t)last * bytes};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }
Span span_of(const void* p, size_t bytes) { return {(uintptr_t)p, (uintptr_t)p + bytes}; }
// Contiguous output rows.
Span span_of(const void* out, int batch, int n, int heads, int d, int bytes) {
  return span_of(out, (size_t)batch * n * heads * d * bytes);
}

// Whether an output of `heads` heads ([batch][n][heads][d], or [batch][heads][n][d] of keys) may be written
// while x is read: apart, or (same) exactly x's own rows, each of which is read before it is written.
bool may_write(const void* out, int heads, bool keys, const Rows& x, bool same, int batch, int n, int d, int bytes, int out_bytes) {
  if (!overlap(span_of(out, batch, n, heads, d, out_bytes), span_of(x, batch, n, d, bytes))) return true;
  const long long st = keys ? d : (long long)heads * d, sh = keys ? (long long)n * d : d, sb = (long long)n * heads * d;
  return same && out == x.p && out_bytes == bytes && (batch == 1 || x.sb == sb) && (n == 1 || x.st == st) &&
         (heads == 1 || x.sh == sh);
}

tq_status check_rotary(const tq_rotary* r, int head_dim, Rotary* out) {
  *out = Rotary{nullptr, 0, 0, 1};
  if (!r || !r->table) return TQ_OK;
  if (r->rotary_dim < 16 || r->rotary_dim % 16 || r->rotary_dim > head_dim)
    return fail(TQ_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [16, head_dim]");
  if (r->interleaved != 0 && r->interleaved != 1) return fail(TQ_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  if (r->num_axes < 1 || r->num_axes > kMaxAxes) return fail(TQ_ERR_INVALID_ARG, "num_axes must be in [1, 4]");
  if (!aligned(r->table, 8)) return fail(TQ_ERR_INVALID_ARG, "the rotary table must be 8-byte aligned");
  *out = Rotary{r->table, r->rotary_dim, r->interleaved, r->num_axes};
  return TQ_OK;
}

tq_status check_batch(int32_t batch, int32_t n, int heads, const char* what) {
  if (batch < 1 || batch > TQ_MAX_BATCH) return fail(TQ_ERR_INVALID_ARG, "batch must be in [1, TQ_MAX_BATCH]");
  if (n < 0) return fail(TQ_ERR_INVALID_ARG, std::string(what) + " must be >= 0");
  if ((int64_t)batch * n * heads > INT32_MAX / 2) return fail(TQ_ERR_INVALID_ARG, "too many rows in one call");
  return TQ_OK;
}

tq_status check_eps(float eps) {
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(TQ_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return TQ_OK;
}

tq_status check_config(const tq_byte_config* c) {
  if (!c) return fail(TQ_ERR_INVALID_ARG, "null config");
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim: the byte cache is built for 64, 128, 256");
  if (c->num_kv_heads < 1 || c->num_q_heads < 1 || c->num_q_heads % c->num_kv_heads)
    return fail(TQ_ERR_INVALID_ARG, "num_q_heads must be a positive multiple of num_kv_heads");
  if (c->num_q_heads > 4096) return fail(TQ_ERR_UNSUPPORTED, "num_q_heads: at most 4096");
  return TQ_OK;
}

tq_status check_pool(const tq_byte_config* c, const void* pool, const tq_page_table* pt, int32_t* err, Pool* out) {
  if (!pool) return fail(TQ_ERR_INVALID_ARG, "null pool");
  if (!pt || !pt->block_table) return fail(TQ_ERR_INVALID_ARG, "null page table");
  if (pt->max_blocks_per_seq < 1 || pt->num_pages < 1) return fail(TQ_ERR_INVALID_ARG, "empty page table");
  if ((int64_t)pt->max_blocks_per_seq * TQ_TILE_TOKENS > INT32_MAX / 2)
    return fail(TQ_ERR_INVALID_ARG, "max_blocks_per_seq too large");
  if (!aligned(pt->block_table, 4)) return fail(TQ_ERR_INVALID_ARG, "block_table must be 4-byte aligned");
  if (!aligned(pool, 256)) return fail(TQ_ERR_INVALID_ARG, "pool must be 256-byte aligned");
  if (!aligned(err, 4)) return fail(TQ_ERR_INVALID_ARG, "dev_error must be 4-byte aligned");
  *out = Pool{(unsigned char*)pool, pt->block_table, pt->max_blocks_per_seq, pt->num_pages, c->num_kv_heads, err};
  return TQ_OK;
}

// a / (2 pi) modulo 1 in 2^-64ths: the quotient in two doubles (the second from the exact remainder)
uint64_t turn_fraction(double a) {
  if (a < 0) return 0 - turn_fraction(-a);  // (the fraction below is exact for a >= 0 only)
  const double two_pi = 6.283185307179586, two_pi_lo = 2.4492935982947064e-16;
  const double hi = a / two_pi;
  const double lo = (std::fma(-hi, two_pi, a) - hi * two_pi_lo) / two_pi;
  const double fr = hi - std::floor(hi);  // exact
  const double two64 = 18446744073709551616.0, two32 = 4294967296.0;
  // fr = top / 2^32 + rest, both exact; then 2^64 (rest + lo) as a signed integer
  const double top = std::floor(fr * two32);
  const double rest = fr - top / two32 + lo;
  return ((uint64_t)top << 32) + (uint64_t)(int64_t)std::nearbyint(rest * two64);
}

}  // namespace

extern "C" {

tq_status tq_rotary_table(int32_t rotary_dim, const double* freqs, const int32_t* axes, int32_t num_axes,
                          uint64_t* out) {
  if (!freqs || !out) return fail(TQ_ERR_INVALID_ARG, "null argument");
  if (rotary_dim < 16 || rotary_dim % 16 || rotary_dim > 512)
    return fail(TQ_ERR_INVALID_ARG, "rotary_dim must be a multiple of 16 in [16, 512]");
  if (num_axes < 1 || num_axes > kMaxAxes) return fail(TQ_ERR_INVALID_ARG, "num_axes must be in [1, 4]");
  for (int i = 0; i < rotary_dim / 2; ++i) {
    if (!(std::fabs(freqs[i]) <= 1e6)) return fail(TQ_ERR_INVALID_ARG, "frequencies must be finite, at most 1e6 in magnitude");
    if (axes && (axes[i] < 0 || axes[i] >= num_axes)) return fail(TQ_ERR_INVALID_ARG, "axes must be in [0, num_axes)");
  }
  for (int i = 0; i < rotary_dim / 2; ++i)
    out[i] = ((turn_fraction(freqs[i]) + 2) & ~(uint64_t)3) | (uint64_t)(axes ? axes[i] : 0);
  return TQ_OK;
}

tq_status tq_norm_rotate(int32_t head_dim, tq_dtype dtype, tq_dtype out_dtype, int32_t batch, int32_t n,
                         const tq_heads* q, const void* q_weight, void* q_out, const tq_heads* k,
                         const void* k_weight, void* k_out, float eps, const tq_rotary* rotary,
                         const int32_t* dev_positions, const int32_t* dev_start, tq_stream stream) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256 && head_dim != 512)
    return fail(TQ_ERR_UNSUPPORTED, "head_dim: norm_rotate is built for 64, 128, 256, 512");
  tq_status s = check_dtype(dtype, "dtype");
  if (s != TQ_OK) return s;
  if (out_dtype != dtype && out_dtype != TQ_F32) return fail(TQ_ERR_INVALID_ARG, "out_dtype must be dtype or TQ_F32");
  if (!q && !k) return fail(TQ_ERR_INVALID_ARG, "neither q nor k given");
  RotateArgs a = {};
  s = check_batch(batch, n, 1, "n");
  if (s != TQ_OK) return s;
  if (q && (s = check_rows(q, "q", 0, batch, n, dtype_bytes(dtype), &a.q)) != TQ_OK) return s;
  if (k && (s = check_rows(k, "k", 0, batch, n, dtype_bytes(dtype), &a.k)) != TQ_OK) return s;
  if (a.q.heads > 4096 || a.k.heads > 4096) return fail(TQ_ERR_UNSUPPORTED, "heads: at most 4096");
  s = check_batch(batch, n, a.q.heads + a.k.heads, "n");
  if (s != TQ_OK) return s;
  if ((q && !q_out) || (k && !k_out)) return fail(TQ_ERR_INVALID_ARG, "null output");
  if (!aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return fail(TQ_ERR_INVALID_ARG, "outputs and weights must be 16-byte aligned");
  if (!aligned(dev_positions, 4) || !aligned(dev_start, 4)) return fail(TQ_ERR_INVALID_ARG, "misaligned pointer");
  if ((s = check_eps(eps)) != TQ_OK) return s;
  if ((s = check_rotary(rotary, head_dim, &a.rot)) != TQ_OK) return s;
  const int in = dtype_bytes(dtype), ob = dtype_bytes(out_dtype);
  if ((q && (!may_write(q_out, a.q.heads, false, a.q, true, batch, n, head_dim, in, ob) ||
             !may_write(q_out, a.q.heads, false, a.k, false, batch, n, head_dim, in, ob))) ||
      (k && (!may_write(k_out, a.k.heads, true, a.k, true, batch, n, head_dim, in, ob) ||
             !may_write(k_out, a.k.heads, true, a.q, false, batch, n, head_dim, in, ob))))
    return fail(TQ_ERR_INVALID_ARG, "an output overlaps an input and is not its own buffer in the same layout");
  if (n == 0) return TQ_OK;
  if (q && k && overlap(span_of(q_out, batch, n, a.q.heads, head_dim, ob), span_of(k_out, batch, n, a.k.heads, head_dim, ob)))
    return fail(TQ_ERR_INVALID_ARG, "the outputs overlap");
  a.d = head_dim;
  a.B = batch;
  a.n = n;
  a.dtype = dtype;
  a.out_dtype = out_dtype;
  a.wq = q_weight;
  a.wk = k_weight;
  a.q_out = q_out;
  a.k_out = k_out;
  a.eps = eps;
  a.pos = Positions{dev_positions, dev_start};
  return launch_norm_rotate(a, stream);
}

size_t tq_byte_pool_bytes(const tq_byte_config* cfg, int32_t num_pages) {
  if (check_config(cfg) != TQ_OK || num_pages < 1) return 0;
  return ((size_t)num_pages + 1) * cfg->num_kv_heads * block_bytes(cfg->head_dim);
}

tq_status tq_byte_append_paged(const tq_byte_config* cfg, void* dev_pool, const tq_page_table* pages,
                               int32_t batch, int32_t n, tq_dtype dtype, const tq_heads* k, const tq_heads* v,
                               const int32_t* dev_start, const int32_t* dev_count, const void* k_weight,
                               float eps, const tq_rotary* rotary, const int32_t* dev_positions,
                               const tq_heads* q, const void* q_weight, void* q_out, int32_t* dev_error,
                               tq_stream stream) {
  tq_status s = check_config(cfg);
  if (s != TQ_OK) return s;
  AppendArgs a = {};
  if ((s = check_pool(cfg, dev_pool, pages, dev_error, &a.pool)) != TQ_OK) return s;
  if ((s = check_dtype(dtype, "dtype")) != TQ_OK) return s;
  if ((s = check_batch(batch, n, cfg->num_q_heads, "n")) != TQ_OK) return s;
  if (!k || !v || !dev_start) return fail(TQ_ERR_INVALID_ARG, "null argument");
  const int bytes = dtype_bytes(dtype);
  if ((s = check_rows(k, "k", cfg->num_kv_heads, batch, n, bytes, &a.k)) != TQ_OK) return s;
  if ((s = check_rows(v, "v", cfg->num_kv_heads, batch, n, bytes, &a.v)) != TQ_OK) return s;
  if (q) {
    if ((s = check_rows(q, "q", cfg->num_q_heads, batch, n, bytes, &a.q)) != TQ_OK) return s;
    if (!q_out) return fail(TQ_ERR_INVALID_ARG, "null q_out");
  }
  if (!aligned(q_out, 16) || !aligned(k_weight, 16) || !aligned(q_weight, 16))
    return fail(TQ_ERR_INVALID_ARG, "q_out and weights must be 16-byte aligned");
  if (!aligned(dev_start, 4) || !aligned(dev_count, 4) || !aligned(dev_positions, 4))
    return fail(TQ_ERR_INVALID_ARG, "misaligned pointer");
  if ((s = check_eps(eps)) != TQ_OK) return s;
  if ((s = check_rotary(rotary, cfg->head_dim, &a.rot)) != TQ_OK) return s;
  if (q && (!may_write(q_out, cfg->num_q_heads, false, a.q, true, batch, n, cfg->head_dim, bytes, bytes) ||
            !may_write(q_out, cfg->num_q_heads, false, a.k, false, batch, n, cfg->head_dim, bytes, bytes) ||
            !may_write(q_out, cfg->num_q_heads, false, a.v, false, batch, n, cfg->head_dim, bytes, bytes)))
    return fail(TQ_ERR_INVALID_ARG, "q_out overlaps an input and is not q's own buffer in the same layout");
  if (n == 0) return TQ_OK;
  const Span pool = span_of(dev_pool, tq_byte_pool_bytes(cfg, pages->num_pages));
  const int d = cfg->head_dim;
  if (overlap(pool, span_of(a.k, batch, n, d, bytes)) || overlap(pool, span_of(a.v, batch, n, d, bytes)) ||
      (q && (overlap(pool, span_of(a.q, batch, n, d, bytes)) || overlap(pool, span_of(q_out, batch, n, cfg->num_q_heads, d, bytes)))))
    return fail(TQ_ERR_INVALID_ARG, "k, v, q and q_out must not overlap the pool");
  a.d = cfg->head_dim;
  a.B = batch;
  a.n = n;
  a.Hq = cfg->num_q_heads;
  a.dtype = dtype;
  a.wk = k_weight;
  a.wq = q_weight;
  a.q_out = q_out;
  a.start = dev_start;
  a.count = dev_count;
  a.eps = eps;
  a.pos = Positions{dev_positions, dev_start};
  return launch_byte_append(a, stream);
}

static tq_status check_attention(const tq_byte_config* cfg, int32_t batch, int32_t nq, tq_dtype dtype) {
  tq_status s = check_config(cfg);
  if (s != TQ_OK) return s;
  if ((s = check_dtype(dtype, "dtype")) != TQ_OK) return s;
  if (nq < 1) return fail(TQ_ERR_INVALID_ARG, "nq must be >= 1");
  if ((s = check_batch(batch, nq, cfg->num_q_heads, "nq")) != TQ_OK) return s;
  if ((int64_t)batch * cfg->num_kv_heads > 65535 * 8ll) return fail(TQ_ERR_UNSUPPORTED, "too many (entry, KV head) pairs");
  return TQ_OK;
}

size_t tq_byte_attention_workspace_bytes(const tq_byte_config* cfg, const tq_page_table* pages, int32_t batch,
                                         int32_t nq, tq_dtype dtype) {
  (void)pages;
  if (check_attention(cfg, batch, nq, dtype) != TQ_OK) return 0;
  return byte_attention_workspace(cfg->head_dim, batch, nq, cfg->num_q_heads, cfg->num_kv_heads, dtype);
}

tq_status tq_byte_attention_paged(const tq_byte_config* cfg, const void* dev_pool, const tq_page_table* pages,
                                  int32_t batch, int32_t nq, tq_dtype dtype, const tq_heads* q,
                                  const int32_t* dev_seq_len, const int32_t* dev_count, float scale, void* out,
                                  void* ws, size_t ws_bytes, int32_t* dev_error, tq_stream stream) {
  tq_status s = check_attention(cfg, batch, nq, dtype);
  if (s != TQ_OK) return s;
  AttnArgs a = {};
  if ((s = check_pool(cfg, dev_pool, pages, dev_error, &a.pool)) != TQ_OK) return s;
  if (!q || !dev_seq_len || !out || !ws) return fail(TQ_ERR_INVALID_ARG, "null argument");
  if ((s = check_rows(q, "q", cfg->num_q_heads, batch, nq, dtype_bytes(dtype), &a.q)) != TQ_OK) return s;
  if (!aligned(out, 16) || !aligned(ws, 256) || !aligned(dev_seq_len, 4) || !aligned(dev_count, 4))
    return fail(TQ_ERR_INVALID_ARG, "misaligned pointer (ws 256 B, out 16 B, lengths 4 B)");
  const int bytes = dtype_bytes(dtype);
  if (!may_write(out, cfg->num_q_heads, false, a.q, false, batch, nq, cfg->head_dim, bytes, bytes))
    return fail(TQ_ERR_INVALID_ARG, "out must not overlap q");
  if (!std::isfinite(scale)) return fail(TQ_ERR_INVALID_ARG, "scale must be finite");
  const size_t need = byte_attention_workspace(cfg->head_dim, batch, nq, cfg->num_q_heads, cfg->num_kv_heads, dtype);
  if (ws_bytes < need) return fail(TQ_ERR_WORKSPACE, "workspace too small");
  const Span pool = span_of(dev_pool, tq_byte_pool_bytes(cfg, pages->num_pages)), w = span_of(ws, need);
  const Span o = span_of(out, batch, nq, cfg->num_q_heads, cfg->head_dim, bytes), x = span_of(a.q, batch, nq, cfg->head_dim, bytes);
  if (overlap(pool, o) || overlap(pool, w) || overlap(pool, x)) return fail(TQ_ERR_INVALID_ARG, "q, out and ws must not overlap the pool");
  if (overlap(w, o) || overlap(w, x)) return fail(TQ_ERR_INVALID_ARG, "ws must not overlap q or out");
  a.d = cfg->head_dim;
  a.B = batch;
  a.nq = nq;
  a.Hq = cfg->num_q_heads;
  a.Hkv = cfg->num_kv_heads;
  a.dtype = dtype;
  a.seq_len = dev_seq_len;
  a.count = dev_count;
  a.scale = scale;
  a.out = out;
  a.ws = ws;
  return launch_byte_attention(a, stream);
}

tq_status tq_byte_dequantize(const tq_byte_config* cfg, const void* dev_pool, const tq_page_table* pages,
                             int32_t batch, int32_t b, int32_t kvh, int32_t t0, int32_t t1, float* k_out,
                             float* v_out, tq_stream stream) {
  tq_status s = check_config(cfg);
  if (s != TQ_OK) return s;
  Pool pool;
  if ((s = check_pool(cfg, dev_pool, pages, nullptr, &pool)) != TQ_OK) return s;
  if (batch < 1 || batch > TQ_MAX_BATCH) return fail(TQ_ERR_INVALID_ARG, "batch must be in [1, TQ_MAX_BATCH]");
  if (b < 0 || b >= batch || kvh < 0 || kvh >= cfg->num_kv_heads) return fail(TQ_ERR_INVALID_ARG, "bad slab");
  if (t0 < 0 || t1 < t0) return fail(TQ_ERR_INVALID_ARG, "bad token range");
  if (t1 > TQ_TILE_TOKENS * pages->max_blocks_per_seq) return fail(TQ_ERR_CAPACITY, "token range beyond the page table");
  if (t0 == t1) return TQ_OK;
  if (!k_out || !v_out || !aligned(k_out, 4) || !aligned(v_out, 4)) return fail(TQ_ERR_INVALID_ARG, "bad output pointer");
  return launch_byte_dequantize(pool, cfg->head_dim, b, kvh, t0, t1, k_out, v_out, stream);
}

}  // extern "C"
