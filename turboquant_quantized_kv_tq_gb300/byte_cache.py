"""Head norms with the position rotation, and the 8-bit paged cache (``tq_norm_rotate`` and the
``tq_byte_*`` entry points of ``include/tq.h``).

``Rotary`` holds a rotation's device table, ``norm_rotate`` applies it (and the norms) to queries and
keys, and ``PagedByteCache`` owns a pool of e4m3 codes with a scale for each 16-token block, KV head
and side.  Tensors may be strided views (a fused projection's slices): only the head dimension has to
be contiguous, with rows on 16-byte boundaries.  Nothing is copied or converted here; a layout that
the kernels do not take is refused.
"""

import numpy as np
import torch

from . import binding as _b
from .binding import check

_CODES = {torch.float32: _b.TQ_F32, torch.bfloat16: _b.TQ_BF16, torch.float16: _b.TQ_F16}

# (the current stream's handle without building a Stream object: a tenth of the cost)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_heads_c, _pages_c, _empty = _b.tq_heads, _b.tq_page_table, torch.empty


def _code(t):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}: float32, bfloat16 or float16") from None


def _heads(t, name, shape, dtype, index, b, n, h):
    """tq_heads of a 4-d view whose dims b, n, h are batch, token and head."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {list(shape)} on cuda:{index}, not {t.dtype} "
                         f"{list(t.shape)} on {t.device}")
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    return _heads_c(t.data_ptr() or None, s[b], s[n], s[h], shape[h])


def _ints(t, name, shape, index):
    if t.dtype is not torch.int32 or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on cuda:{index}")
    return t.data_ptr()


def _dense(t, name, shape, dtype, index):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{index}")
    return t


def _launch(index, device, stream, inputs, go):
    """go(handle) with the device current and ``stream`` (default: the device's current one) the current
    stream, so that outputs and workspaces allocated in it belong to the stream that uses them."""
    if stream is None and torch._C._cuda_getDevice() == index:
        return go(_raw_stream(index))
    with torch.cuda.device(device):
        if stream is None:
            return go(_raw_stream(index))
        with torch.cuda.stream(stream):
            got = go(stream.cuda_stream)
    for t in inputs:  # (their memory is not handed out again before the stream is done with it)
        if t is not None:
            t.record_stream(stream)
    return got


def _device(device):
    d = torch.device(device)
    if d.type == "cuda" and d.index is None:
        d = torch.device("cuda", torch.cuda.current_device())
    return d


class Rotary:
    """A position rotation of the first ``rotary_dim`` coordinates of a head.

    Pair i turns by ``freqs[i]`` radians per position (default ``base ** (-2 i / rotary_dim)``);
    ``interleaved`` pairs coordinates 2i and 2i + 1, otherwise i and i + rotary_dim / 2.
    ``sections``: the numbers of consecutive pairs that follow each axis of the positions (their sum
    is rotary_dim / 2); ``axes`` gives each pair's axis instead.  Default: one axis.
    """

    def __init__(self, rotary_dim, base=10000.0, freqs=None, sections=None, axes=None, interleaved=False,
                 device="cuda"):
        half = int(rotary_dim) // 2
        if sections is not None:
            if axes is not None:
                raise ValueError("give sections or axes, not both")
            if sum(sections) != half or any(int(s) < 0 for s in sections):
                raise ValueError("sections must be non-negative and sum to rotary_dim / 2")
            axes = [a for a, s in enumerate(sections) for _ in range(int(s))]
            self.num_axes = len(sections)
        else:
            self.num_axes = max(axes) + 1 if axes is not None and len(axes) else 1
        if axes is not None and len(axes) != half:
            raise ValueError("axes must have rotary_dim / 2 entries")
        if freqs is None:
            freqs = [float(base) ** (-2.0 * i / rotary_dim) for i in range(half)]
        freqs = np.ascontiguousarray(freqs, dtype=np.float64)
        if freqs.shape != (half,):
            raise ValueError("freqs must have rotary_dim / 2 entries")
        ax = np.ascontiguousarray(axes, dtype=np.int32) if axes is not None else None
        host = np.zeros(half, dtype=np.uint64)
        check(_b.tq_rotary_table(int(rotary_dim), freqs.ctypes.data, ax.ctypes.data if ax is not None else None,
                                 self.num_axes, host.ctypes.data))
        self.rotary_dim, self.interleaved = int(rotary_dim), bool(interleaved)
        self.host_table = host
        self.table = torch.from_numpy(host.view(np.int64)).to(_device(device))
        self.index = self.table.get_device()
        self._c = _b.tq_rotary(self.table.data_ptr(), self.rotary_dim, int(self.interleaved), self.num_axes)


def _rotary(rotary, index):
    if rotary is None:
        return None, 1
    if rotary.index != index:
        raise ValueError(f"the rotary table must be on cuda:{index}")
    return rotary._c, rotary.num_axes


def norm_rotate(q=None, k=None, rotary=None, positions=None, start=None, q_weight=None, k_weight=None, eps=1e-6,
                out_dtype=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head (where a weight is given) and position rotation (where ``rotary`` is), in
    one pass.

    q: CUDA tensor [batch][n][q_heads][d]; k: [batch][k_heads][n][d] (either may be None); any strides
    along the first three dims.  ``positions``: int32 CUDA [num_axes][batch][n]; None: token j of entry b
    is at ``start[b] + j`` (``start``: int32 CUDA [batch]; None: 0).  ``out_dtype``: q's dtype (default) or float32, which the packed caches'
    queries need.  Returns (q_out, k_out), contiguous in the shapes of q and k.
    """
    x = q if q is not None else k
    if x is None:
        raise ValueError("neither q nor k given")
    if x.dim() != 4 or not x.is_cuda:
        raise ValueError("q and k must be CUDA tensors of 4 dims")
    code, index, dt, device = _code(x), x.get_device(), x.dtype, x.device
    shape = x.shape
    batch, d = shape[0], shape[3]
    n = shape[1 if q is not None else 2]
    odt = dt if out_dtype is None else out_dtype
    if odt is not dt and odt is not torch.float32:
        raise ValueError("out_dtype must be the inputs' dtype or float32")
    rc, axes = _rotary(rotary, index)
    qs = ks = None
    q_shape = k_shape = None
    if q is not None:
        q_shape = (batch, n, shape[2], d)
        qs = _heads(q, "q", q_shape, dt, index, 0, 1, 2)
    if k is not None:
        k_shape = (batch, k.shape[1] if k.dim() == 4 else 0, n, d)
        ks = _heads(k, "k", k_shape, dt, index, 0, 2, 1)
    pos = None if positions is None else _ints(positions, "positions", (axes, batch, n), index)
    st = None if start is None else _ints(start, "start", (batch,), index)
    wq = None if q_weight is None else _dense(q_weight, "q_weight", (d,), dt, index).data_ptr()
    wk = None if k_weight is None else _dense(k_weight, "k_weight", (d,), dt, index).data_ptr()

    def go(handle):
        qo = ko = qp = kp = None
        if qs is not None:
            qo = _empty(q_shape, dtype=odt, device=device) if q_out is None else _dense(q_out, "q_out", q_shape, odt, index)
            qp = qo.data_ptr()
        if ks is not None:
            ko = _empty(k_shape, dtype=odt, device=device) if k_out is None else _dense(k_out, "k_out", k_shape, odt, index)
            kp = ko.data_ptr()
        if batch and n:
            status = _b.tq_norm_rotate(d, code, _CODES[odt], batch, n, qs, wq, qp, ks, wk, kp, eps, rc, pos, st, handle)
            if status:
                check(status)
        return qo, ko

    return _launch(index, device, stream, (q, k, positions, start, q_weight, k_weight, q_out, k_out), go)


class PagedByteCache:
    """A pool of ``num_pages`` pages on a CUDA device, each holding one 16-token block per KV head: e4m3
    codes of keys and values with a power-of-two scale per side (``tq_byte_config``).  ``block_table``
    is an int32 CUDA tensor [batch][max_blocks_per_seq] of page indices owned by the caller, as for
    PagedKVCache; positions, lengths and counts are int32 CUDA tensors [batch].  All are read on the
    device, so they may change between replays of a captured CUDA graph.  The batch is that of each
    call's block table.  Head dim 64, 128 or 256; any num_q_heads / num_kv_heads.

    ``error`` (int32 CUDA, one element) receives a TQ_DEVERR_* code of any call: see ``device_error``.
    """

    def __init__(self, head_dim, num_q_heads, num_kv_heads, num_pages, max_blocks_per_seq, device="cuda"):
        self.cfg = _b.tq_byte_config(int(head_dim), int(num_q_heads), int(num_kv_heads))
        need = int(_b.tq_byte_pool_bytes(self.cfg, int(num_pages)))
        if need == 0:
            raise _b.TQError(_b.TQ_ERR_INVALID_ARG, _b.lib.tq_last_error().decode() or "num_pages must be >= 1")
        self.head_dim, self.num_q_heads, self.num_kv_heads = int(head_dim), int(num_q_heads), int(num_kv_heads)
        self.num_pages, self.max_blocks_per_seq = int(num_pages), int(max_blocks_per_seq)
        if self.max_blocks_per_seq < 1:
            raise ValueError("max_blocks_per_seq must be >= 1")
        self.block_bytes = 32 * self.head_dim + 32
        self.device = _device(device)
        self.pool = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self.error = torch.zeros(1, dtype=torch.int32, device=self.device)
        self._index = self.pool.get_device()
        self._pool, self._error = self.pool.data_ptr(), self.error.data_ptr()
        self._need = {}  # workspace bytes by (batch, nq, dtype)

    def _pages(self, table):
        if (table.dtype is not torch.int32 or table.dim() != 2 or table.shape[1] != self.max_blocks_per_seq
                or table.get_device() != self._index or not table.is_contiguous()):
            raise ValueError(f"block_table must be a contiguous int32 tensor [batch][{self.max_blocks_per_seq}] "
                             f"on {self.device}")
        return _pages_c(table.data_ptr(), self.max_blocks_per_seq, self.num_pages)

    def device_error(self):
        """The recorded TQ_DEVERR_* code (0: none), cleared by the call.  Waits for the device."""
        code = int(self.error.item())
        if code:
            self.error.zero_()
        return code

    def append(self, k, v, start, block_table, count=None, rotary=None, positions=None, k_weight=None, q=None,
               q_weight=None, eps=1e-6, q_out=None, stream=None):
        """Append k, v ([batch][num_kv_heads][n][d], any strides along the first three dims) at positions
        ``start[b] + j``, keys normed (``k_weight``) and rotated (``rotary``) on the way.

        ``positions`` ([num_axes][batch][n]) are the rotation's positions; None: ``start[b] + j``.
        ``count[b]``: entry b appends only its first count[b] tokens.  ``q`` ([batch][n][num_q_heads][d]) is
        normed and rotated alike in the same launch: returns q_out (None without q)."""
        d, dev, index = self.head_dim, self.device, self._index
        pt = self._pages(block_table)
        batch, n = block_table.shape[0], k.shape[2] if k.dim() == 4 else 0
        code, dt = _code(k), k.dtype
        shape = (batch, self.num_kv_heads, n, d)
        ks, vs = _heads(k, "k", shape, dt, index, 0, 2, 1), _heads(v, "v", shape, dt, index, 0, 2, 1)
        rc, axes = _rotary(rotary, index)
        if start is None:
            raise ValueError("start must be given")
        st = _ints(start, "start", (batch,), index)
        cn = None if count is None else _ints(count, "count", (batch,), index)
        pos = None if positions is None else _ints(positions, "positions", (axes, batch, n), index)
        wq = None if q_weight is None else _dense(q_weight, "q_weight", (d,), dt, index).data_ptr()
        wk = None if k_weight is None else _dense(k_weight, "k_weight", (d,), dt, index).data_ptr()
        qs = None
        if q is not None:
            q_shape = (batch, n, self.num_q_heads, d)
            qs = _heads(q, "q", q_shape, dt, index, 0, 1, 2)

        def go(handle):
            qo = qp = None
            if qs is not None:
                qo = _empty(q_shape, dtype=dt, device=dev) if q_out is None else _dense(q_out, "q_out", q_shape, dt, index)
                qp = qo.data_ptr()
            if batch and n:
                status = _b.tq_byte_append_paged(self.cfg, self._pool, pt, batch, n, code, ks, vs, st, cn, wk, eps, rc, pos,
                                                 qs, wq, qp, self._error, handle)
                if status:
                    check(status)
            return qo

        return _launch(index, dev, stream, (k, v, start, block_table, count, positions, k_weight, q, q_weight, q_out), go)

    def attention(self, q, seq_len, block_table, count=None, scale=None, out=None, stream=None):
        """q: CUDA tensor [batch][nq][num_q_heads][d] (or [batch][num_q_heads][d] for one query), any
        strides along the first dims.  The last ``count[b]`` (default nq) positions of sequence b are its
        queries: query i attends to the first ``seq_len[b] - count[b] + 1 + i`` tokens, and rows
        i >= count[b] come out as zeros.  ``scale`` multiplies the scores (default 1 / sqrt(d)).  Returns
        out, contiguous in q's shape and dtype."""
        dev, index = self.device, self._index
        pt = self._pages(block_table)
        q4 = q.unsqueeze(1) if q.dim() == 3 else q
        batch, nq = block_table.shape[0], q4.shape[1] if q4.dim() == 4 else 0
        code, dt = _code(q), q.dtype
        qs = _heads(q4, "q", (batch, nq, self.num_q_heads, self.head_dim), dt, index, 0, 1, 2)
        if seq_len is None:
            raise ValueError("seq_len must be given")
        sl = _ints(seq_len, "seq_len", (batch,), index)
        cn = None if count is None else _ints(count, "count", (batch,), index)
        if scale is None:
            scale = self.head_dim ** -0.5

        def go(handle):
            o = _empty(q.shape, dtype=dt, device=dev) if out is None else _dense(out, "out", q.shape, dt, index)
            if batch and nq:
                need = self._need.get((batch, nq, code))
                if need is None:
                    need = _b.tq_byte_attention_workspace_bytes(self.cfg, pt, batch, nq, code)
                    self._need[(batch, nq, code)] = need
                ws = _empty(need, dtype=torch.uint8, device=dev)
                status = _b.tq_byte_attention_paged(self.cfg, self._pool, pt, batch, nq, code, qs, sl, cn, scale,
                                                    o.data_ptr(), ws.data_ptr(), need, self._error, handle)
                if status:
                    check(status)
            return o

        return _launch(index, dev, stream, (q, seq_len, block_table, count, out), go)

    def dequantize(self, b, kvh, t0, t1, block_table, stream=None):
        """Tokens [t0, t1) of KV head kvh of entry b as fp32 (k, v) [t1 - t0][d]."""
        pt = self._pages(block_table)

        def go(handle):
            k = _empty((max(t1 - t0, 0), self.head_dim), dtype=torch.float32, device=self.device)
            v = torch.empty_like(k)
            check(_b.tq_byte_dequantize(self.cfg, self._pool, pt, block_table.shape[0], b, kvh, t0, t1,
                                        k.data_ptr() or None, v.data_ptr() or None, handle))
            return k, v

        return _launch(self._index, self.device, stream, (block_table,), go)
