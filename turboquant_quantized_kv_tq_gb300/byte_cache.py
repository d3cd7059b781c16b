"""Head norms with the position rotation, and the 8-bit paged cache (``tq_norm_rotate`` and the
``tq_byte_*`` entry points of ``include/tq.h``).

``Rotary`` holds a rotation's device table, ``norm_rotate`` applies it (and the norms) to queries and
keys, and ``PagedByteCache`` owns a pool of e4m3 codes with a scale for each 16-token block, KV head
and side.  Tensors may be strided views (a fused projection's slices): only the head dimension has to
be contiguous, with rows on 16-byte boundaries.  Nothing is copied or converted here; a layout that
the kernels do not take is refused.
"""

import contextlib

import numpy as np
import torch

from . import binding as _b
from .binding import check

_CODES = {torch.float32: _b.TQ_F32, torch.bfloat16: _b.TQ_BF16, torch.float16: _b.TQ_F16}


def _code(t):
    try:
        return _CODES[t.dtype]
    except KeyError:
        raise ValueError(f"unsupported dtype {t.dtype}: float32, bfloat16 or float16") from None


def _heads(t, name, order, shape, dtype, device):
    """tq_heads of a 4-d view; ``order``: its dims of (batch, token, head)."""
    if t.dim() != 4 or tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, not {list(t.shape)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.stride(3) != 1:
        raise ValueError(f"{name}: the head dimension must be contiguous")
    if t.numel() and t.data_ptr() % 16:
        raise ValueError(f"{name} must be 16-byte aligned")
    b, n, h = order
    return _b.tq_heads(t.data_ptr() or None, t.stride(b), t.stride(n), t.stride(h), t.shape[h])


def _ints(t, name, shape, device):
    if t is None:
        return None
    if t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on {device}")
    return t.data_ptr()


def _weight(w, name, d, dtype, device):
    if w is None:
        return None
    if tuple(w.shape) != (d,) or w.dtype != dtype or w.device != device or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape [{d}] on {device}")
    return w.data_ptr()


def _out(t, name, shape, dtype, device):
    if tuple(t.shape) != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on {device}")
    return t


@contextlib.contextmanager
def _on_other(device, stream, inputs):
    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
            return
        with torch.cuda.stream(stream):
            yield stream.cuda_stream
    for t in inputs:  # (their memory is not handed out again before the stream is done with it)
        if t is not None:
            t.record_stream(stream)


class _Here:
    """The current stream of the current device: nothing to switch."""

    def __init__(self, handle):
        self.handle = handle

    def __enter__(self):
        return self.handle

    def __exit__(self, *exc):
        return False


def _launch_on(device, stream, *inputs):
    """Context for a launch on ``stream`` (default: the device's current one): outputs and workspaces
    are allocated in it, so their memory belongs to the stream that uses them."""
    if stream is None and torch.cuda.current_device() == device.index:
        return _Here(torch.cuda.current_stream().cuda_stream)
    return _on_other(device, stream, inputs)


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
        self._c = _b.tq_rotary(self.table.data_ptr(), self.rotary_dim, int(self.interleaved), self.num_axes)


def _rotary(rotary, device):
    if rotary is None:
        return None, 1
    if rotary.table.device != device:
        raise ValueError(f"the rotary table must be on {device}")
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
    if x.dim() != 4:
        raise ValueError("q and k must have 4 dims")
    if not x.is_cuda:
        raise ValueError("q and k must be CUDA tensors")
    code, device, d = _code(x), x.device, x.shape[3]
    batch, n = x.shape[0], x.shape[1 if q is not None else 2]
    dt = x.dtype
    odt = dt if out_dtype is None else out_dtype
    if odt != dt and odt != torch.float32:
        raise ValueError("out_dtype must be the inputs' dtype or float32")
    rc, axes = _rotary(rotary, device)
    qs = ks = None
    if q is not None:
        qs = _heads(q, "q", (0, 1, 2), (batch, n, q.shape[2], d), dt, device)
    if k is not None:
        ks = _heads(k, "k", (0, 2, 1), (batch, k.shape[1] if k.dim() == 4 else 0, n, d), dt, device)
    pos = _ints(positions, "positions", (axes, batch, n), device)
    st = _ints(start, "start", (batch,), device)
    wq, wk = _weight(q_weight, "q_weight", d, dt, device), _weight(k_weight, "k_weight", d, dt, device)
    with _launch_on(device, stream, q, k, positions, start, q_weight, k_weight) as handle:
        if q is not None:
            q_out = torch.empty(q.shape, dtype=odt, device=device) if q_out is None else _out(q_out, "q_out", tuple(q.shape), odt, device)
        if k is not None:
            k_out = torch.empty(k.shape, dtype=odt, device=device) if k_out is None else _out(k_out, "k_out", tuple(k.shape), odt, device)
        if batch and n:
            check(_b.tq_norm_rotate(d, code, _CODES[odt], batch, n, qs, wq, q_out.data_ptr() if q is not None else None,
                                    ks, wk, k_out.data_ptr() if k is not None else None, eps, rc, pos, st, handle))
    return (q_out if q is not None else None), (k_out if k is not None else None)


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

    def _pages(self, block_table):
        if (block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous()
                or block_table.shape[1] != self.max_blocks_per_seq or block_table.device != self.device):
            raise ValueError(f"block_table must be a contiguous int32 tensor [batch][{self.max_blocks_per_seq}] "
                             f"on {self.device}")
        return _b.tq_page_table(block_table.data_ptr(), self.max_blocks_per_seq, self.num_pages)

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
        d, dev = self.head_dim, self.device
        pt = self._pages(block_table)
        batch, n = block_table.shape[0], k.shape[2] if k.dim() == 4 else 0
        code, dt = _code(k), k.dtype
        shape = (batch, self.num_kv_heads, n, d)
        ks, vs = _heads(k, "k", (0, 2, 1), shape, dt, dev), _heads(v, "v", (0, 2, 1), shape, dt, dev)
        rc, axes = _rotary(rotary, dev)
        st, cn = _ints(start, "start", (batch,), dev), _ints(count, "count", (batch,), dev)
        if st is None:
            raise ValueError("start must be given")
        pos = _ints(positions, "positions", (axes, batch, n), dev)
        wk, wq = _weight(k_weight, "k_weight", d, dt, dev), _weight(q_weight, "q_weight", d, dt, dev)
        qs = None
        if q is not None:
            qs = _heads(q, "q", (0, 1, 2), (batch, n, self.num_q_heads, d), dt, dev)
        with _launch_on(dev, stream, k, v, start, block_table, count, positions, k_weight, q, q_weight) as handle:
            qp = None
            if q is not None:
                q_out = torch.empty(q.shape, dtype=dt, device=dev) if q_out is None else _out(q_out, "q_out", tuple(q.shape), dt, dev)
                qp = q_out.data_ptr()
            if batch and n:
                check(_b.tq_byte_append_paged(self.cfg, self.pool.data_ptr(), pt, batch, n, code, ks, vs, st, cn, wk, eps,
                                              rc, pos, qs, wq, qp, self.error.data_ptr(), handle))
        return q_out if q is not None else None

    def attention(self, q, seq_len, block_table, count=None, scale=None, out=None, stream=None):
        """q: CUDA tensor [batch][nq][num_q_heads][d] (or [batch][num_q_heads][d] for one query), any
        strides along the first dims.  The last ``count[b]`` (default nq) positions of sequence b are its
        queries: query i attends to the first ``seq_len[b] - count[b] + 1 + i`` tokens, and rows
        i >= count[b] come out as zeros.  ``scale`` multiplies the scores (default 1 / sqrt(d)).  Returns
        out, contiguous in q's shape and dtype."""
        d, dev = self.head_dim, self.device
        pt = self._pages(block_table)
        q4 = q.unsqueeze(1) if q.dim() == 3 else q
        batch, nq = block_table.shape[0], q4.shape[1] if q4.dim() == 4 else 0
        code = _code(q)
        qs = _heads(q4, "q", (0, 1, 2), (batch, nq, self.num_q_heads, d), q.dtype, dev)
        sl, cn = _ints(seq_len, "seq_len", (batch,), dev), _ints(count, "count", (batch,), dev)
        if sl is None:
            raise ValueError("seq_len must be given")
        with _launch_on(dev, stream, q, seq_len, block_table, count) as handle:
            out = torch.empty(q.shape, dtype=q.dtype, device=dev) if out is None else _out(out, "out", tuple(q.shape), q.dtype, dev)
            if batch and nq:
                need = _b.tq_byte_attention_workspace_bytes(self.cfg, pt, batch, nq, code)
                ws = torch.empty(need, dtype=torch.uint8, device=dev)
                check(_b.tq_byte_attention_paged(self.cfg, self.pool.data_ptr(), pt, batch, nq, code, qs, sl, cn,
                                                 d ** -0.5 if scale is None else float(scale), out.data_ptr(),
                                                 ws.data_ptr(), need, self.error.data_ptr(), handle))
        return out

    def dequantize(self, b, kvh, t0, t1, block_table, stream=None):
        """Tokens [t0, t1) of KV head kvh of entry b as fp32 (k, v) [t1 - t0][d]."""
        pt = self._pages(block_table)
        with _launch_on(self.device, stream, block_table) as handle:
            k = torch.empty(t1 - t0, self.head_dim, dtype=torch.float32, device=self.device)
            v = torch.empty_like(k)
            check(_b.tq_byte_dequantize(self.cfg, self.pool.data_ptr(), pt, block_table.shape[0], b, kvh, t0, t1,
                                        k.data_ptr() or None, v.data_ptr() or None, handle))
        return k, v
