"""Head norms with the position rotation, and the 8-bit paged cache (``tq_norm_rotate`` and the
``tq_byte_*`` entry points of ``include/tq.h``).

``Rotary`` holds a rotation's device table, ``norm_rotate`` applies it (and the norms) to queries and
keys, ``draft_tree`` makes the masks and positions of trees of drafted tokens, and ``PagedByteCache`` owns a
pool of e4m3 codes with a scale for each 16-token block, KV head and side.  Tensors may be strided views (a fused
projection's slices): only the head dimension has to be contiguous, with rows on 16-byte boundaries.  Nothing is copied or converted here; a layout that
the kernels do not take is refused.

The calls compute no gradients: while grad mode is on, inputs that require one are refused.

Calls launch on the current stream of the tensors' device, or on ``stream``.  A call given ``stream``
does not wait for other streams, but holds the memory that it uses, the objects' own included, until
that stream is done with it.  Under ``torch.cuda.stream`` torch's rule for tensors made on another
stream applies to the objects too: keep them until the stream is done, or call with ``stream``.
"""

import importlib.machinery
import importlib.util
import os

import numpy as np
import torch

from . import _build
from . import binding as _b
from .binding import check


def _load_ext():
    path = _build.EXT_PATH
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build the library first, where torch with CUDA is installed "
                          "(python -c 'import __graft_entry__ as g; g.build()')")
    loader = importlib.machinery.ExtensionFileLoader("_tq_torch", path)
    mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_tq_torch", loader))
    loader.exec_module(mod)
    mod.set_error(_b.TQError)
    return mod


# The calls from tensors to the C ABI (csrc/python/tq_torch.cpp): they check the tensors, allocate what
# is returned and launch on the current stream of the tensors' device.
_c = _load_ext()


def _on_stream(stream, held, call, *args):
    """The call with ``stream`` as the current one, so that what it allocates belongs to that stream.
    ``held``: every tensor that its kernels reach, the inputs and what the call's objects own; their memory
    is not handed out again before the stream is done with it."""
    for t in held:
        if t is not None and t.get_device() != stream.device_index:
            raise ValueError("the tensors must be on the stream's device")
    with torch.cuda.stream(stream):
        out = call(*args)
    for t in held:
        if t is not None:
            t.record_stream(stream)
    return out


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
        self._table = torch.from_numpy(host.view(np.int64)).to(_device(device))
        self._args = (self._table, self.rotary_dim, int(self.interleaved), self.num_axes)


def _table(rotary):
    return None if rotary is None else rotary._table


def norm_rotate(q=None, k=None, rotary=None, positions=None, start=None, q_weight=None, k_weight=None, eps=1e-6,
                out_dtype=None, q_out=None, k_out=None, stream=None):
    """RMS norm of every head (where a weight is given) and position rotation (where ``rotary`` is), in
    one pass.

    q: CUDA tensor [batch][n][q_heads][d]; k: [batch][k_heads][n][d] (either may be None); any strides
    along the first three dims.  ``positions``: int32 CUDA [num_axes][batch][n]; None: token j of entry b
    is at ``start[b] + j`` (``start``: int32 CUDA [batch]; None: 0).  ``out_dtype``: q's dtype (default) or float32, which the packed caches'
    queries need.  Returns (q_out, k_out), contiguous in the shapes of q and k.
    """
    if q is None and k is None:
        raise ValueError("neither q nor k given")
    if out_dtype is not None and out_dtype is not torch.float32 and out_dtype != (k if q is None else q).dtype:
        raise ValueError("out_dtype must be the inputs' dtype or float32")
    args = (q, k, None if rotary is None else rotary._args, positions, start, q_weight, k_weight, eps,
            out_dtype is torch.float32, q_out, k_out)
    if stream is None:
        return _c.norm_rotate(*args)
    return _on_stream(stream, (q, k, positions, start, q_weight, k_weight, q_out, k_out, _table(rotary)), _c.norm_rotate,
                      *args)


def draft_tree(parents, start=None, count=None, masks=None, positions=None, stream=None):
    """Masks and positions of trees of drafted tokens.

    parents: int32 CUDA [batch][n], the parent of each draft, which comes before it; -1: the sequence before the
    drafts.  ``count[b]``: entry b has only its first count[b] drafts.  Returns masks ([batch][n][(n + 31) // 32]
    int32: bit j % 32 of word j // 32 of draft i is set where j is i or one of its ancestors), which
    ``PagedByteCache.attention`` takes as ``tree``, and positions ([1][batch][n] int32: ``start[b]``, default 0, plus
    the number of ancestors), which ``PagedByteCache.append`` and ``norm_rotate`` take.  A draft past the count, with a
    parent outside [-1, i), or below such a one has no bits and the position ``start[b]``.  n: at most 1024.
    """
    args = (parents, start, count, masks, positions)
    if stream is None:
        return _c.draft_tree(*args)
    return _on_stream(stream, args, _c.draft_tree, *args)


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
        self._pool = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self._error = torch.zeros(1, dtype=torch.int32, device=self.device)
        # (of tensors, not of their addresses: copies of the object have their own)
        self._args = (self.head_dim, self.num_q_heads, self.num_kv_heads, self.num_pages, self.max_blocks_per_seq,
                      self._pool, self._error)

    # (read-only: the calls hold the tensors)
    @property
    def pool(self):
        return self._pool

    @property
    def error(self):
        return self._error

    def device_error(self):
        """The recorded TQ_DEVERR_* code (0: none), cleared by the call.  Waits for the device: calls may have
        run on any of its streams, and the next may, so the word is read behind all and cleared before the return."""
        torch.cuda.synchronize(self.device)
        code = int(self._error.item())
        if code:
            self._error.zero_()
            torch.cuda.synchronize(self.device)
        return code

    def append(self, k, v, start, block_table, count=None, rotary=None, positions=None, k_weight=None, q=None,
               q_weight=None, eps=1e-6, q_out=None, stream=None):
        """Append k, v ([batch][num_kv_heads][n][d], any strides along the first three dims) at positions
        ``start[b] + j``, keys normed (``k_weight``) and rotated (``rotary``) on the way.

        ``positions`` ([num_axes][batch][n]) are the rotation's positions; None: ``start[b] + j``.
        ``count[b]``: entry b appends only its first count[b] tokens.  ``q`` ([batch][n][num_q_heads][d]) is
        normed and rotated alike in the same launch: returns q_out (None without q)."""
        args = (self._args, k, v, start, block_table, count, None if rotary is None else rotary._args, positions,
                k_weight, q, q_weight, eps, q_out)
        if stream is None:
            return _c.append(*args)
        return _on_stream(stream, (k, v, start, block_table, count, positions, k_weight, q, q_weight, q_out, _table(rotary),
                                   self._pool, self._error), _c.append, *args)

    def attention(self, q, seq_len, block_table, count=None, scale=None, out=None, stream=None, tree=None):
        """q: CUDA tensor [batch][nq][num_q_heads][d] (or [batch][num_q_heads][d] for one query), any
        strides along the first dims.  The last ``count[b]`` (default nq) positions of sequence b are its
        queries: query i attends to the first ``seq_len[b] - count[b] + 1 + i`` tokens, and rows
        i >= count[b] come out as zeros.  ``scale`` multiplies the scores (default 1 / sqrt(d)).  Returns
        out, contiguous in q's shape and dtype.

        ``tree`` (``draft_tree``'s masks, int32 [batch][nq][(nq + 31) // 32]): query i attends to the first
        ``seq_len[b] - count[b]`` tokens and, of the count[b] after them, to those whose bit is set in its mask."""
        args = (self._args, q, seq_len, block_table, count, self.head_dim ** -0.5 if scale is None else scale, out, tree)
        if stream is None:
            return _c.attention(*args)
        return _on_stream(stream, (q, seq_len, block_table, count, out, tree, self._pool, self._error), _c.attention, *args)

    def keep(self, path, start, block_table, count=None, seq_len=None, stream=None):
        """Keep a path of drafts: the token at ``start[b] + path[b][j]`` moves to ``start[b] + j``, for j < count[b]
        (default all).  path: int32 CUDA [batch][n], rising from 0 or more over the count; an entry whose path does
        not rise is left as it is (TQ_DEVERR_BAD_PATH).  Blocks that receive tokens take the largest scale of the blocks
        that these and their other tokens come from.  Returns seq_len, int32 [batch]: ``start[b]`` plus the number of kept
        tokens.  n: at most 1024."""
        args = (self._args, path, start, block_table, count, seq_len)
        if stream is None:
            return _c.keep(*args)
        return _on_stream(stream, (path, start, block_table, count, seq_len, self._pool, self._error), _c.keep, *args)

    def read(self, start, block_table, n, count=None, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
        """Values of n tokens of every entry from ``start[b]`` on: (k, v), contiguous [batch][num_kv_heads][n][d] of
        dtype (float32, bfloat16 or float16), the layout that the appends take.  ``count[b]``: rows from count[b] on are
        zeros.  A value is its code times its block's scale, rounded once."""
        args = (self._args, start, block_table, n, count, dtype, k_out, v_out)
        if stream is None:
            return _c.read(*args)
        return _on_stream(stream, (start, block_table, count, k_out, v_out, self._pool, self._error), _c.read, *args)

    def dequantize(self, b, kvh, t0, t1, block_table):
        """Tokens [t0, t1) of KV head kvh of entry b as fp32 (k, v) [t1 - t0][d]."""
        if (block_table.dtype != torch.int32 or block_table.dim() != 2 or not block_table.is_contiguous()
                or block_table.shape[1] != self.max_blocks_per_seq or block_table.device != self.device):
            raise ValueError(f"block_table must be a contiguous int32 tensor [batch][{self.max_blocks_per_seq}] "
                             f"on {self.device}")
        pt = _b.tq_page_table(block_table.data_ptr(), self.max_blocks_per_seq, self.num_pages)
        with torch.cuda.device(self.device):
            k = torch.empty(max(t1 - t0, 0), self.head_dim, dtype=torch.float32, device=self.device)
            v = torch.empty_like(k)
            check(_b.tq_byte_dequantize(self.cfg, self.pool.data_ptr(), pt, block_table.shape[0], b, kvh, t0, t1,
                                        k.data_ptr() or None, v.data_ptr() or None,
                                        torch.cuda.current_stream().cuda_stream))
        return k, v
