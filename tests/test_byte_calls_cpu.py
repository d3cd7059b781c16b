"""Python side of the byte cache's calls without a GPU: what a call on a given stream holds on to."""

import contextlib

import pytest

torch = pytest.importorskip("torch")


class _Tensor:
    """A stand-in that notes on which streams its memory is held."""

    def __init__(self, device=0):
        self.device_index, self.streams = device, []

    def get_device(self):
        return self.device_index

    def record_stream(self, stream):
        self.streams.append(stream)


class _Stream:
    device_index = 0


def _calls(monkeypatch):
    """byte_cache with launches replaced by notes of their arguments."""
    from turboquant_quantized_kv_tq_gb300 import byte_cache

    class Launches:
        seen = []

        def __getattr__(self, name):
            return lambda *args: self.seen.append((name, args))

    monkeypatch.setattr(byte_cache, "_c", Launches())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    return byte_cache


def test_a_call_on_a_stream_holds_what_its_kernels_reach(monkeypatch):
    """The rotary table, the pool and the error word are passed to a launch as addresses: their memory is held on
    the stream as the inputs' is, so that objects may be dropped once the call has returned."""
    m = _calls(monkeypatch)
    rot, cache, s = m.Rotary(64, device="cpu"), m.PagedByteCache(64, 2, 2, 4, 2, device="cpu"), _Stream()
    rot._table, cache._pool, cache._error = _Tensor(), _Tensor(), _Tensor()
    x = [_Tensor() for _ in range(5)]
    m.norm_rotate(x[0], rotary=rot, stream=s)
    assert rot._table.streams == [s] and x[0].streams == [s]
    cache.append(x[1], x[2], x[3], x[4], rotary=rot, stream=s)
    assert rot._table.streams == [s, s] and cache._pool.streams == [s] and cache._error.streams == [s]
    cache.append(x[1], x[2], x[3], x[4], stream=s)
    cache.attention(x[1], x[3], x[4], stream=s)
    assert cache._pool.streams == [s] * 3 and cache._error.streams == [s] * 3
    assert [name for name, _ in m._c.seen] == ["norm_rotate", "append", "append", "attention"]


def test_a_call_on_a_stream_of_another_device_is_refused(monkeypatch):
    m = _calls(monkeypatch)
    rot, x = m.Rotary(64, device="cpu"), _Tensor()
    rot._table = _Tensor(device=1)
    with pytest.raises(ValueError):
        m.norm_rotate(x, rotary=rot, stream=_Stream())
    assert not x.streams and not rot._table.streams and not m._c.seen


# ---- buffers over buffers (made-up addresses: a refused call touches none of them)

P = 1 << 24           # the pool: 9 x 2 blocks of 4128 bytes
A, B, C, OUT, WS = (P + (i << 20) for i in range(1, 6))
POOL_END = P + 9 * 2 * 4128


def _bind():
    return pytest.importorskip("turboquant_quantized_kv_tq_gb300.binding")


def _rows(b, heads, data, n=3, d=128):
    return b.tq_heads(data, n * heads * d, heads * d, d, heads)


@pytest.mark.parametrize("kw", [dict(k=P), dict(v=POOL_END - 16), dict(q=P + 4096), dict(qo=P), dict(qo=POOL_END - 256),
                                dict(qo=P - 6144 + 16)])
def test_append_refuses_buffers_in_the_pool(kw):
    b = _bind()
    at = dict(dict(k=A, v=B, q=C, qo=OUT), **kw)
    st = b.tq_byte_append_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(WS, 4, 8), 1, 3, b.TQ_BF16, _rows(b, 2, at["k"]),
                                _rows(b, 2, at["v"]), WS, None, None, 1e-6, None, None, _rows(b, 8, at["q"]), None, at["qo"], None, None)
    assert st == b.TQ_ERR_INVALID_ARG and b"pool" in b.tq_last_error()


@pytest.mark.parametrize("kw,word", [(dict(out=P), b"pool"), (dict(out=POOL_END - 32), b"pool"), (dict(ws=P), b"pool"),
                                     (dict(ws=P - 256), b"pool"), (dict(out=WS + 1024), b"ws"), (dict(ws=A), b"ws"),
                                     (dict(ws=A - 256), b"ws"), (dict(q=P), b"pool")])
def test_attention_refuses_buffers_over_each_other(kw, word):
    b = _bind()
    at = dict(dict(q=A, out=OUT, ws=WS), **kw)
    cfg, pt = b.tq_byte_config(128, 8, 2), b.tq_page_table(C, 4, 8)
    need = b.tq_byte_attention_workspace_bytes(cfg, pt, 1, 3, b.TQ_BF16)
    st = b.tq_byte_attention_paged(cfg, P, pt, 1, 3, b.TQ_BF16, _rows(b, 8, at["q"]), C, None, 0.1, at["out"], at["ws"], need, None, None)
    assert st == b.TQ_ERR_INVALID_ARG and word in b.tq_last_error()


@pytest.mark.parametrize("ko", [OUT, OUT + 6144 - 16, OUT - 1536 + 16])
def test_norm_rotate_refuses_outputs_over_each_other(ko):
    b = _bind()
    st = b.tq_norm_rotate(128, b.TQ_BF16, b.TQ_BF16, 1, 3, _rows(b, 8, A), None, OUT, _rows(b, 2, B), None, ko, 1e-6, None, None, None, None)
    assert st == b.TQ_ERR_INVALID_ARG and b"outputs" in b.tq_last_error()


# ---- inputs

def test_inputs_that_require_a_gradient_are_refused():
    """The calls compute no gradients: they say so instead of returning tensors without a graph."""
    from turboquant_quantized_kv_tq_gb300 import PagedByteCache
    c = PagedByteCache(64, 2, 2, 4, 2, device="cpu")
    x, start, table = torch.zeros(1, 2, 3, 64), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    q, w = torch.zeros(1, 3, 2, 64), torch.ones(64)

    def grad(t):
        return t.clone().requires_grad_()

    calls = [lambda: c.append(grad(x), x, start, table), lambda: c.append(x, grad(x), start, table),
             lambda: c.append(x, x, start, table, k_weight=grad(w)), lambda: c.append(x, x, start, table, q=grad(q)),
             lambda: c.append(x, x, start, table, q=q, q_weight=grad(w)),
             lambda: c.attention(grad(q), start, table), lambda: c.attention(grad(q[:, 0]), start, table)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):  # (what stops it here)
            call()


def test_negated_views_are_refused():
    """A view whose negation is pending (torch.imag of a conjugate) holds other numbers in memory than it stands for."""
    from turboquant_quantized_kv_tq_gb300 import PagedByteCache
    c = PagedByteCache(64, 2, 2, 4, 2, device="cpu")
    q = torch._neg_view(torch.ones(1, 2, 64))
    with pytest.raises(ValueError, match="negat"):
        c.attention(q, torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32))


# ---- copies of the objects

@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_copies_use_their_own_memory(monkeypatch, how):
    """A copied (or saved and loaded) object's calls reach the copy's tensors, not those it was copied from: a model
    that holds a Rotary is copied as a whole, and the first may be gone."""
    import copy
    import pickle
    m = _calls(monkeypatch)
    make = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda x: pickle.loads(pickle.dumps(x))}[how]

    def address(x):
        return x.data_ptr() if isinstance(x, torch.Tensor) else x

    rot, cache = m.Rotary(64, device="cpu"), m.PagedByteCache(64, 2, 2, 4, 2, device="cpu")
    cache.pool.fill_(7)
    r, c = make(rot), make(cache)
    assert (r._table.data_ptr() == rot._table.data_ptr()) == (how == "copy")
    assert torch.equal(c.pool, cache.pool) and torch.equal(r._table, rot._table)
    m._c.seen.clear()
    c.append(None, None, None, None, rotary=r)
    c.attention(None, None, None)
    m.norm_rotate(torch.zeros(1), rotary=r)
    (_, app), (_, att), (_, nr) = m._c.seen
    for args in (app[0], att[0]):
        assert {c.pool.data_ptr(), c.error.data_ptr()} <= {address(x) for x in args}
    for args in (app[6], nr[2]):
        assert address(args[0]) == r._table.data_ptr()


def test_resized_pools_are_refused():
    from turboquant_quantized_kv_tq_gb300 import PagedByteCache
    c = PagedByteCache(64, 2, 2, 4, 2, device="cpu")
    q, seq, table = torch.zeros(1, 2, 64), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 2, dtype=torch.int32)
    c.pool.resize_(c.pool.numel() - 1)
    with pytest.raises(ValueError, match="pool"):
        c.attention(q, seq, table)
