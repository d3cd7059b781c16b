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
