"""Trees of drafts, keep and read without a GPU: what the calls refuse (made-up addresses: a refused call touches
none of them), what they hold on a stream, and the plain forms against each other."""

import contextlib

import numpy as np
import pytest

import byte_reference as ref
import tree_reference as tree

P = 1 << 24           # the pool: 9 x 2 blocks of 4128 bytes
A, B, C, OUT, WS, M = (P + (i << 20) for i in range(1, 7))
POOL_END = P + 9 * 2 * 4128


def _bind():
    return pytest.importorskip("turboquant_quantized_kv_tq_gb300.binding")


def _refused(b, status, code, word):
    assert status == code and word in b.tq_last_error(), (status, b.tq_last_error())


# ---- refusals

@pytest.mark.parametrize("kw,code,word", [
    (dict(batch=0), "INVALID_ARG", b"batch"), (dict(batch=513), "INVALID_ARG", b"batch"), (dict(n=-1), "INVALID_ARG", b"n must"),
    (dict(n=1025), "UNSUPPORTED", b"TQ_MAX_DRAFTS"), (dict(parents=None), "INVALID_ARG", b"null"),
    (dict(masks=None), "INVALID_ARG", b"null"), (dict(positions=None), "INVALID_ARG", b"null"),
    (dict(parents=A + 2), "INVALID_ARG", b"misaligned"), (dict(count=A + 1), "INVALID_ARG", b"misaligned"),
    (dict(masks=A + 4), "INVALID_ARG", b"overlaps"), (dict(positions=B + 4), "INVALID_ARG", b"overlaps"),
    (dict(count=M), "INVALID_ARG", b"overlaps"), (dict(positions=M + 4 * 2 * 40 * 2 - 4), "INVALID_ARG", b"overlap")])
def test_draft_tree_refuses(kw, code, word):
    b = _bind()
    a = dict(dict(batch=2, n=40, parents=A, start=B, count=C, masks=M, positions=OUT), **kw)
    st = b.tq_draft_tree(a["batch"], a["n"], a["parents"], a["start"], a["count"], a["masks"], a["positions"], None)
    _refused(b, st, getattr(b, "TQ_ERR_" + code), word)


def test_draft_tree_of_nothing():
    b = _bind()
    assert b.tq_draft_tree(3, 0, A, None, None, M, OUT, None) == b.TQ_OK


@pytest.mark.parametrize("kw,code,word", [
    (dict(masks=None), "INVALID_ARG", b"null masks"), (dict(masks=M + 2), "INVALID_ARG", b"masks"),
    (dict(nq=1025), "UNSUPPORTED", b"TQ_MAX_DRAFTS"), (dict(masks=OUT + 64), "INVALID_ARG", b"masks"),
    (dict(masks=WS + 256), "INVALID_ARG", b"masks"), (dict(out=P), "INVALID_ARG", b"pool"), (dict(ws=POOL_END - 32), "INVALID_ARG", b""),
    (dict(ws_bytes=0), "WORKSPACE", b"workspace"), (dict(scale=float("nan")), "INVALID_ARG", b"scale"),
    (dict(q=OUT), "INVALID_ARG", b"overlap"), (dict(nq=0), "INVALID_ARG", b"nq"), (dict(seq=None), "INVALID_ARG", b"null")])
def test_tree_attention_refuses(kw, code, word):
    b = _bind()
    a = dict(dict(nq=6, q=A, seq=B, masks=M, scale=0.1, out=OUT, ws=WS, ws_bytes=1 << 28), **kw)
    rows = b.tq_heads(a["q"], 6 * 8 * 128, 8 * 128, 128, 8)
    st = b.tq_byte_tree_attention_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(C, 4, 8), 1, a["nq"], b.TQ_BF16, rows, a["seq"],
                                        None, a["masks"], a["scale"], a["out"], a["ws"], a["ws_bytes"], None, None)
    _refused(b, st, getattr(b, "TQ_ERR_" + code), word)


@pytest.mark.parametrize("d,dt", [(64, 0), (64, 1), (128, 0), (128, 1), (128, 2), (256, 1)])
def test_tree_attention_workspace(d, dt):
    """Enough for two partials of every block of either kernel, whatever the drafts are; none for refused calls."""
    b = _bind()
    code = (b.TQ_F32, b.TQ_BF16, b.TQ_F16)[dt]
    for nq in (1, 2, 16, 33, 1024):
        need = b.tq_byte_tree_attention_workspace_bytes(b.tq_byte_config(d, 32, 8), 4, nq, code)
        rows = min(4 * nq, 128)
        assert need >= 2 * 152 * (8 if rows <= 8 or d == 256 else 16) * (d + 2) * 4
    assert b.tq_byte_tree_attention_workspace_bytes(b.tq_byte_config(d, 32, 8), 4, 1025, code) == 0
    assert b.tq_byte_tree_attention_workspace_bytes(b.tq_byte_config(d, 32, 8), 4, 0, code) == 0


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=1025), "UNSUPPORTED", b"TQ_MAX_DRAFTS"), (dict(n=-1), "INVALID_ARG", b"n must"), (dict(batch=0), "INVALID_ARG", b"batch"),
    (dict(path=None), "INVALID_ARG", b"null"), (dict(start=None), "INVALID_ARG", b"null"), (dict(path=A + 1), "INVALID_ARG", b"misaligned"),
    (dict(out=A + 8), "INVALID_ARG", b"seq_len"), (dict(out=B), "INVALID_ARG", b"seq_len"), (dict(out=C), "INVALID_ARG", b"seq_len"),
    (dict(out=WS + 4), "INVALID_ARG", b"seq_len"), (dict(path=P + 64), "INVALID_ARG", b"pool"), (dict(out=POOL_END - 4), "INVALID_ARG", b"pool")])
def test_keep_refuses(kw, code, word):
    b = _bind()
    a = dict(dict(batch=2, n=5, path=A, start=B, count=C, out=OUT), **kw)
    st = b.tq_byte_keep_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(WS, 4, 8), a["batch"], a["n"], a["path"], a["start"],
                              a["count"], a["out"], None, None)
    _refused(b, st, getattr(b, "TQ_ERR_" + code), word)


@pytest.mark.parametrize("kw,code,word", [
    (dict(n=-1), "INVALID_ARG", b"n must"), (dict(batch=0), "INVALID_ARG", b"batch"), (dict(start=None), "INVALID_ARG", b"null"),
    (dict(k=None), "INVALID_ARG", b"null"), (dict(k=OUT + 8), "INVALID_ARG", b"aligned"), (dict(dtype=7), "INVALID_ARG", b"dtype"),
    (dict(k=P + 256), "INVALID_ARG", b"pool"), (dict(v=OUT + 1024), "INVALID_ARG", b"outputs overlap"), (dict(v=B), "INVALID_ARG", b"input"),
    (dict(k=WS), "INVALID_ARG", b"input"), (dict(count=C + 2), "INVALID_ARG", b"misaligned")])
def test_read_refuses(kw, code, word):
    b = _bind()
    a = dict(dict(batch=1, n=5, k=OUT, v=M, start=B, count=C, dtype=b.TQ_BF16), **kw)
    st = b.tq_byte_read_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(WS, 4, 8), a["batch"], a["n"], a["dtype"], a["start"],
                              a["count"], a["k"], a["v"], None, None)
    _refused(b, st, getattr(b, "TQ_ERR_" + code), word)
    assert b.tq_byte_read_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(WS, 4, 8), 1, 0, b.TQ_BF16, B, None, None, None, None,
                                None) == b.TQ_OK


def test_python_refuses_what_is_not_on_the_device():
    torch = pytest.importorskip("torch")
    tq = pytest.importorskip("turboquant_quantized_kv_tq_gb300")
    if not hasattr(tq, "draft_tree"):
        pytest.skip("no torch extension")
    with pytest.raises(ValueError):
        tq.draft_tree(torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError):
        tq.draft_tree([[0, 1]])


# ---- what a call on a stream holds

class _Tensor:
    def __init__(self, device=0):
        self.device_index, self.streams = device, []

    def get_device(self):
        return self.device_index

    def record_stream(self, stream):
        self.streams.append(stream)


class _Stream:
    device_index = 0


def test_calls_on_a_stream_hold_what_their_kernels_reach(monkeypatch):
    torch = pytest.importorskip("torch")
    from turboquant_quantized_kv_tq_gb300 import byte_cache as m

    seen = []

    class Launches:
        def __getattr__(self, name):
            return lambda *args: seen.append(name)

    monkeypatch.setattr(m, "_c", Launches())
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    cache, s = m.PagedByteCache(64, 2, 2, 4, 2, device="cpu"), _Stream()
    cache._pool, cache._error = _Tensor(), _Tensor()
    x = [_Tensor() for _ in range(16)]
    m.draft_tree(x[0], start=x[1], count=x[2], masks=x[3], positions=x[4], stream=s)
    cache.attention(x[5], x[6], x[7], tree=x[8], stream=s)
    cache.keep(x[9], x[10], x[7], count=x[11], seq_len=x[12], stream=s)
    cache.read(x[13], x[7], 3, count=x[14], k_out=x[15], stream=s)
    assert seen == ["draft_tree", "attention", "keep", "read"]
    assert [len(t.streams) for t in x] == [1] * 7 + [3] + [1] * 8
    assert len(cache._pool.streams) == 3 and len(cache._error.streams) == 3
    with pytest.raises(ValueError):
        m.draft_tree(_Tensor(device=1), stream=s)


# ---- the plain forms

def test_reference_masks_of_a_hand_made_tree():
    #     0         5 (second root)
    #    / \        |
    #   1   2       6
    #       |
    #       3 - 4 (4's parent is 3)
    sees, pos = tree.masks_positions(np.array([[-1, 0, 0, 2, 3, -1, 5, 9]]), [8], [10])
    want = [{0}, {1, 0}, {2, 0}, {3, 2, 0}, {4, 3, 2, 0}, {5}, {6, 5}, set()]
    assert [set(np.flatnonzero(r)) for r in sees[0]] == want
    assert pos[0].tolist() == [10, 11, 11, 12, 13, 10, 11, 10]
    assert tree.pack(sees)[0, :, 0].tolist() == [1, 3, 5, 13, 29, 32, 96, 0]


def test_reference_keep_equals_a_cache_of_the_kept_tokens_alone():
    """With one scale everywhere nothing is rounded twice: the values are those of an append of the path alone."""
    rs = np.random.RandomState(0)
    B, H, d, n = 2, 2, 64, 20
    table = np.arange(B * 4).reshape(B, 4)
    pool = ref.Pool(np.zeros(9 * H * (32 * d + 32), dtype=np.uint8), H, d)
    x = rs.uniform(0.6, 1.0, (2, B, H, 40, d)) * rs.choice([-1, 1], (2, B, H, 40, d))
    for side in (0, 1):
        pool.append(side, x[side, :, :, :13 + n], [0, 0], table)
    path, cnt = np.array([[0, 2, 5, 17, 19], [1, 4, 18, 0, 0]]), [5, 3]
    tree.keep(pool, path, [13, 13], cnt, table)
    other = ref.Pool(np.zeros(9 * H * (32 * d + 32), dtype=np.uint8), H, d)
    for b in range(B):
        kept = list(range(13)) + [13 + p for p in path[b, :cnt[b]]]
        for side in (0, 1):
            other.append(side, x[side][:, :, kept], [0, 0], table)
        for side in (0, 1):
            for h in range(H):
                assert np.array_equal(pool.read(side, h, table[b], len(kept)), other.read(side, h, table[b], len(kept)))
