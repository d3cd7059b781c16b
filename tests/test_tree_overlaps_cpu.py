"""Outputs over what a call reads besides its tensors, refused before anything is launched (made-up addresses)."""

import pytest

P = 1 << 24  # the pool: 9 x 2 blocks of 4128 bytes
A, SEQ, TABLE, OUT, WS, M, COUNT, ERR = (P + (i << 20) for i in range(1, 9))


def _bind():
    return pytest.importorskip("turboquant_quantized_kv_tq_gb300.binding")


@pytest.mark.parametrize("kw", [dict(out=SEQ), dict(out=COUNT - 16), dict(out=TABLE), dict(out=ERR), dict(ws=SEQ - 256), dict(ws=TABLE), dict(ws=ERR),
                                dict(ws=COUNT)])
def test_tree_attention_outputs(kw):
    b = _bind()
    a = dict(dict(out=OUT, ws=P + (64 << 20)), **kw)
    rows = b.tq_heads(A, 6 * 8 * 128, 8 * 128, 128, 8)
    st = b.tq_byte_tree_attention_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(TABLE, 4, 8), 1, 6, b.TQ_BF16, rows, SEQ, COUNT, M,
                                        0.1, a["out"], a["ws"], 1 << 28, ERR, None)
    assert st == b.TQ_ERR_INVALID_ARG and b"overlap" in b.tq_last_error()


def test_keep_lengths_over_the_error_word():
    b = _bind()
    st = b.tq_byte_keep_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(TABLE, 4, 8), 2, 5, A, SEQ, COUNT, ERR - 4, ERR, None)
    assert st == b.TQ_ERR_INVALID_ARG and b"seq_len" in b.tq_last_error()


@pytest.mark.parametrize("kw", [dict(k=ERR), dict(v=ERR - 256)])
def test_read_outputs_over_the_error_word(kw):
    b = _bind()
    a = dict(dict(k=OUT, v=M), **kw)
    st = b.tq_byte_read_paged(b.tq_byte_config(128, 8, 2), P, b.tq_page_table(TABLE, 4, 8), 1, 5, b.TQ_BF16, SEQ, COUNT, a["k"], a["v"], ERR, None)
    assert st == b.TQ_ERR_INVALID_ARG and b"overlap" in b.tq_last_error()
