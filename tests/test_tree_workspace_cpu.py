"""The tree attention's workspace holds what either of its kernels writes there."""

import pytest

HEADS = 16384   # heads of the ranges, before the partials
SMS = 152


def _bind():
    return pytest.importorskip("turboquant_quantized_kv_tq_gb300.binding")


@pytest.mark.parametrize("dtype", ["TQ_F32", "TQ_BF16", "TQ_F16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Hq,H", [(32, 8), (8, 1), (5, 5)])
def test_partials_of_every_block_fit(d, dtype, Hq, H):
    """Two partials (M, l and O of each row) a block.  On tensor memory: 128 rows, a block per SM, and (M, l) of 256 threads.
    Otherwise 8 or 16 rows and up to 512 blocks, two to an SM."""
    b = _bind()
    code = getattr(b, dtype)
    for nq in (1, 2, 3, 8, 9, 16, 33, 64, 1024):
        rows = nq * Hq // H
        need = b.tq_byte_tree_attention_workspace_bytes(b.tq_byte_config(d, Hq, H), 4, nq, code)
        wide = rows > 8 and d * (2 if dtype == "TQ_F32" else 1) <= 256
        assert need >= HEADS + 2 * 512 * (16 if wide else 8) * (d + 2) * 4
        if dtype != "TQ_F32" and d < 256 and rows > 8:
            assert need >= HEADS + SMS * (2 * 128 * (d + 2) + 2 * 256) * 4
