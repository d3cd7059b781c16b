"""Counts of drafts that pass what a call holds reach the kernels as they are: they count as nq, and nothing behind the
masks', the queries' or the output's rows is read or written."""

import numpy as np
import pytest
import torch

import byte_reference as ref
import tree_reference as tree
from test_gpu_byte_cache import DT, _i32, _np
from test_gpu_tree import _check, _filled, _terms

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d,Hq,H,nq", [("bf16", 128, 4, 2, 3), ("bf16", 128, 4, 2, 20), ("f16", 128, 8, 2, 33), ("bf16", 64, 4, 2, 20),
                                             ("f16", 64, 8, 1, 17), ("f32", 128, 4, 2, 12), ("f32", 64, 4, 4, 2), ("bf16", 256, 4, 2, 20)])
def test_counts_past_the_drafts(dtype, d, Hq, H, nq):
    seq, cnt = [300, 129, 5, 0, 64], [nq + 5, 2147483647, nq + 1, nq + 9, -2147483648]
    B, words = len(seq), (nq + 31) // 32
    c, table, g = _filled(d, Hq, H, seq, 20, dtype, seed=nq)
    sees = np.random.RandomState(nq).rand(B, nq, nq) < 0.5
    # inputs and output in the middle of larger buffers: NaN queries and full masks around them, a mark around the output
    masks = torch.full((B + 2, nq, words), -1, dtype=torch.int32, device="cuda")
    masks[1:-1] = _i32(tree.pack(sees))
    q = torch.full((B + 2, nq, Hq, d), float("nan"), dtype=DT[dtype], device="cuda")
    q[1:-1] = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    out = torch.full_like(q, 77.0)
    got = c.attention(q[1:-1], _i32(seq), _i32(table), count=_i32(cnt), tree=masks[1:-1], out=out[1:-1])
    assert got.data_ptr() == out[1].data_ptr() and torch.all(out[0] == 77) and torch.all(out[-1] == 77)
    pool, live = ref.Pool(c.pool.cpu().numpy(), H, d), [min(max(k, 0), nq) for k in cnt]
    want, spread, reach, least = tree.attention(_np(q[1:-1]), pool, seq, live, table, d ** -0.5, sees, 2.0 ** -31)
    wide = _terms(_np(q[1:-1]), pool, seq, live, table, d ** -0.5, dtype != "f32" and d != 256 and Hq // H * nq > 8)
    _check(got, want, spread, reach, max(seq), d, DT[dtype], wide, least)
    assert torch.all(got[3:] == 0) and c.device_error() == 0
