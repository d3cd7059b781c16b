"""The head norm at the ends of its range: rows whose squares leave fp32, eps = 0, and its fp32 error."""

import numpy as np
import pytest
import torch

import byte_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _api():
    import turboquant_quantized_kv_tq_gb300 as tq
    return tq


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,start", [(1, 0), (1, 7), (1, 31), (5, 13), (21, 3)])
def test_append_without_eps_records_nothing(dtype, d, n, start):
    """eps = 0: a block's slots without a new token are no rows.  1e-30 is nothing beside a mean square of ordinary
    keys, so the bytes are those of that call."""
    tq = _api()
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    B, H = 2, 3
    k, v = (torch.randn(B, H, n, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    head = torch.randn(B, H, 40, d, generator=g, device="cuda").to(DT[dtype])
    w = torch.ones(d, device="cuda", dtype=DT[dtype])
    table = _i32([[5, 0, 3], [1, 4, 2]])
    pools = []
    for eps in (0.0, 1e-30):
        c = tq.PagedByteCache(d, H, H, 6, 3)
        c.append(head[:, :, :start], head[:, :, :start], _i32([0, 0]), table)
        c.append(k, v, _i32([start, start]), table, k_weight=w, eps=eps, rotary=tq.Rotary(d))
        assert c.device_error() == 0
        pools.append(c.pool)
    assert torch.equal(*pools)
