"""Byte attention at the ends of its range: infinite queries, queries with outlier channels, fp32's own precision,
whole prompts."""

import numpy as np
import pytest
import torch

import byte_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def _np(t):
    return t.detach().to(torch.float64).cpu().numpy()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _filled(d, hq, hkv, lens, keys, values):
    """A cache with the first lens[b] tokens of keys and values ([B][hkv][T][d]), its block table and its bytes."""
    import turboquant_quantized_kv_tq_gb300 as tq
    B, blocks = len(lens), max(1, (max(lens) + 15) // 16)
    c = tq.PagedByteCache(d, hq, hkv, B * blocks + 1, blocks)
    table = np.random.RandomState(d).permutation(B * blocks).reshape(B, blocks).astype(np.int32)
    c.append(keys, values, _i32([0] * B), _i32(table), count=_i32(lens))
    assert c.device_error() == 0
    return c, table, ref.Pool(c.pool.cpu().numpy(), hkv, d)


@pytest.mark.parametrize("dtype,d,hq,nq", [("bf16", 128, 4, 1), ("f16", 64, 4, 1), ("bf16", 256, 4, 3), ("f16", 128, 4, 4), ("f32", 128, 4, 1),
                                           ("f16", 64, 2, 50), ("bf16", 256, 1, 70), ("f32", 128, 2, 40), ("bf16", 128, 4, 40)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_query_is_nan_in_its_row(dtype, d, hq, nq, sign):
    """A key channel of one sign (and one-token sequences) turns an infinite query into scores that are all +inf or
    all -inf; infinity minus infinity is NaN either way."""
    lens = [300, nq, 17 + nq]
    g = torch.Generator(device="cuda")
    g.manual_seed(nq)
    k, v = (torch.randn(3, 1, 300, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    k[..., 5] = 0.5 + k[..., 5].abs()
    c, table, _ = _filled(d, hq, 1, lens, k, v)
    q = torch.randn(3, nq, hq, d, generator=g, device="cuda").to(DT[dtype])
    clean = c.attention(q, _i32(lens), _i32(table))
    assert torch.isfinite(clean).all()
    hit = torch.zeros(3, nq, hq, dtype=torch.bool, device="cuda")
    hit[:, 0, 0] = hit[:, nq - 1, hq - 1] = hit[0, nq // 2, 0] = True
    q[..., 5] = torch.where(hit, torch.full_like(q[..., 5], sign * float("inf")), q[..., 5])
    out = c.attention(q, _i32(lens), _i32(table))
    assert torch.isnan(out[hit]).all()
    assert torch.equal(out[~hit], clean[~hit])
