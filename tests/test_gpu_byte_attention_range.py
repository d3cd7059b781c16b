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


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,nq", [(4, 4, 1), (8, 2, 3), (8, 1, 6), (2, 1, 40)])
@pytest.mark.parametrize("outlier", [0, 12, 14])
def test_fp32_keeps_its_bits(d, hq, hkv, nq, outlier):
    """The 2-norm of an fp32 result's error, with ordinary queries and with one channel 2^outlier above the others
    that the keys hold zeros for (so that the others decide).

    A score is the sum of d / 8 products (two terms of 16 coordinates each) in the tensor cores' truncating
    accumulator, at most 2^-23 of the running sum each, and a handful of fp32 roundings; with S the scores' rms it is
    off by less than (d / 8 + 8) 2^-23 S.  Weights are off by that and by 2^-21 (ex2, the second fp16 term, sums), and
    both enter the result at most twice (numerator and denominator).  One fp16 term alone for the queries or the weights
    would be off by 2^-12 / sqrt 3 = 1.4e-4, ten times that and more."""
    g = torch.Generator(device="cuda")
    g.manual_seed(d + nq)
    lens = [301, 95]
    k, v = (torch.randn(2, hkv, 301, d, generator=g, device="cuda") for _ in range(2))
    q = torch.randn(2, nq, hq, d, generator=g, device="cuda")
    if outlier:
        k[..., 3] = 0.0
        q[..., 3] = 2.0 ** outlier * (1 + q[..., 3].abs())
    c, table, pool = _filled(d, hq, hkv, lens, k, v)
    out = _np(c.attention(q, _i32(lens), _i32(table)))
    want, _, _ = ref.attention(_np(q), pool, lens, [nq] * 2, table, d ** -0.5)
    keys = np.concatenate([pool.read(0, h, table[0], 301) for h in range(hkv)])
    S = np.sqrt(np.mean((_np(q[0]).reshape(-1, d) @ keys.T) ** 2) / d)
    tol = 2 * ((d / 8 + 8) * 2.0 ** -23 * S + 2.0 ** -21)
    assert tol <= 1.5e-5
    err = np.linalg.norm(out - want) / np.linalg.norm(want)
    assert err <= tol, (err, tol)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_whole_prompts(dtype):
    """Prompts of thousands of queries in one call (64 row groups), of unlike lengths."""
    lens, count, nq, d = [4096, 5000, 130], [4096, 3333, 130], 4096, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    k, v = (torch.randn(3, 1, 5000, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    c, table, pool = _filled(d, 4, 1, lens, k, v)
    q = torch.randn(3, nq, 4, d, generator=g, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32(lens), _i32(table), count=_i32(count))
    assert torch.equal(out, c.attention(q, _i32(lens), _i32(table), count=_i32(count)))
    assert c.device_error() == 0
    half = torch.finfo(DT[dtype]).eps / 2
    for b in range(3):
        assert not out[b, count[b]:].any()
        K, V = (torch.from_numpy(pool.read(s, 0, table[b][:(lens[b] + 15) // 16], lens[b])).cuda() for s in (0, 1))
        for i0 in range(0, count[b], 512):
            m = min(512, count[b] - i0)
            x = q[b, i0:i0 + m].double().transpose(0, 1)                                  # [4][m][d]
            limit = lens[b] - count[b] + 1 + i0 + torch.arange(m, device="cuda")
            s = (x @ K.T * d ** -0.5).masked_fill_(torch.arange(lens[b], device="cuda") >= limit[:, None], -np.inf)
            p = torch.softmax(s, -1)
            want, spread = p @ V, p @ V.abs()
            reach = (x.abs() @ K.abs().T).amax(-1, keepdim=True) * d ** -0.5
            # as for the smaller chunks: weights rounded to fp16, twice the scores' error, sums; the output's own step
            score = (d + lens[b] / 16 + 64) * 2.0 ** -22 * (1 + reach)
            tol = spread * (2.0 ** -11 + 2 * score + (lens[b] / 16 + 64) * 2.0 ** -23) + want.abs() * half + 2.0 ** -24
            got = out[b, i0:i0 + m].double().transpose(0, 1)
            assert bool(((got - want).abs() <= tol).all()), (b, i0)
