"""Sums of tree attention over long sequences: a batch large enough that one SM walks a whole sequence."""

import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _batch(d, Hq, H, B, T, nq, dtype, parts=False):
    """B entries that share the pages of one sequence of T tokens, and draft masks of which every bit is set.  Values have the
    mean 1, so that sums grow all the way, or (parts) a mean of its own in every 2048 tokens, so that none can be missed."""
    import turboquant_quantized_kv_tq_gb300 as tq
    blocks = (T + 15) // 16
    c = tq.PagedByteCache(d, Hq, H, blocks, blocks)
    g = torch.Generator(device="cuda")
    g.manual_seed(d + nq)
    k, v = (torch.randn(1, H, T, d, generator=g, device="cuda") for _ in range(2))
    table = torch.arange(blocks, dtype=torch.int32, device="cuda")[None]
    if parts:
        v = 0.3 * v + torch.randn(1, H, T // 2048 + 1, d, generator=g, device="cuda").repeat_interleave(2048, 2)[:, :, :T]
    else:
        v = 1 + v
    c.append(k.to(DT[dtype]), v.to(DT[dtype]), _i32([0]), table)
    assert c.device_error() == 0
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    tree = torch.full((B, nq, (nq + 31) // 32), -1, dtype=torch.int32, device="cuda")
    return c, table, q, tree


def _exact(c, table, q, n, H, d):
    """float64 [nq][Hq][d] of one entry whose queries all attend to n tokens; sum p |v|; and the rows' largest scale sum |q||k|
    and scale max |q| sum |k| ([nq][Hq][1])."""
    K, V = (x[0].double() for x in c.read(_i32([0]), table, n, dtype=torch.float32))
    x = q.double().view(q.shape[0], H, -1, d)
    p = torch.softmax(torch.einsum("nhgd,htd->nhgt", x, K) * d ** -0.5, -1)
    out, spread = (torch.einsum("nhgt,htd->nhgd", p, y).reshape(q.shape) for y in (V, V.abs()))
    reach = torch.einsum("nhgd,htd->nhgt", x.abs(), K.abs()).amax(-1).reshape(*q.shape[:2], 1) * d ** -0.5
    wide = (x.abs().amax(-1) * K.abs().sum(-1).amax(-1)[None, :, None]).reshape(*q.shape[:2], 1) * d ** -0.5
    return out, spread, reach, wide


@pytest.mark.parametrize("d,nq", [(64, 8), (64, 40), (128, 8), (128, 16), (128, 40), (256, 8)])
def test_long_sequences_keep_their_sums(d, nq):
    """The part of the result along the exact one, over 100000 tokens of a batch with a (sequence, head) for every SM.

    A product added to the tensor cores' fp32 sum may truncate up to 2^-23 of the sum.  Over a chain of n products whose
    sum grows evenly that is n / 2 2^-23 of it; 1024 products of 16 tokens: 6.1e-5.  The outputs' roundings (2^-11 at most each, 2^-11 / sqrt 3
    deviation, 4000 values or more) and the weights' (as many, and more tokens) cancel but for 5 deviations of them: 2.3e-5.  (A
    chain over the whole sequence, 6250 products, lost 1.9e-4 with 64 rows or less and 4.1e-4 above.)"""
    Hq, H, B, T = 8, 4, 38, 100000
    c, table, q, tree = _batch(d, Hq, H, B, T, nq, "f16")
    out = c.attention(q, _i32([T] * B), table.expand(B, -1).contiguous(), tree=tree)
    for b in (0, B // 2, B - 1):
        want, got = _exact(c, table, q[b], T, H, d)[0], out[b].double()
        assert abs(float((got * want).sum() / (want * want).sum()) - 1) <= 6.1e-5 + 2.3e-5, b


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,Hq,nq", [(64, 4, 9), (64, 4, 70), (128, 4, 9), (128, 4, 64), (128, 7, 23)])
def test_stretches_of_one_range_join(dtype, d, Hq, nq):
    """Sequences of lengths about those where a block's part of one is cut (128 tiles of 128 tokens and multiples of them), counts that
    leave warps without a row that asks, a slab that a range ends in, and few slabs; each entry against float64."""
    H, T, B = 1, 50000, 150
    c, table, q, tree = _batch(d, Hq, H, B, T, nq, dtype, parts=True)
    some = {0: 16384, 1: 16385, 2: 16383, 3: 32768, 4: 32769, 40: 49999, 41: 1, 42: 0, 77: 128 * 257, 120: 33000, 149: 50000}
    seq = [some.get(b, 40000 + 61 * b) for b in range(B)]
    cnt = [0 if b == 3 else 1 if b == 77 else nq // 2 if b % 3 == 1 else nq for b in range(B)]
    out = c.attention(q, _i32(seq), table.expand(B, -1).contiguous(), count=_i32(cnt), tree=tree)
    assert torch.equal(out, c.attention(q, _i32(seq), table.expand(B, -1).contiguous(), count=_i32(cnt), tree=tree))
    assert c.device_error() == 0
    half = torch.finfo(DT[dtype]).eps / 2
    for b in sorted(some) + [5, 60, 148]:
        k = min(cnt[b], nq) if seq[b] else 0
        assert not out[b, k:].any()
        if k == 0:
            continue
        want, spread, reach, wide = _exact(c, table, q[b, :k], seq[b], H, d)
        # weights rounded to fp16 (2^-11); scores in fp32 ((d + 64) 2^-22 of the row's reach and of 1) of queries whose e4m3 terms are
        # exact to 2^-18 of the row's largest value, twice; sums cut as above (6.1e-5) and joined (64 2^-23)
        score = (d + 64) * 2.0 ** -22 * (1 + reach) + 2.0 ** -18 * wide
        tol = spread * (2.0 ** -11 + 2 * score + 6.1e-5 + 64 * 2.0 ** -23) + want.abs() * half + 2.0 ** -24
        err = (out[b, :k].double() - want).abs() / tol
        assert float(err.max()) <= 1, (b, float(err.max()))
