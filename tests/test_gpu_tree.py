"""Trees of drafted tokens over the byte cache, keep and read on the GPU against their plain forms.

Tolerances: attention as in test_gpu_byte_cache.py (the same arithmetic; bits select tokens and add none).  16-bit
queries of more than 8 rows may enter as e4m3 terms, off by 2^-18 of the row's largest value a coordinate: a score is off
by at most 2^-18 d max|q| max|k| scale, which is counted on top.  Everything else is equal: masks, positions, bytes and
values (a value of 4 significant bits times a power of two is rounded by no type but where it leaves the range).
"""

import numpy as np
import pytest
import torch

import byte_reference as ref
import tree_reference as tree
from test_gpu_byte_cache import DT, _api, _cache, _half_step, _i32, _np, _table

pytestmark = pytest.mark.gpu


def _parents(rs, B, n, reach):
    back = rs.randint(1, reach + 1, (B, n))
    return np.maximum(np.arange(n)[None] - back, -1).astype(np.int32)


# ---- masks and positions

@pytest.mark.parametrize("B,n,reach", [(1, 1, 1), (1, 8, 3), (3, 31, 4), (2, 32, 40), (5, 33, 1), (2, 64, 9), (64, 257, 30), (2, 1024, 1),
                                       (3, 1000, 200)])
def test_draft_tree(B, n, reach):
    rs = np.random.RandomState(n)
    parents = _parents(rs, B, n, reach)
    start = rs.randint(0, 1 << 30, B).astype(np.int32)
    count = rs.randint(-1, n + 3, B).astype(np.int32)
    sees, pos = tree.masks_positions(parents, np.minimum(count, n), start)
    m, p = _api().draft_tree(_i32(parents), start=_i32(start), count=_i32(count))
    assert m.shape == (B, n, (n + 31) // 32) and p.shape == (1, B, n) and m.dtype == p.dtype == torch.int32
    assert np.array_equal(m.cpu().numpy(), tree.pack(sees))
    assert np.array_equal(p[0].cpu().numpy(), pos)
    sees, pos = tree.masks_positions(parents, [n] * B, [0] * B)
    mine = torch.full_like(m, -1)
    m, p = _api().draft_tree(_i32(parents), masks=mine)
    assert m is mine and np.array_equal(m.cpu().numpy(), tree.pack(sees)) and np.array_equal(p[0].cpu().numpy(), pos)


def test_draft_tree_with_bad_parents():
    """A parent that does not come before its child, or is below -1, takes its draft and what hangs on it out."""
    rs = np.random.RandomState(5)
    B, n = 16, 70
    parents = _parents(rs, B, n, 6)
    wrong = rs.rand(B, n) < 0.1
    parents[wrong] = rs.choice([-2, -2147483648, 2147483647, 70, 69], wrong.sum())
    parents[0, 5] = 5
    sees, pos = tree.masks_positions(parents, [n] * B, [3] * B)
    assert not sees.any(-1).all()
    m, p = _api().draft_tree(_i32(parents), start=_i32([3] * B))
    assert np.array_equal(m.cpu().numpy(), tree.pack(sees)) and np.array_equal(p[0].cpu().numpy(), pos)
    e, x = _api().draft_tree(_i32(parents)[:, :0])
    assert e.shape == (B, 0, 0) and x.shape == (1, B, 0)
    for bad in (dict(count=_i32([1])), dict(start=_i32([1] * B).long()), dict(masks=m[:, :, :1]), dict(positions=p[0])):
        with pytest.raises(ValueError):
            _api().draft_tree(_i32(parents), **bad)


# ---- attention

def _check(out, want, spread, reach, T, d, dtype, wide, least=0.0):
    two = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    score = (d + T / 16 + 64) * 2.0 ** -22 * (1 + reach[..., None]) + wide
    tol = spread * (two + 2 * score + (T / 16 + 64) * 2.0 ** -23) + np.abs(want) * _half_step(dtype) + 1e-30
    tol = tol + torch.finfo(dtype).smallest_normal * _half_step(dtype) + least
    got = _np(out)
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1.0, worst


def _terms(q, pool, seq, cnt, table, scale, on):
    """What e4m3 terms of the queries may move a score by, [B][nq][Hq][1]."""
    B, nq, Hq, d = q.shape
    off = np.zeros((B, nq, Hq, 1))
    if on:
        for b in range(B):
            pages = table[b][:(seq[b] + 15) // 16]
            for h in range(pool.heads):
                K = pool.read(0, h, pages, seq[b])
                top = np.abs(K).sum(-1).max() if len(K) else 0.0
                g = slice(h * Hq // pool.heads, (h + 1) * Hq // pool.heads)
                off[b, :, g, 0] = 2.0 ** -18 * np.abs(q[b, :, g]).max(-1) * top * abs(scale)
    return off


def _filled(d, Hq, H, seq, blocks, dtype, seed=0):
    """A cache of the given lengths, whatever lies behind them included, and its table."""
    B = len(seq)
    pages = B * blocks + 3
    c = _cache(d, Hq, H, pages, blocks, seed=seed)
    table = _table(B, blocks, pages, seed=seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 1)
    n = max(max(seq), 1)
    x = torch.randn(2, B, H, n, d, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(2, 1, H, 1, d, generator=g, device="cuda"))
    x = x.to(DT[dtype])
    c.append(x[0], x[1], _i32([0] * B), _i32(table), count=_i32(seq))
    assert c.device_error() == 0
    return c, table, g


def _run(d, dtype, Hq, H, seq, cnt, nq, scale=None, seed=0, bits=0.5, from_tree=False):
    blocks = max(1, (max(seq) + 15) // 16)
    c, table, g = _filled(d, Hq, H, seq, blocks, dtype, seed)
    B, rs = len(seq), np.random.RandomState(seed)
    if from_tree:
        sees, _ = tree.masks_positions(_parents(rs, B, nq, 4), np.minimum(cnt, nq), [0] * B)
        masks = tree.pack(sees)
    else:
        sees = rs.rand(B, nq, nq) < bits
        masks = tree.pack(sees)
        if nq % 32:  # (bits that no draft has)
            masks[..., -1] |= np.int32(-1) << np.int32(nq % 32)
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt), scale=scale, tree=_i32(masks))
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    s = d ** -0.5 if scale is None else scale
    # (least: a weight is an fp16 number below 2^M, M at least 7 under the row's largest, so it has a smallest step of
    # 2^-31 of the largest and is off by half of one.  It shows where the heaviest token's value is 0: all that is left there
    # are weights near the step.)
    want, spread, reach, least = tree.attention(_np(q), pool, seq, cnt, table, s, sees, 2.0 ** -31)
    wide = _terms(_np(q), pool, seq, cnt, table, s, dtype != "f32" and d != 256 and Hq // H * nq > 8)
    _check(out, want, spread, reach, max(seq), d, DT[dtype], wide, least)
    assert c.device_error() == 0
    dead = np.ones(want.shape[:2], dtype=bool)
    for b in range(B):
        dead[b, :max(0, cnt[b])] = False
    assert np.all(_np(out)[dead] == 0)
    assert np.all(_np(out)[spread == 0] == 0)
    return out


SHAPES = [(128, 4, 1, 3), (128, 8, 2, 5), (128, 8, 2, 17), (128, 8, 1, 33), (128, 7, 1, 70), (128, 32, 8, 16), (64, 4, 4, 2), (64, 8, 2, 12),
          (64, 16, 2, 40), (256, 2, 1, 3), (256, 8, 2, 9), (128, 6, 6, 1), (128, 5, 5, 40)]


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,Hq,H,nq", SHAPES)
def test_tree_attention(d, Hq, H, nq, dtype):
    """Any bits; empty sequences, sequences of one token, more drafts than tokens, no drafts, drafts that end at and
    begin beside the borders of blocks and tiles."""
    seq = [0, 1, 16, 127, 128, 129, 300, 515, 513, 40, nq, nq + 1, max(1, nq - 1)]
    cnt = [nq, nq, nq, nq, max(1, nq - 1), nq, 0, nq, 1, -3, nq, nq + 5, nq]
    _run(d, dtype, Hq, H, seq, [min(c, nq) for c in cnt], nq, seed=nq)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", [("bf16", 128, 8, 2, 16), ("f16", 128, 8, 2, 40), ("bf16", 64, 4, 2, 30), ("f32", 128, 4, 2, 7),
                                             ("bf16", 128, 4, 2, 4), ("f16", 256, 4, 2, 6)])
def test_tree_attention_long(dtype, d, Hq, H, nq):
    """Long sequences beside short ones: ranges that split a slab's tokens, and join."""
    _run(d, dtype, Hq, H, [9000, 33, 4097, 0, 6001], [nq, nq, max(1, nq // 2), nq, nq], nq, seed=3, from_tree=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [200, 600])
def test_tree_attention_of_many_drafts(dtype, nq):
    """Drafts that fill several tiles; rows that see none of the drafts of a whole tile, or nothing at all."""
    _run(128, dtype, 4, 2, [nq, nq + 300, 64], [nq, nq - 7, 64], nq, seed=1, bits=0.004)


@pytest.mark.parametrize("dtype,nq", [("bf16", 2), ("bf16", 20), ("f32", 3), ("f16", 70)])
def test_rows_that_see_nothing_are_zeros(dtype, nq):
    c, table, g = _filled(128, 8, 2, [nq, nq - 1], 8, dtype)
    q = torch.randn(2, nq, 8, 128, generator=g, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32([nq, nq - 1]), _i32(table), tree=torch.zeros(2, nq, (nq + 31) // 32, dtype=torch.int32, device="cuda"))
    assert torch.all(out == 0)


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 128, 3), ("bf16", 128, 24), ("f16", 128, 60), ("f32", 128, 9), ("bf16", 64, 24), ("bf16", 256, 9)])
def test_a_chain_is_causal_attention(dtype, d, nq):
    seq, cnt = [700, 1300, 5, 2000], [nq, max(1, nq // 2), min(nq, 5), nq]
    c, table, g = _filled(d, 8, 2, seq, 125, dtype)
    q = torch.randn(4, nq, 8, d, generator=g, device="cuda").to(DT[dtype])
    masks, _ = _api().draft_tree(_i32(np.tile(np.arange(-1, nq - 1), (4, 1))))
    a = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt))
    b = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt), tree=masks)
    # two results of the same formula: each within its bound of it, 2^-9 (2^-20) of values of order 1 by the roundings above
    step = 2.0 ** -16 if dtype == "f32" else 2.0 ** -6 if dtype == "bf16" else 2.0 ** -8
    assert (a.double() - b.double()).abs().max() <= step * float(a.double().abs().max())


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 128, 20), ("f16", 64, 20), ("f32", 128, 4), ("bf16", 128, 80), ("bf16", 256, 3)])
def test_unlike_scales_and_odd_queries(dtype, d, nq):
    """Value blocks of very unlike scales; a query row with an infinity or a NaN is NaN and alone; what rows past the
    count hold reaches nothing."""
    seq, cnt = [400, 290], [nq, nq - 1]
    c, table, g = _filled(d, 8, 2, seq, 25, dtype)
    blocks = c.pool.view(-1, 32 * d + 32)
    size = torch.exp2(torch.randint(-9, 6, (blocks.shape[0],), generator=g, device="cuda").float())
    blocks[:, 32 * d + 4:32 * d + 8] = size.view(-1, 1).view(torch.uint8)
    q = torch.randn(2, nq, 8, d, generator=g, device="cuda").to(DT[dtype])
    sees = np.random.RandomState(2).rand(2, nq, nq) < 0.6
    args = _i32(seq), _i32(table)
    plain = c.attention(q, *args, count=_i32(cnt), tree=_i32(tree.pack(sees)))
    pool = ref.Pool(c.pool.cpu().numpy(), 2, d)
    want, spread, reach, least = tree.attention(_np(q), pool, seq, cnt, table, d ** -0.5, sees, 2.0 ** -31)
    wide = _terms(_np(q), pool, seq, cnt, table, d ** -0.5, dtype != "f32" and d != 256 and 4 * nq > 8)
    _check(plain, want, spread, reach, 400, d, DT[dtype], wide, least)
    odd = q.clone()
    odd[0, 1, 3, 5] = float("inf")
    odd[1, 0, 6, 0] = float("nan")
    odd[1, nq - 1] = float("nan")  # past the count
    got = c.attention(odd, *args, count=_i32(cnt), tree=_i32(tree.pack(sees)))
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[0, 1, 3] = bad[1, 0, 6] = True
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], plain[~bad])
    assert torch.all(got[1, nq - 1] == 0)


ROUTES = [("bf16", 128, 8, 2, 2), ("bf16", 128, 8, 2, 12), ("f16", 128, 8, 2, 25), ("bf16", 128, 8, 1, 40), ("bf16", 64, 8, 2, 30),
          ("f16", 64, 4, 2, 6), ("bf16", 256, 8, 2, 5), ("f32", 128, 8, 2, 3), ("f32", 64, 8, 2, 9)]


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
@pytest.mark.parametrize("rise", [0.13, -0.13, 0.5])
def test_maxima_that_rise_and_fall(dtype, d, Hq, H, nq, rise):
    """Scores that grow (fall) by 17 (64) powers of two a tile of 128 tokens: the running reference rises in every tile, and
    the sums so far are rescaled each time."""
    seq, cnt = [1500, 700, 200], [nq, nq, max(1, nq - 1)]
    c, table, g = _filled(d, Hq, H, seq, 94, dtype)
    n, B = max(seq), len(seq)
    u = torch.sign(torch.randn(d, generator=g, device="cuda"))
    level = (torch.arange(n, device="cuda") - n / 2) * rise / 1.4427 / d ** 0.5
    k = level[None, None, :, None] * u + 0.2 * torch.randn(B, H, n, d, generator=g, device="cuda")
    v = torch.randn(B, H, n, d, generator=g, device="cuda")
    c.append(k.to(DT[dtype]), v.to(DT[dtype]), _i32([0] * B), _i32(table), count=_i32(seq))
    q = (u + 0.05 * torch.randn(B, nq, Hq, d, generator=g, device="cuda")).to(DT[dtype])
    sees = np.random.RandomState(1).rand(B, nq, nq) < 0.6
    out = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt), tree=_i32(tree.pack(sees)))
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    want, spread, reach, least = tree.attention(_np(q), pool, seq, cnt, table, d ** -0.5, sees, 2.0 ** -31)
    wide = _terms(_np(q), pool, seq, cnt, table, d ** -0.5, dtype != "f32" and d != 256 and Hq // H * nq > 8)
    _check(out, want, spread, reach, max(seq), d, DT[dtype], wide, least)


MANY = [("bf16", 64, 8, 2, 17), ("bf16", 64, 8, 2, 40), ("f16", 64, 16, 2, 24), ("f16", 128, 8, 1, 24), ("f16", 128, 7, 1, 13), ("bf16", 128, 16, 2, 33)]


@pytest.mark.parametrize("dtype,d,Hq,H,nq", MANY)
def test_more_than_64_rows(dtype, d, Hq, H, nq):
    """Groups of 128 rows, the last one partly filled: long sequences beside short ones, and trees of few drafts beside those of many."""
    _run(d, dtype, Hq, H, [9000, 33, 4097, 0, 6001, 700], [nq, nq, max(1, nq // 2), nq, 1, 0], nq, seed=5, from_tree=True)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", MANY)
@pytest.mark.parametrize("rise", [0.13, -0.13])
def test_maxima_of_more_than_64_rows(dtype, d, Hq, H, nq, rise):
    test_maxima_that_rise_and_fall(dtype, d, Hq, H, nq, rise)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES + MANY)
def test_tables_that_end_with_the_sequence(dtype, d, Hq, H, nq):
    """The longest sequence fills its table and its last tile; others end with a tile or a block before it."""
    _run(d, dtype, Hq, H, [512, 384, 496, 128, 16], [nq, nq, nq, nq, min(nq, 16)], nq, seed=6)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
@pytest.mark.parametrize("scale", [0.0, -0.07, 1e-30, 3.0])
def test_scales_of_the_scores(dtype, d, Hq, H, nq, scale):
    """No scale at all leaves the mean of what a row sees, and hides what it does not."""
    _run(d, dtype, Hq, H, [300, 128, 31], [nq, max(1, nq - 1), min(nq, 31)], nq, scale=scale, seed=2)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
def test_queries_near_the_ends_of_the_range(dtype, d, Hq, H, nq):
    """Rows of 1e-30 (fp16: 1e-7, subnormal) and of zeros attend evenly; rows of 1e4 to what they hit hardest."""
    seq, cnt = [260, 129], [nq, nq]
    c, table, g = _filled(d, Hq, H, seq, 17, dtype)
    q = torch.randn(2, nq, Hq, d, generator=g, device="cuda")
    q[0, 0] *= 1e-7 if dtype == "f16" else 1e-30
    q[0, 1] = 0
    q[1, 0] *= 1e4
    q = q.to(DT[dtype])
    sees = np.random.RandomState(3).rand(2, nq, nq) < 0.6
    out = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt), tree=_i32(tree.pack(sees)))
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    want, spread, reach, least = tree.attention(_np(q), pool, seq, cnt, table, d ** -0.5, sees, 2.0 ** -31)
    wide = _terms(_np(q), pool, seq, cnt, table, d ** -0.5, dtype != "f32" and d != 256 and Hq // H * nq > 8)
    _check(out, want, spread, reach, max(seq), d, DT[dtype], wide, least)


@pytest.mark.parametrize("dtype,d,nq", [("bf16", 128, 6), ("bf16", 128, 20), ("bf16", 64, 12), ("f32", 128, 3), ("bf16", 128, 3)])
def test_a_batch_of_512(dtype, d, nq):
    """The largest batch: most entries short, some empty, some without drafts."""
    rs = np.random.RandomState(nq)
    B, Hq, H = 512, 8, 2
    seq = [int(x) for x in rs.randint(0, 40, B)]
    seq[300], seq[511] = 700, 260
    cnt = [int(x) for x in rs.randint(0, nq + 1, B)]
    c, table, g = _filled(d, Hq, H, seq, 44, dtype)
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    sees = rs.rand(B, nq, nq) < 0.5
    out = c.attention(q, _i32(seq), _i32(table), count=_i32(cnt), tree=_i32(tree.pack(sees)))
    some = [0, 1, 2, 100, 299, 300, 301, 400, 510, 511]
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    pick = lambda x: [x[b] for b in some]  # noqa: E731
    want, spread, reach, least = tree.attention(_np(q)[some], pool, pick(seq), pick(cnt), table[some], d ** -0.5, sees[some])
    wide = _terms(_np(q)[some], pool, pick(seq), pick(cnt), table[some], d ** -0.5, dtype != "f32" and Hq // H * nq > 8)
    _check(out[some], want, spread, reach, 700, d, DT[dtype], wide)
    dead = torch.arange(nq, device="cuda")[None] >= _i32(cnt)[:, None]
    assert torch.all(out[dead] == 0)
    assert torch.all(out[[b for b in range(B) if seq[b] == 0]] == 0) and torch.isfinite(out.float()).all()
    with pytest.raises(_api().TQError):
        c.attention(torch.zeros(513, nq, Hq, d, dtype=DT[dtype], device="cuda"), torch.zeros(513, dtype=torch.int32, device="cuda"),
                    torch.zeros(513, 44, dtype=torch.int32, device="cuda"), tree=torch.zeros(513, nq, 1, dtype=torch.int32, device="cuda"))


def test_strided_queries_one_query_outputs_and_refusals():
    d, nq = 128, 5
    c, table, g = _filled(d, 8, 2, [100, 37], 8, "bf16")
    wide = torch.randn(2, nq, 24, d, generator=g, device="cuda").to(torch.bfloat16)
    q = wide[:, :, 8:16]
    masks, _ = _api().draft_tree(_i32([[-1, 0, 0, 1, 1], [-1, -1, 1, 1, 3]]))
    want = c.attention(q.contiguous(), _i32([100, 37]), _i32(table), tree=masks)
    out = torch.empty_like(want)
    assert c.attention(q, _i32([100, 37]), _i32(table), tree=masks, out=out) is out and torch.equal(out, want)
    one = c.attention(q[:, 0], _i32([100, 37]), _i32(table), tree=masks[:, :1, :1].contiguous())
    assert one.shape == (2, 8, d)
    bare = c.attention(q[:, 0], _i32([100, 37]), _i32(table))
    assert torch.equal(one, bare)  # one draft that sees itself is one token
    for bad in (masks[:1], masks.long(), masks.cpu(), torch.zeros(2, nq, 2, dtype=torch.int32, device="cuda"),
                torch.zeros(2, nq, 2, dtype=torch.int32, device="cuda")[:, :, :1]):
        with pytest.raises(ValueError):
            c.attention(q, _i32([100, 37]), _i32(table), tree=bad)
    with pytest.raises(_api().TQError):
        c.attention(q, _i32([100, 37]), _i32(table), tree=masks, scale=float("inf"))
    empty = c.attention(q[:, :0], _i32([100, 37]), _i32(table), tree=masks[:, :0, :0].contiguous())
    assert empty.shape == (2, 0, 8, d)


def test_bad_pages_and_lengths_reach_only_their_entry():
    for nq in (3, 24):
        c, table, g = _filled(128, 8, 2, [300, 300, 300], 19, "bf16")
        q = torch.randn(3, nq, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
        masks = _i32(np.full((3, nq, 1), -1))
        want = c.attention(q, _i32([300, 300, 300]), _i32(table), tree=masks)
        t = table.copy()
        t[1, 4], t[1, 18] = 1 << 30, -7
        got = c.attention(q, _i32([300, 300, 300]), _i32(t), tree=masks)
        assert c.device_error() == 3  # TQ_DEVERR_BAD_PAGE
        assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
        got = c.attention(q, _i32([300, -5, 300]), _i32(table), tree=masks)
        assert c.device_error() == 4 and torch.all(got[1] == 0) and torch.equal(got[2], want[2])


def test_captured_steps_follow_their_tensors():
    """draft_tree, append, attention, keep and read in one graph: lengths, trees, paths and tables of each replay."""
    tq = _api()
    d, Hq, H, nq, B, blocks = 128, 8, 2, 24, 3, 40
    c, table, g = _filled(d, Hq, H, [60, 333, 16], blocks, "bf16")
    rs = np.random.RandomState(0)
    rot = tq.Rotary(d)
    base, tab = _i32([60, 333, 16]), _i32(table)
    parents, count, seq = _i32(_parents(rs, B, nq, 3)), _i32([nq, 5, 11]), _i32([0] * B)
    path, kept = _i32(np.tile(np.arange(4), (B, 1))), _i32([4, 2, 0])
    other, mine = torch.cuda.Stream(), torch.zeros(B, nq, 1, dtype=torch.int32, device="cuda")
    k, v = (torch.randn(B, H, nq, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(torch.bfloat16)

    def step():
        masks, pos = tq.draft_tree(parents, start=base, count=count)
        qr = c.append(k, v, base, tab, count=count, rotary=rot, positions=pos, q=q)
        # a copy, and work of another stream, right before the attention
        ready = torch.cuda.Event()
        main = torch.cuda.current_stream()
        ready.record()
        with torch.cuda.stream(other):
            other.wait_event(ready)
            torch.add(base, count, out=seq)
        main.wait_stream(other)
        mine.copy_(masks)
        out = c.attention(qr, seq, tab, count=count, tree=mine)
        length = c.keep(path, base, tab, count=kept)
        return out, length, *c.read(base, tab, 4, count=kept, dtype=torch.float32)

    first = c.pool.clone()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for turn in range(3):
        base.copy_(_i32([60 + turn, 333 - 7 * turn, 16 * turn]))
        parents.copy_(_i32(_parents(rs, B, nq, 2 + turn)))
        count.copy_(_i32([nq - turn, 5 + turn, 11]))
        path.copy_(_i32(np.sort(np.stack([rs.permutation(5)[:4] for _ in range(B)]), -1)))
        kept.copy_(_i32([min(4, turn + 1), 4, 3]))
        q.normal_()
        k.normal_()
        c.pool.copy_(first)
        want = [x.clone() for x in step()]
        pool = c.pool.clone()
        c.pool.copy_(first)
        graph.replay()
        # bit by bit: a base past the filled tokens takes what lay there in, NaN codes among it
        for x, y in zip(got, want):
            assert torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
        assert torch.equal(c.pool, pool)
    assert c.device_error() == 0


def test_on_a_stream_and_two_calls_at_once():
    tq = _api()
    nq = 40
    c, table, g = _filled(128, 16, 2, [5000, 4000], 320, "bf16")
    q = torch.randn(2, nq, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    parents = _i32(_parents(np.random.RandomState(1), 2, nq, 4))
    seq, tab = _i32([5000, 4000]), _i32(table)
    want = c.attention(q, seq, tab, tree=tq.draft_tree(parents)[0])
    few = c.attention(q[:, :2], seq, tab, tree=tq.draft_tree(parents[:, :2].contiguous())[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for _ in range(20):
        got = []
        for i, s in enumerate(streams):
            m, _ = tq.draft_tree(parents if i != 1 else parents[:, :2].contiguous(), stream=None if i == 1 else s)
            if i == 1:
                s.wait_stream(torch.cuda.current_stream())
            got.append(c.attention(q if i != 1 else q[:, :2], seq, tab, tree=m, stream=s))
            del m
        torch.cuda.synchronize()
        assert torch.equal(got[0], want) and torch.equal(got[2], want) and torch.equal(got[1], few)


# ---- keep

@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,most", [(1, 1), (7, 4), (40, 12), (100, 60), (1024, 300)])
def test_keep_bytes(d, n, most):
    """Every byte of the pool: scales that differ from block to block, codes at the ends of their range."""
    rs = np.random.RandomState(n + d)
    B, H, blocks = 4, 3, (n + 40) // 16 + 2
    pages = B * blocks + 2
    c = _cache(d, H, H, pages, blocks, seed=n)
    pool = c.pool.cpu().numpy().reshape(-1, H, 32 * d + 32)
    pool[..., :32 * d][(pool[..., :32 * d] & 127) == 127] = 126
    scale = (2.0 ** rs.randint(-30, 31, pool.shape[:2] + (2,))).astype(np.float32)
    near = rs.rand(*scale.shape) < 0.7
    scale[near] = (2.0 ** rs.randint(-3, 4, scale.shape).astype(np.float32))[near]
    pool[..., 32 * d:32 * d + 8] = scale.view(np.uint8)
    c.pool.copy_(torch.from_numpy(pool.reshape(-1)).cuda())
    table = _table(B, blocks, pages, seed=d)
    want = ref.Pool(pool, H, d)
    start = rs.randint(0, 33, B)
    path = np.stack([np.sort(rs.permutation(n)[:most]) for _ in range(B)]).astype(np.int32)
    path[1] = np.arange(most)                      # all where they are
    cnt = [most, most, rs.randint(0, most + 1), most + 9]
    tree.keep(want, path, start, cnt, table)
    length = c.keep(_i32(path), _i32(start), _i32(table), count=_i32(cnt))
    assert length.cpu().tolist() == [int(s) + min(k, most) for s, k in zip(start, cnt)]
    assert np.array_equal(c.pool.cpu().numpy().reshape(want.blocks.shape), want.blocks)
    assert c.device_error() == 0


def test_keep_with_paths_that_do_not_rise():
    """An entry with a bad path stays, the others do not mind; so does one whose path rises up to its count."""
    d, H, blocks = 128, 2, 6
    paths = [[1, 2, 2], [-1, 3, 4], [3, 2, 4], [1, 3, -7], [0, 5, 9], [2, 4, 6], [1, 2, 3]]
    cnt, start = [3, 3, 3, 2, 3, -4, 3], [5, 5, 5, 5, 5, 9, -3]
    B = len(paths)
    c, table, _ = _filled(d, 2, H, [60] * B, blocks, "bf16")
    want = ref.Pool(c.pool.cpu().numpy(), H, d)
    tree.keep(want, np.array(paths), start, cnt, table)
    mine = _i32([77] * B)
    got = c.keep(_i32(paths), _i32(start), _i32(table), count=_i32(cnt), seq_len=mine)
    assert got is mine and got.cpu().tolist() == [5, 5, 5, 7, 8, 9, -3]
    assert np.array_equal(c.pool.cpu().numpy().reshape(want.blocks.shape), want.blocks)
    assert c.device_error() == 6  # TQ_DEVERR_BAD_PATH
    assert c.device_error() == 0
    # a path out of the table, and bad pages: nothing outside the pool, and the other entries are right
    t = table.copy()
    t[0, 1] = 1 << 29
    want = ref.Pool(c.pool.cpu().numpy(), H, d)
    tree.keep(want, np.array([[0, 4, 8]]), [5], [3], table[4:5])
    c.keep(_i32([[20, 30, 2147483647], [0, 4, 8]]), _i32([5, 5]), _i32(np.stack([t[0], table[4]])))
    assert c.device_error() == 3
    own = table[4]
    assert np.array_equal(c.pool.cpu().numpy().reshape(want.blocks.shape)[own], want.blocks[own])
    assert c.keep(_i32(np.zeros((2, 0))), _i32([5, 6]), _i32(table[:2])).cpu().tolist() == [5, 6]
    for bad in (dict(count=_i32([1])), dict(seq_len=_i32([1, 2, 3]))):
        with pytest.raises(ValueError):
            c.keep(_i32([[0], [0]]), _i32([5, 6]), _i32(table[:2]), **bad)


# ---- read

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_read(d, dtype):
    H, seq, blocks, n = 3, [130, 200, 17, 5], 14, 75
    c, table, _ = _filled(d, H, H, seq, blocks, dtype)
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    start, cnt = [0, 125, 16, 1], [n, n + 20, 1, -2]
    got = c.read(_i32(start), _i32(table), n, count=_i32(cnt), dtype=DT[dtype])
    for x, y in zip(got, tree.read(pool, start, cnt, n, table)):
        assert x.shape == (4, H, n, d) and x.is_contiguous() and x.dtype == DT[dtype]
        assert torch.equal(x, torch.from_numpy(y).to(DT[dtype]).cuda())
    # the default type and count, one token, none, the caller's outputs
    k, v = c.read(_i32([3, 3]), _i32(table[:2]), 1)
    want = tree.read(pool, [3, 3], [1, 1], 1, table)
    assert k.dtype == torch.bfloat16 and np.array_equal(_np(k), want[0]) and np.array_equal(_np(v), want[1])
    assert c.read(_i32([3, 3]), _i32(table[:2]), 0)[0].shape == (2, H, 0, d)
    mine = torch.empty(2, 2, H, 1, d, device="cuda")
    k, v = c.read(_i32([3, 3]), _i32(table[:2]), 1, dtype=torch.float32, k_out=mine[0], v_out=mine[1])
    assert np.array_equal(_np(mine[0]), want[0]) and np.array_equal(_np(mine[1]), want[1])
    assert c.device_error() == 0
    with pytest.raises(ValueError):
        c.read(_i32([3, 3]), _i32(table[:2]), 1, dtype=torch.float32, k_out=mine[0].double())
    with pytest.raises(ValueError):
        c.read(_i32([3, 3]), _i32(table[:2]), 1, dtype=torch.int32)
    with pytest.raises(_api().TQError):
        c.read(_i32([3, 3]), _i32(table[:2]), 1, dtype=torch.float32, k_out=mine[0], v_out=mine[0])


def test_read_out_of_range_values_and_positions():
    d, H = 128, 2
    c, table, _ = _filled(d, H, H, [32], 2, "f32")
    c.pool.view(-1, 32 * d + 32)[:, 32 * d:32 * d + 4] = torch.tensor([2.0 ** 30], device="cuda").view(torch.uint8)
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    k, v = c.read(_i32([0]), _i32(table), 32, dtype=torch.float16)
    want = torch.from_numpy(tree.read(pool, [0], [32], 32, table)[0]).to(torch.float16)  # infinities, as torch rounds
    assert torch.isinf(want).any() and torch.equal(k.cpu(), want)
    # positions before 0 and past the table read the extra page; those inside are right
    k, v = c.read(_i32([-5]), _i32(table), 45, dtype=torch.float32)
    assert c.device_error() == 3
    assert np.array_equal(_np(k[0, :, 5:37]), tree.read(pool, [0], [32], 32, table)[0][0])


def test_read_moves_a_cache():
    """What is read in 32 bits and appended to another cache gives the same values: codes of one scale stay codes."""
    d, H, n = 128, 2, 50
    c, table, _ = _filled(d, H, H, [n, 33], 4, "bf16")
    k, v = c.read(_i32([0, 0]), _i32(table), n, count=_i32([n, 33]), dtype=torch.float32)
    other = _cache(d, H, H, 9, 4, garbage=False)
    t = np.arange(8).reshape(2, 4)
    other.append(k, v, _i32([0, 0]), _i32(t), count=_i32([n, 33]))
    a = c.read(_i32([0, 0]), _i32(table), n, count=_i32([n, 33]), dtype=torch.float32)
    b = other.read(_i32([0, 0]), _i32(t), n, count=_i32([n, 33]), dtype=torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ---- together, and far into a pool

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_steps_of_a_drafted_decode(dtype):
    """Steps of append, attention and keep: the outputs of each against the definition on the pool as it then is, and
    the pool's bytes after each keep."""
    tq = _api()
    d, Hq, H, nq, B, blocks = 128, 8, 2, 12, 3, 12
    rs = np.random.RandomState(4)
    base = [37, 0, 95]
    c, table, g = _filled(d, Hq, H, base, blocks, dtype)
    rot = tq.Rotary(d)
    tab = _i32(table)
    for step in range(4):
        cnt = [nq, rs.randint(1, nq + 1), nq]
        parents = _parents(rs, B, nq, 3)
        sees, pos = tree.masks_positions(parents, cnt, base)
        masks, positions = tq.draft_tree(_i32(parents), start=_i32(base), count=_i32(cnt))
        assert np.array_equal(positions[0].cpu().numpy(), pos)
        k, v = (torch.randn(B, H, nq, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
        q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
        qr = c.append(k, v, _i32(base), tab, count=_i32(cnt), rotary=rot, positions=positions, q=q)
        seq = [x + y for x, y in zip(base, cnt)]
        out = c.attention(qr, _i32(seq), tab, count=_i32(cnt), tree=masks)
        pool = ref.Pool(c.pool.cpu().numpy(), H, d)
        want, spread, reach, least = tree.attention(_np(qr), pool, seq, cnt, table, d ** -0.5, sees)
        _check(out, want, spread, reach, max(seq), d, DT[dtype], _terms(_np(qr), pool, seq, cnt, table, d ** -0.5, dtype != "f32"))
        # the path to the deepest draft
        path, kept = np.zeros((B, nq), dtype=np.int32), []
        for b in range(B):
            leaf = int(np.argmax(pos[b, :cnt[b]]))
            way = np.flatnonzero(sees[b, leaf])
            path[b, :len(way)] = way
            kept.append(len(way))
        tree.keep(pool, path, base, kept, table)
        length = c.keep(_i32(path), _i32(base), tab, count=_i32(kept))
        base = [x + y for x, y in zip(base, kept)]
        assert length.cpu().tolist() == base
        assert np.array_equal(c.pool.cpu().numpy().reshape(pool.blocks.shape), pool.blocks)
    assert c.device_error() == 0


def test_pages_past_32_bits():
    """Blocks whose byte offsets pass 2^32."""
    d, H, blocks = 256, 8, 4
    pages = (1 << 32) // (H * (32 * d + 32)) + 10
    c = _api().PagedByteCache(d, H, H, pages, blocks)
    low = _api().PagedByteCache(d, H, H, 10, blocks)
    t = np.array([[pages - 1, 1, pages - 3, 0]])
    u = np.array([[0, 1, 2, 3]])
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    k, v = (torch.randn(1, H, 60, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(1, 9, H, d, generator=g, device="cuda").to(torch.bfloat16)
    masks, _ = _api().draft_tree(_i32([[-1, 0, 0, 1, 1, 2, 3, 3, 4]]))
    got = []
    for x, tab in ((c, _i32(t)), (low, _i32(u))):
        x.append(k, v, _i32([0]), tab)
        a = x.attention(q, _i32([60]), tab, tree=masks)
        x.keep(_i32([[0, 1, 4, 8]]), _i32([51]), tab)
        got.append((a, *x.read(_i32([0]), tab, 60)))
        assert x.device_error() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
