"""What a tree's masks hide reaches nothing, whatever lies there: against the definition on the visible tokens alone.

Tolerances: as in test_gpu_tree.py, whose comments derive them."""

import numpy as np
import pytest
import torch

import byte_reference as ref
import tree_reference as tree
from test_gpu_byte_cache import DT, _api, _i32, _np, _table
from test_gpu_tree import _check, _terms

pytestmark = pytest.mark.gpu

# up to 8 rows, 9 to 64 and more at head dims 64 and 128, the other kernel's types and head dim
ROUTES = [("bf16", 128, 4, 2, 2), ("bf16", 128, 4, 2, 20), ("f16", 128, 8, 2, 40), ("bf16", 64, 4, 2, 20), ("f16", 64, 8, 2, 40),
          ("f32", 128, 4, 2, 20), ("bf16", 256, 4, 2, 20)]


def _prompt(d, Hq, H, seq, blocks, dtype, zeroed=True):
    """A cache whose first seq[b] tokens were appended, into a pool that was zeroed, or held anything, before."""
    B = len(seq)
    pages = B * blocks + 1
    c = _api().PagedByteCache(d, Hq, H, pages, blocks)
    g = torch.Generator(device="cuda")
    g.manual_seed(d + Hq)
    if not zeroed:
        c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
    table = _table(B, blocks, pages, seed=d)
    k, v = (torch.randn(B, H, max(seq), d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    c.append(k, v, _i32([0] * B), _i32(table), count=_i32(seq))
    assert c.device_error() == 0
    return c, table, g


def _by_definition(c, table, q, seq, there, H, d, dtype, sees):
    """Values and bounds by the definition; the first there[b] tokens were appended and what lies behind them is hidden (put
    to zeros here: the reference reads it and gives it no weight)."""
    n, Hq = q.shape[1:3]
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    lens, cnt = [s + n for s in seq], [n] * len(seq)
    for b, s in enumerate(there):
        for t in range(s, lens[b]):
            for h in range(H):
                for side in (0, 1):
                    pool.blocks[table[b][t // 16], h][pool.at[side, t % 16]] = 0
                    if t % 16 == 0:
                        pool.set_scale(table[b][t // 16], h, side, 0)
    want, spread, reach, least = tree.attention(_np(q), pool, lens, cnt, table, d ** -0.5, sees, 2.0 ** -31)
    wide = _terms(_np(q), pool, lens, cnt, table, d ** -0.5, dtype != "f32" and d != 256 and Hq // H * n > 8)
    return want, spread, reach, least, wide


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
@pytest.mark.parametrize("seq", [[96, 128, 37], [256, 16, 1]])
def test_hidden_drafts_that_were_never_appended(dtype, d, Hq, H, nq, seq):
    """The drafts' blocks are as a zeroed pool has them, scales of 0 among them."""
    blocks = (max(seq) + nq + 15) // 16
    c, table, g = _prompt(d, Hq, H, seq, blocks, dtype)
    q = torch.randn(len(seq), nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    sees = np.zeros((len(seq), nq, nq), dtype=bool)
    out = c.attention(q, _i32([s + nq for s in seq]), _i32(table), tree=_i32(tree.pack(sees)))
    want, spread, reach, least, wide = _by_definition(c, table, q, seq, seq, H, d, dtype, sees)
    _check(out, want, spread, reach, max(seq) + nq, d, DT[dtype], wide, least)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
@pytest.mark.parametrize("odd", [float("inf"), -float("inf"), float("nan")])
def test_odd_queries_of_rows_that_see_nothing(dtype, d, Hq, H, nq, odd):
    """Rows that attend to nothing are zeros whatever their queries hold; the same queries are NaN where they attend to a
    token, and no other row minds."""
    seq = [nq, 200 + nq, 130]
    c, table, g = _prompt(d, Hq, H, seq, 17, dtype)
    q = torch.randn(3, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    sees = np.zeros((3, nq, nq), dtype=bool)
    sees[0, nq // 2:, 0] = True   # the first entry has no tokens before its drafts
    args = _i32(seq), _i32(table)
    clean = c.attention(q, *args, tree=_i32(tree.pack(sees)))
    hit = torch.zeros(3, nq, Hq, dtype=torch.bool, device="cuda")
    hit[:, 0, 1] = hit[:, nq - 1, Hq - 1] = True
    q[..., 3] = torch.where(hit, torch.full_like(q[..., 3], odd), q[..., 3])
    out = c.attention(q, *args, tree=_i32(tree.pack(sees)))
    blind = torch.zeros_like(hit)
    blind[0, :nq // 2] = True
    assert not out[blind].any()
    assert torch.isnan(out[hit & ~blind]).all()
    assert torch.equal(out[~hit], clean[~hit]) and torch.isfinite(clean.float()).all()


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES)
@pytest.mark.parametrize("seq", [[96, 128, 37], [256, 15, 1]])
def test_hidden_drafts_of_a_pool_that_held_anything(dtype, d, Hq, H, nq, seq):
    """The same where the pool held NaN codes and senseless scales before; a draft that was appended is visible among them."""
    blocks = (max(seq) + nq + 15) // 16
    c, table, g = _prompt(d, Hq, H, seq, blocks, dtype, zeroed=False)
    B = len(seq)
    k, v = (torch.randn(B, H, 1, d, generator=g, device="cuda").to(DT[dtype]) for _ in range(2))
    c.append(k, v, _i32(seq), _i32(table))
    q = torch.randn(B, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    sees = np.zeros((B, nq, nq), dtype=bool)
    sees[:, ::2, 0] = True
    out = c.attention(q, _i32([s + nq for s in seq]), _i32(table), tree=_i32(tree.pack(sees)))
    want, spread, reach, least, wide = _by_definition(c, table, q, seq, [s + 1 for s in seq], H, d, dtype, sees)
    _check(out, want, spread, reach, max(seq) + nq, d, DT[dtype], wide, least)


@pytest.mark.parametrize("dtype,d,Hq,H,nq", ROUTES + [("f32", 64, 4, 1, 40), ("f16", 256, 8, 1, 30), ("bf16", 128, 8, 1, 60), ("f16", 64, 8, 1, 60)])
def test_rows_past_the_count_beside_drafts_that_were_never_appended(dtype, d, Hq, H, nq):
    """Groups of rows of which none asks, in sequences that are shared out and joined: zeros, whatever the drafts' places hold."""
    seq, cnt = [4010, 3001, 5005], [max(1, nq // 2), nq, max(1, nq // 3)]  # (drafts on both sides of a block's end)
    blocks = (max(seq) + nq + 15) // 16
    c, table, g = _prompt(d, Hq, H, seq, blocks, dtype, zeroed=False)
    q = torch.randn(3, nq, Hq, d, generator=g, device="cuda").to(DT[dtype])
    none = torch.zeros(3, nq, (nq + 31) // 32, dtype=torch.int32, device="cuda")
    out = c.attention(q, _i32([s + k for s, k in zip(seq, cnt)]), _i32(table), count=_i32(cnt), tree=none)
    for b in range(3):
        assert not out[b, cnt[b]:].any()
        assert torch.isfinite(out[b, :cnt[b]].float()).all() and out[b, :cnt[b]].any()
