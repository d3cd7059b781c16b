"""Byte cache, head norms and position rotation on the GPU against their float64 forms.

Tolerances are bounds from the arithmetic:
* rotation: the angle is off by at most 2^-22 (fp32 fraction of a turn, sincospi's 2 ulp); the norm's
  factor by 2^-22 (rsqrt) + 14 2^-24 (fp32 sums of at most 21 steps halved, three products).  A
  coordinate is off by at most 2^-19 (|a| + |b|) of its pair, and half a step of its type.
* attention: a probability is off by its fp16 rounding (2^-11; fp32 inputs: two terms, 2^-22) and by
  twice the score's error, which is at most (d + T / 16 + 64) 2^-22 of the row's largest
  scale sum |q||k| (fp32 sums, the log2(e) product, ex2 and the join of the parts); sums of
  probabilities and values add (T / 16 + 64) 2^-23.  All of it is relative to sum p |v| / sum p.
"""

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


def _half_step(dtype):
    return torch.finfo(dtype).eps / 2


def _table(B, blocks, pages, seed=0):
    order = np.random.RandomState(seed).permutation(pages)[:B * blocks].reshape(B, blocks)
    return order.astype(np.int32)


def _cache(d, hq, hkv, pages, blocks, seed=0, garbage=True):
    c = _api().PagedByteCache(d, hq, hkv, pages, blocks)
    if garbage:  # anything at all, NaN codes and senseless scales among it
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        c.pool.copy_(torch.randint(0, 256, c.pool.shape, generator=g, device="cuda", dtype=torch.uint8))
    return c


def _check_attention(out, want, spread, reach, T, d, dtype, least=0.0):
    two = 2.0 ** -22 if dtype == torch.float32 else 2.0 ** -11
    score = (d + T / 16 + 64) * 2.0 ** -22 * (1 + reach[..., None])
    tol = spread * (two + 2 * score + (T / 16 + 64) * 2.0 ** -23) + np.abs(want) * _half_step(dtype) + 1e-30
    # the output's own type: below its smallest normal value it has equal steps, eps * smallest_normal (fp16:
    # 2^-24), so that rounding is off by up to half of one (2^-25) and not by half an eps of the value
    tol = tol + torch.finfo(dtype).smallest_normal * _half_step(dtype) + least
    got = _np(out)
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - want) / tol)
    assert worst <= 1.0, worst


# ---- norm and rotation

@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("d,r,inter,axes", [(64, 64, False, 1), (64, 32, True, 3), (128, 128, True, 1), (128, 64, False, 2),
                                            (256, 256, False, 1), (256, 16, True, 1), (512, 512, False, 4), (128, 0, False, 1)])
@pytest.mark.parametrize("B,n,Hq,Hk,norm", [(1, 1, 4, 1, True), (3, 37, 5, 2, False), (2, 300, 7, 7, True)])
def test_norm_rotate(dtype, out, d, r, inter, axes, B, n, Hq, Hk, norm):
    tq = _api()
    g = torch.Generator(device="cuda")
    g.manual_seed(d + n)
    dt = DT[dtype]
    qkv = torch.randn(B, n, Hq + 2 * Hk, d, generator=g, device="cuda").to(dt)
    q, k = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hk].transpose(1, 2)
    wq = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if norm else None
    wk = (1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dt) if norm else None
    freqs = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    axis_of = [i % axes for i in range(r // 2)]
    rot = tq.Rotary(r, axes=axis_of, interleaved=inter) if r else None
    pos = np.random.RandomState(n).randint(-5, 1 << 20, (axes, B, n)).astype(np.int32)
    qo, ko = tq.norm_rotate(q, k, rotary=rot, positions=_i32(pos) if r else None, q_weight=wq, k_weight=wk, out_dtype=DT[out])
    assert qo.is_contiguous() and ko.is_contiguous() and qo.dtype == DT[out] and ko.shape == k.shape
    for b in range(B):
        for x, w, y, to in ((q[b].transpose(0, 1), wq, qo[b].transpose(0, 1), "q"), (k[b], wk, ko[b], "k")):
            want, size = ref.norm_rotate(_np(x), _np(w) if norm else None, 1e-6, freqs if r else None, axis_of, inter, pos[:, b])
            tol = 2.0 ** -19 * size + np.abs(want) * _half_step(DT[out]) + 2.0 ** -25
            assert np.all(np.abs(_np(y) - want) <= tol), to


def test_norm_rotate_starts_in_place_and_sides():
    tq = _api()
    B, n, H, d = 2, 5, 3, 128
    q = torch.randn(B, n, H, d, device="cuda")
    rot = tq.Rotary(d)
    start = np.array([7, 1 << 30], dtype=np.int32)
    pos = (start[:, None] + np.arange(n)).astype(np.int32)[None]
    a, none = tq.norm_rotate(q, rotary=rot, positions=_i32(pos))
    assert none is None
    b, _ = tq.norm_rotate(q, rotary=rot, start=_i32(start))
    assert torch.equal(a, b)
    # zero position, no norm: the values themselves
    z, _ = tq.norm_rotate(q, rotary=rot, positions=torch.zeros(1, B, n, dtype=torch.int32, device="cuda"))
    assert torch.equal(z, q)
    # in place, and keys alone in their own layout
    same = q.clone()
    got, _ = tq.norm_rotate(same, rotary=rot, start=_i32(start), q_out=same)
    assert got is same and torch.equal(same, a)
    with pytest.raises(tq.TQError):
        tq.norm_rotate(same[:, :, 1:], rotary=rot, q_out=same.view(-1)[:B * n * 2 * d].view(B, n, 2, d))
    _, k = tq.norm_rotate(None, q.transpose(1, 2), rotary=rot, start=_i32(start))
    assert torch.equal(k, a.transpose(1, 2))
    # no tokens
    e, _ = tq.norm_rotate(q[:, :0], rotary=rot)
    assert e.shape == (B, 0, H, d)


# ---- append

@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("steps", [[1] * 20, [5, 1, 33, 16, 1, 2], [16, 48, 15, 17], [100]])
def test_append_bytes(d, dtype, steps):
    """Without norm and rotation nothing is rounded before the codes: the pool's bytes are those of the
    definition, those behind the appended tokens included."""
    B, H, blocks, pages = 2, 3, 8, 20
    c = _cache(d, 6, H, pages, blocks, seed=d)
    table = _table(B, blocks, pages, seed=1)
    want = ref.Pool(c.pool.cpu().numpy(), H, d)
    rs = np.random.RandomState(len(steps))
    at = np.array([0, 0])
    first = True
    for n in steps:
        # magnitudes that rise and fall, so that scales rise inside blocks
        size = 2.0 ** rs.uniform(-6, 6, (2, B, H, n, 1))
        x = torch.from_numpy(rs.randn(2, B, H, n, d) * size).to(DT[dtype]).cuda()
        if first:
            x[0, 0, 0, 0, :4] = torch.tensor([0.0, -0.0, 1e-9, 448.0], device="cuda").to(DT[dtype])
            first = False
        start = _i32(at.tolist())
        c.append(x[0], x[1], start, _i32(table))
        for side in (0, 1):
            want.append(side, _np(x[side]), at.tolist(), table)
        at += n
    got = c.pool.cpu().numpy().reshape(want.blocks.shape)
    assert np.array_equal(got, want.blocks)
    assert c.device_error() == 0


def test_append_counts_and_offsets():
    d, B, H, n, blocks, pages = 128, 4, 2, 20, 5, 24
    c = _cache(d, 2, H, pages, blocks)
    table = _table(B, blocks, pages)
    want = ref.Pool(c.pool.cpu().numpy(), H, d)
    x = torch.randn(2, B, n, H, d, device="cuda").to(torch.bfloat16).transpose(2, 3)
    zero = [0, 0, 0, 0]
    head = torch.randn(2, B, H, 13, d, device="cuda").to(torch.bfloat16)
    c.append(head[0], head[1], _i32(zero), _i32(table))
    start, count = [0, 13, 5, 13], [0, 20, 3, -2]
    c.append(x[0], x[1], _i32(start), _i32(table), count=_i32(count))
    for side in (0, 1):
        want.append(side, _np(head[side]), zero, table)
        want.append(side, _np(x[side]), start, table, count)
    assert np.array_equal(c.pool.cpu().numpy().reshape(want.blocks.shape), want.blocks)
    for bb, kvh in ((1, 1), (2, 0)):
        k, v = c.dequantize(bb, kvh, 0, start[bb] + max(0, count[bb]), _i32(table))
        for side, got in ((0, k), (1, v)):
            assert np.array_equal(_np(got), want.read(side, kvh, table[bb], len(got)))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,r,inter,norm,n,start", [(128, 128, False, True, 37, 11), (128, 64, True, True, 1, 15),
                                                    (64, 64, False, False, 70, 0), (256, 256, True, True, 18, 30),
                                                    (256, 128, False, False, 1, 16)])
def test_append_rotates_keys_and_queries(dtype, d, r, inter, norm, n, start):
    tq = _api()
    B, H, Hq, pages, blocks = 2, 5, 10, 40, 10
    dt = DT[dtype]
    c = _cache(d, Hq, H, pages, blocks, garbage=False)
    table = _table(B, blocks, pages)
    qkv = torch.randn(B, n, Hq + 2 * H, d, device="cuda").to(dt)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + H].transpose(1, 2), qkv[:, :, Hq + H:].transpose(1, 2)
    wq, wk = ((1 + 0.2 * torch.randn(d, device="cuda")).to(dt) if norm else None for _ in range(2))
    rot = tq.Rotary(r, interleaved=inter)
    st = [start, start + 3]
    if start:  # earlier tokens, small ones, so that the blocks' scales rise
        pre = torch.randn(B, H, start + 3, d, device="cuda").to(dt) * 0.01
        c.append(pre, pre, _i32([0, 0]), _i32(table))
    qo = c.append(k, v, _i32(st), _i32(table), rotary=rot, k_weight=wk, q=q, q_weight=wq)
    both = tq.norm_rotate(q, k, rotary=rot, start=_i32(st), q_weight=wq, k_weight=wk, out_dtype=dt)
    assert torch.equal(qo, both[0])
    freqs = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    for b in range(B):
        pos = (st[b] + np.arange(n))[None]
        want, size = ref.norm_rotate(_np(k[b]), _np(wk) if norm else None, 1e-6, freqs, [0] * (r // 2), inter, pos)
        for h in range(H):
            got = pool.read(0, h, table[b], st[b] + n)[st[b]:]
            page_scale = np.array([pool.scale(table[b][t // 16], h, 0) for t in range(st[b], st[b] + n)])[:, None]
            # half an e4m3 step, normal (2^-4) or subnormal (2^-10 of the scale); a scale is at most twice its need
            tol = np.maximum(2.0 ** -4 * np.abs(want[h]), 2.0 ** -10 * page_scale) * (1 + 2.0 ** -10) + 2.0 ** -18 * size[h]
            assert np.all(np.abs(got - want[h]) <= tol)
            assert np.all(page_scale <= 2.0 ** np.ceil(np.log2(np.abs(want[h]).max() * 1.001 / 448) + 1e-9) * 1.0 + 0)
            gv = pool.read(1, h, table[b], st[b] + n)[st[b]:]
            vs = np.array([pool.scale(table[b][t // 16], h, 1) for t in range(st[b], st[b] + n)])[:, None]
            assert np.array_equal(gv, ref.VALUES[ref.e4m3_encode(_np(v[b, h]) / vs)] * vs)
    assert c.device_error() == 0


def test_append_reports():
    b = _api().binding
    d, B, H, pages, blocks = 64, 3, 2, 6, 2
    x = torch.randn(B, H, 4, d, device="cuda")
    table = np.array([[0, 1], [2, 3], [4, 99]], dtype=np.int32)
    c = _cache(d, 2, H, pages, blocks, garbage=False)
    c.append(x, x, _i32([0, 0, 16]), _i32(table))           # a page outside the pool
    assert c.device_error() == b.TQ_DEVERR_BAD_PAGE
    c.append(x, x, _i32([0, 30, 0]), _i32(table))           # positions behind the table
    assert c.device_error() == b.TQ_DEVERR_BAD_PAGE
    before = c.pool.clone()
    c.append(x, x, _i32([-100, -100, -100]), _i32(table))   # positions before it
    assert c.device_error() == b.TQ_DEVERR_BAD_PAGE
    used = pages * H * c.block_bytes
    assert torch.equal(before[:used], c.pool[:used])        # only the redirect page took them
    y = x.clone()
    y[1, 0, 2, 5], y[1, 0, 3, 6], y[1, 0, 1, 7] = float("inf"), float("nan"), -float("inf")
    c.append(y, x, _i32([0, 0, 0]), _i32(table))
    assert c.device_error() == b.TQ_DEVERR_NONFINITE
    k, _ = c.dequantize(1, 0, 0, 4, _i32(table))
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    s = pool.scale(2, 0, 0)
    assert s == 2.0 ** ref.need(float(x[1, 0].abs()[torch.isfinite(y[1, 0])].max()))
    assert k[2, 5] == 448 * s and k[3, 6] == 0 and k[1, 7] == -448 * s
    assert torch.isfinite(k).all()


# ---- attention

def _filled(d, hq, hkv, lens, dtype, seed, spread=1.0, extra=2):
    B, top = len(lens), max(max(lens), 1)
    blocks = (top + 15) // 16 + 1
    pages = B * blocks + extra
    c = _cache(d, hq, hkv, pages, blocks, seed=seed)
    table = _table(B, blocks, pages, seed=seed)
    rs = np.random.RandomState(seed)
    chan = 2.0 ** rs.uniform(-spread, spread, (2, hkv, 1, d))
    x = torch.from_numpy(rs.randn(2, B, hkv, top, d) * chan[:, None]).to(dtype).cuda()
    c.append(x[0], x[1], _i32([0] * B), _i32(table), count=_i32(lens))
    assert c.device_error() == 0
    return c, table, ref.Pool(c.pool.cpu().numpy(), hkv, d)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv,nq", [(4, 4, 1), (8, 1, 1), (7, 1, 1), (8, 2, 3), (32, 2, 1), (6, 2, 11), (4, 1, 40), (71, 1, 1),
                                       (130, 1, 1)])
def test_attention(dtype, d, hq, hkv, nq):
    lens = [0, 1, 15, 16, 17, 300, nq, 95]
    c, table, pool = _filled(d, hq, hkv, lens, DT[dtype], seed=d + nq)
    B = len(lens)
    q = torch.randn(B, nq, hq, d, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32(lens), _i32(table))
    want, spread, reach = ref.attention(_np(q), pool, lens, [nq] * B, table, d ** -0.5)
    _check_attention(out, want, spread, reach, max(lens), d, DT[dtype])
    assert torch.equal(out, c.attention(q, _i32(lens), _i32(table)))
    assert c.device_error() == 0


@pytest.mark.parametrize("dtype,d,hq,hkv,nq", [("bf16", 128, 8, 2, 200), ("f16", 128, 8, 2, 200), ("f32", 128, 4, 2, 150),
                                               ("bf16", 64, 4, 1, 260), ("f16", 256, 3, 3, 130), ("bf16", 128, 5, 1, 77),
                                               ("f32", 256, 2, 1, 90), ("f16", 128, 1, 1, 333), ("bf16", 128, 16, 1, 64)])
def test_attention_chunks(dtype, d, hq, hkv, nq):
    lens = [nq, 500, 50, 1, 0, 257]
    count = [nq, nq, 50, 1, nq, 31]
    c, table, pool = _filled(d, hq, hkv, lens, DT[dtype], seed=nq)
    B = len(lens)
    # queries out of a fused projection
    q = torch.randn(B, nq, 3, hq, d, device="cuda").to(DT[dtype])[:, :, 1]
    for cnt in (None, count):
        out = c.attention(q, _i32(lens), _i32(table), count=None if cnt is None else _i32(cnt))
        want, spread, reach = ref.attention(_np(q), pool, lens, cnt or [nq] * B, table, d ** -0.5)
        _check_attention(out, want, spread, reach, max(lens), d, DT[dtype])
        dead = np.arange(nq)[None] >= np.array(cnt or [nq] * B)[:, None]
        assert not _np(out)[dead].any()
    assert torch.equal(out, c.attention(q, _i32(lens), _i32(table), count=_i32(count)))
    assert c.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("hq,hkv,nq,lens,count", [
    (8, 2, 32, [32, 1000, 129], None), (8, 2, 33, [33, 4000, 128], [33, 20, 0]), (6, 2, 128, [128, 127, 300], [128, 100, 1]),
    (4, 4, 300, [300, 2000, 301], None), (16, 1, 50, [777, 64, 50], [50, 7, 50]), (3, 1, 400, [400], None)])
def test_attention_row_groups(dtype, hq, hkv, nq, lens, count):
    """Row groups that end inside a block's rows, ranges that end inside a group's tokens."""
    c, table, pool = _filled(128, hq, hkv, lens, DT[dtype], seed=nq + 1)
    B = len(lens)
    q = torch.randn(B, nq, hq, 128, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32(lens), _i32(table), count=None if count is None else _i32(count))
    cnt = count or [nq] * B
    want, spread, reach = ref.attention(_np(q), pool, lens, cnt, table, 128 ** -0.5)
    _check_attention(out, want, spread, reach, max(lens), 128, DT[dtype])
    # a negative and a zero scale
    for scale in (-0.05, 0.0):
        out = c.attention(q, _i32(lens), _i32(table), count=None if count is None else _i32(count), scale=scale)
        want, spread, reach = ref.attention(_np(q), pool, lens, cnt, table, scale)
        _check_attention(out, want, spread, reach, max(lens), 128, DT[dtype])
    assert c.device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("nq", [1, 70])
def test_attention_split_over_long_sequences(dtype, nq):
    lens = [6001, 3, 20000]
    c, table, pool = _filled(128, 8, 2, lens, DT[dtype], seed=5)
    q = torch.randn(3, nq, 8, 128, device="cuda").to(DT[dtype])
    out = c.attention(q, _i32(lens), _i32(table))
    want, spread, reach = ref.attention(_np(q), pool, lens, [nq] * 3, table, 128 ** -0.5)
    _check_attention(out, want, spread, reach, max(lens), 128, DT[dtype])


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("f16", 64), ("f16", 128)])
def test_attention_long_chunks_keep_their_sums(dtype, d):
    """One warp (or one SM) walks 100000 tokens: its sums may not drift.  The part of the result along the
    exact one: roundings to nearest cancel in it (fp16: 2^-11 each, over 9000 values or more, 5 deviations
    are 2.6e-5; fp32: 6250 additions of 2^-24, 2^-24 sqrt(6250) = 4.7e-6 if all fell alike), a truncating sum
    does not.  fp32 is held to that in the 2-norm too."""
    lens, nq = [100000], 70
    c, table, pool = _filled(d, 2, 1, lens, DT[dtype], seed=7)
    q = torch.randn(1, nq, 2, d, device="cuda").to(DT[dtype])
    out = _np(c.attention(q, _i32(lens), _i32(table)))
    want, _, _ = ref.attention(_np(q), pool, lens, [nq], table, d ** -0.5)
    gain = abs((out * want).sum() / (want * want).sum() - 1)
    assert gain <= (4.7e-6 if dtype == "f32" else 2.6e-5)
    if dtype == "f32":
        assert np.linalg.norm(out - want) <= 4.7e-6 * np.linalg.norm(want)


def _unlike_scales(d, hq, hkv, lens):
    B, blocks, pages = 2, 27, 60
    c = _cache(d, hq, hkv, pages, blocks)
    table = _table(B, blocks, pages)
    rs = np.random.RandomState(1)
    size = 2.0 ** rs.uniform(-12, 12, (B, 1, 27, 1, 1))
    v = (rs.randn(B, 1, 27, 16, d) * size).reshape(B, 1, 432, d)[:, :, :400]
    k = rs.randn(B, 1, 400, d) * np.repeat(2.0 ** rs.uniform(-4, 1, (B, 1, 25, 1)), 16, axis=2)
    # (fp32 input of both whatever the queries' type is: the pool does not remember)
    c.append(torch.from_numpy(k).float().cuda(), torch.from_numpy(v).float().cuda(), _i32([0, 0]), _i32(table), count=_i32(lens))
    return c, table, ref.Pool(c.pool.cpu().numpy(), hkv, d)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("nq", [1, 3, 140])
def test_attention_unlike_scales(dtype, nq):
    """Value blocks whose scales lie 2^24 apart, keys that make the softmax sharp, large and small queries."""
    lens = [400, 163]
    d, hq, hkv = 128, 4, 1
    B = 2
    c, table, pool = _unlike_scales(d, hq, hkv, lens)
    q = (torch.randn(B, nq, hq, d, device="cuda") * torch.tensor([1e-3, 1.0, 3.0, 6.0], device="cuda")[:, None]).to(DT[dtype])
    _check_unlike_scales(c, pool, table, lens, q)


def _check_unlike_scales(c, pool, table, lens, q):
    # Weights are stored as fp16, whose smallest step is 2^-24, relative to 2^M.  M lies at least 7 below the
    # row's largest exponent (bf16 and fp16 chunks; 14 elsewhere), so the largest weight is stored as 2^7 (2^14)
    # or more and the step is at most 2^-31 (2^-38 for fp32, whose second term has the same step) of it.  Where
    # scales differ by 2^24, weights of the small blocks get there, and a coordinate that the large blocks hold
    # zeros for shows it.
    B, nq, d = q.shape[0], q.shape[1], q.shape[3]
    out = c.attention(q, _i32(lens), _i32(table))
    args = (_np(q), pool, lens, [nq] * B, table, d ** -0.5)
    want, spread, reach = ref.attention(*args)
    least = ref.attention_least(*args, 2.0 ** (-38 if q.dtype == torch.float32 else -31))
    _check_attention(out, want, spread, reach, max(lens), d, q.dtype, least)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_attention_least_weights(dtype):
    """Queries for which some outputs rest on the smallest weights, or are subnormal fp16 values."""
    lens, d, hq, hkv, nq = [400, 163], 128, 4, 1, 140
    c, table, pool = _unlike_scales(d, hq, hkv, lens)
    for seed in (40, 51, 186, 445, 693, 1130, 1195, 2807):
        torch.manual_seed(seed)
        size = torch.tensor([1e-3, 1.0, 3.0, 6.0], device="cuda")[:, None]
        _check_unlike_scales(c, pool, table, lens, (torch.randn(2, nq, hq, d, device="cuda") * size).to(DT[dtype]))


def test_attention_nonfinite_queries_stay_in_their_rows():
    lens = [100, 40]
    c, table, pool = _filled(128, 4, 2, lens, torch.bfloat16, seed=2)
    for nq in (1, 60):
        q = torch.randn(2, nq, 4, 128, device="cuda").to(torch.bfloat16)
        clean = c.attention(q, _i32(lens), _i32(table))
        q[0, -1, 1, 5] = float("nan")
        q[1, -1, 3, 7] = float("inf")
        out = c.attention(q, _i32(lens), _i32(table))
        assert torch.isnan(out[0, -1, 1]).all() and torch.isnan(out[1, -1, 3]).all()
        keep = torch.ones(out.shape[:3], dtype=torch.bool, device="cuda")
        keep[0, -1, 1] = keep[1, -1, 3] = False
        assert torch.equal(out[keep], clean[keep])


def test_attention_reports():
    b = _api().binding
    lens = [40, 20]
    c, table, pool = _filled(64, 2, 2, lens, torch.float16, seed=3)
    q = torch.randn(2, 1, 2, 64, device="cuda").half()
    good = c.attention(q, _i32(lens), _i32(table))
    bad = table.copy()
    bad[0, 1] = -7
    out = c.attention(q, _i32(lens), _i32(bad))
    assert c.device_error() == b.TQ_DEVERR_BAD_PAGE
    assert torch.equal(out[1], good[1])
    c.attention(q, _i32([-5, 20]), _i32(table))
    assert c.device_error() == b.TQ_DEVERR_BAD_LENGTH
    c.attention(q, _i32([40, 1 << 30]), _i32(table))
    assert c.device_error() == b.TQ_DEVERR_BAD_LENGTH
    assert c.device_error() == 0


def test_pool_beyond_32_bits():
    """Blocks past 2^32 bytes of a large pool."""
    d, H, blocks = 256, 8, 4
    pages = (1 << 32) // (H * (32 * d + 32)) + 400
    c = _cache(d, 8, H, pages, blocks, garbage=False)
    table = np.array([[pages - 1, 3, pages - 77, pages // 2]], dtype=np.int32)
    x = torch.randn(2, 1, H, 55, d, device="cuda").to(torch.bfloat16)
    c.append(x[0], x[1], _i32([0]), _i32(table))
    at = [int(p) * H * c.block_bytes for p in table[0]]
    blk = np.stack([c.pool[a:a + H * c.block_bytes].cpu().numpy() for a in at])
    pool = ref.Pool(blk, H, d)
    want = ref.Pool(np.zeros_like(blk), H, d)
    for side in (0, 1):
        want.append(side, _np(x[side]), [0], [[0, 1, 2, 3]])
    assert np.array_equal(pool.blocks, want.blocks)
    q = torch.randn(1, 1, 8, d, device="cuda").to(torch.bfloat16)
    out = c.attention(q, _i32([55]), _i32(table))
    o, spread, reach = ref.attention(_np(q), pool, [55], [1], [[0, 1, 2, 3]], d ** -0.5)
    _check_attention(out, o, spread, reach, 55, d, torch.bfloat16)


# ---- as they are used together

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prefill_then_steps(dtype):
    """A prompt in one chunk, then tokens one by one, against the same tokens appended one by one."""
    tq = _api()
    d, hq, hkv, B, n, more = 128, 8, 2, 2, 45, 6
    dt = DT[dtype]
    rot = tq.Rotary(d, base=500000.0)
    wq, wk = ((1 + 0.1 * torch.randn(d, device="cuda")).to(dt) for _ in range(2))
    qkv = torch.randn(B, n + more, hq + 2 * hkv, d, device="cuda").to(dt)
    blocks, pages = 5, 12
    table = _table(B, blocks, pages)

    def run(parts):
        c = _cache(d, hq, hkv, pages, blocks, garbage=False)
        outs, at = [], 0
        for m in parts:
            x = qkv[:, at:at + m]
            q = c.append(x[:, :, hq:hq + hkv].transpose(1, 2), x[:, :, hq + hkv:].transpose(1, 2), _i32([at] * B), _i32(table),
                         rotary=rot, k_weight=wk, q=x[:, :, :hq], q_weight=wq)
            at += m
            outs.append((c, q, c.attention(q, _i32([at] * B), _i32(table))))
        return outs

    a = run([n] + [1] * more)
    for side_run in (a,):
        at = 0
        for c, q, out in side_run:
            at += q.shape[1]
        pool = ref.Pool(c.pool.cpu().numpy(), hkv, d)
        want, spread, reach = ref.attention(_np(q), pool, [at] * B, [1] * B, table, d ** -0.5)
        _check_attention(out, want, spread, reach, at, d, dt)
    # one by one: the scales of a block rise as it fills, so codes may be one rounding apart
    b = run([1] * (n + more))
    pa, pb = (ref.Pool(r[-1][0].pool.cpu().numpy(), hkv, d) for r in (a, b))
    for bb in range(B):
        for h in range(hkv):
            for side in (0, 1):
                x, y = (p.read(side, h, table[bb], n + more) for p in (pa, pb))
                s = np.array([pa.scale(table[bb][t // 16], h, side) for t in range(n + more)])[:, None]
                assert np.array_equal(s, np.array([pb.scale(table[bb][t // 16], h, side) for t in range(n + more)])[:, None])
                # each rounding to a larger scale moves a code by at most half a subnormal step of it
                assert np.all(np.abs(x - y) <= 2.0 ** -9 * s + 2.0 ** -3 * np.abs(x) * (np.abs(x) < 2.0 ** -5 * s))


def test_rotated_rows_feed_the_packed_cache():
    """norm_rotate's fp32 outputs are what the packed caches take."""
    tq = _api()
    B, n, hq, hkv, d = 2, 64, 8, 2, 128
    qkv = torch.randn(B, n, hq + 2 * hkv, d, device="cuda").to(torch.bfloat16)
    rot = tq.Rotary(d)
    q, k = tq.norm_rotate(qkv[:, :, :hq], qkv[:, :, hq:hq + hkv].transpose(1, 2), rotary=rot, out_dtype=torch.float32)
    v = qkv[:, :, hq + hkv:].transpose(1, 2).float()
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    packed = tq.PagedKVCache(d, hq, hkv, B, 8, 4, scheme="tq", n=4)
    packed.append(k, v, _i32([0, 0]), table)
    byte = tq.PagedByteCache(d, hq, hkv, 8, 4)
    byte.append(k, v, _i32([0, 0]), table)
    last = q[:, -1:].contiguous()
    a, b = packed.decode(last, _i32([n, n]), table), byte.attention(last, _i32([n, n]), table)
    kk, vv = (x.repeat_interleave(hq // hkv, 1).double() for x in (k, v))
    want = torch.softmax(torch.einsum("bhd,bhtd->bht", last[:, 0].double(), kk) / d ** 0.5, -1)[:, :, None] @ vv
    err = [float((x[:, 0].double() - want[:, :, 0]).norm() / want.norm()) for x in (a, b)]
    # e4m3 codes are off by at most 2^-4 of themselves, 4-bit ones by far more on average
    assert err[1] < 2.0 ** -4 and err[1] < err[0]


def test_graph_replay_follows_device_state():
    tq = _api()
    d, hq, hkv, B, blocks, pages = 128, 8, 2, 2, 6, 16
    rot = tq.Rotary(d)
    table, start, seq = _i32(_table(B, blocks, pages)), _i32([0, 0]), _i32([1, 1])
    x = torch.zeros(B, 1, hq + 2 * hkv, d, device="cuda", dtype=torch.bfloat16)
    c, e = (_cache(d, hq, hkv, pages, blocks, garbage=False) for _ in range(2))

    def step(cache):
        q = cache.append(x[:, :, hq:hq + hkv].transpose(1, 2), x[:, :, hq + hkv:].transpose(1, 2), start, table, rotary=rot,
                         q=x[:, :, :hq])
        return cache.attention(q, seq, table)

    step(c)  # warm
    c.pool.zero_()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):  # two graphs of one cache: each has its own workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(c)
        graphs.append((g, out))
    for t in range(40):
        x.copy_(torch.randn(B, 1, hq + 2 * hkv, d, device="cuda"))
        start.copy_(_i32([t, t // 2]))
        seq.copy_(_i32([t + 1, t // 2 + 1]))
        if t == 20:  # other pages
            new = _i32(_table(B, blocks, pages, seed=9))
            for cache in (c, e):
                old = cache.pool.view(pages + 1, -1).clone()
                cache.pool.view(pages + 1, -1)[new.view(-1).long()] = old[table.view(-1).long()]
            table.copy_(new)
        g, out = graphs[t % 2]
        g.replay()
        want = step(e)
        assert torch.equal(out, want), t
    assert torch.equal(c.pool, e.pool)


def test_streams_and_calls_at_once():
    tq = _api()
    lens = [3000, 1, 777]
    c, table, pool = _filled(128, 8, 2, lens, torch.bfloat16, seed=8)
    tb, seq = _i32(table), _i32(lens)
    qs = [torch.randn(3, nq, 8, 128, device="cuda").to(torch.bfloat16) for nq in (1, 2, 1, 50)]
    want = [c.attention(q, seq, tb) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    got = []
    for _ in range(5):
        got.append([c.attention(q, seq, tb, stream=s) for q, s in zip(qs, streams)])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    rot = tq.Rotary(128)
    s = streams[0]
    a = tq.norm_rotate(qs[3], rotary=rot, stream=s)[0]
    s.synchronize()
    assert torch.equal(a, tq.norm_rotate(qs[3], rotary=rot)[0])


def test_empty_batches_and_single_query_shape():
    tq = _api()
    c, table, pool = _filled(64, 4, 2, [30, 9], torch.float32, seed=4)
    q = torch.randn(2, 4, 64, device="cuda")
    out = c.attention(q, _i32([30, 9]), _i32(table))
    assert out.shape == q.shape
    assert torch.equal(out, c.attention(q[:, None], _i32([30, 9]), _i32(table))[:, 0])
    # a plain scale argument
    other = c.attention(q, _i32([30, 9]), _i32(table), scale=0.0)
    mean = np.stack([[pool.read(1, h // 2, table[b], n).mean(0) for h in range(4)] for b, n in ((0, 30), (1, 9))])
    assert np.allclose(_np(other), mean, atol=1e-5 * np.abs(mean).max())
    none = torch.zeros(0, table.shape[1], dtype=torch.int32, device="cuda")
    assert c.attention(q[:0], _i32([]), none).shape == (0, 4, 64)
    before = c.pool.clone()
    k = torch.zeros(2, 2, 0, 64, device="cuda")
    assert c.append(k, k, _i32([0, 0]), _i32(table)) is None
    assert torch.equal(before, c.pool)
    assert tq.binding.TQ_DEVERR_NONFINITE == 5
