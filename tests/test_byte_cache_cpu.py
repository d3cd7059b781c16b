"""Byte cache and rotation without a GPU: the rotary table against the definition, the reference's own
properties, and every refusal of the C entry points (all of them before any launch)."""

import ctypes
import math

import numpy as np
import pytest

import byte_reference as ref

b = pytest.importorskip("turboquant_quantized_kv_tq_gb300.binding")


def _table(dim, freqs, axes=None, num_axes=1):
    f = np.ascontiguousarray(freqs, dtype=np.float64)
    a = np.ascontiguousarray(axes, dtype=np.int32) if axes is not None else None
    out = np.zeros(dim // 2, dtype=np.uint64)
    st = b.tq_rotary_table(dim, f.ctypes.data, a.ctypes.data if a is not None else None, num_axes, out.ctypes.data)
    return st, out


@pytest.mark.parametrize("dim,base", [(16, 10000.0), (64, 500000.0), (128, 10000.0), (512, 1e6)])
def test_rotary_table_holds_turn_fractions(dim, base):
    from fractions import Fraction
    # 2 pi to 60 digits
    two_pi = Fraction("6.28318530717958647692528676655900576839433879875021164194988918")
    freqs = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    freqs[1] = -freqs[1]
    axes = [i % 3 for i in range(dim // 2)]
    st, out = _table(dim, freqs, axes, 3)
    assert st == b.TQ_OK
    for f, a, e in zip(freqs, axes, out.tolist()):
        assert e & 3 == a
        exact = Fraction(f) / two_pi * 2 ** 64
        diff = (Fraction(e & ~3) - exact) % 2 ** 64
        # rounded to a multiple of 4 (2), plus the quotient's second double (2^-106 relative: nothing)
        assert min(diff, 2 ** 64 - diff) <= Fraction(5, 2)


@pytest.mark.parametrize("dim,freqs,axes,num_axes", [
    (8, [1.0] * 4, None, 1), (24, [1.0] * 12, None, 1), (1024, [1.0] * 512, None, 1),
    (16, [math.nan] + [1.0] * 7, None, 1), (16, [math.inf] + [1.0] * 7, None, 1),
    (16, [1.0] * 8, [0] * 7 + [2], 2), (16, [1.0] * 8, [-1] + [0] * 7, 2), (16, [1.0] * 8, None, 0),
    (16, [1.0] * 8, None, 5),
])
def test_rotary_table_refusals(dim, freqs, axes, num_axes):
    assert _table(dim, freqs, axes, num_axes)[0] == b.TQ_ERR_INVALID_ARG
    assert b.tq_last_error()


def test_reference_encode_is_nearest_even():
    v = ref.VALUES[:127]
    assert v[126] == 448 and v[1] == 2.0 ** -9
    assert np.array_equal(ref.e4m3_encode(v), np.arange(127))
    mid = (v[:-1] + v[1:]) / 2
    got = ref.e4m3_encode(mid)
    assert np.all(got % 2 == 0)
    assert np.array_equal(ref.e4m3_encode(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert np.array_equal(ref.e4m3_encode([1e9, -1e9, np.inf, np.nan, -0.0]), [126, 254, 126, 0, 128])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_reference_places_cover_a_block(d):
    p = ref.places(d)
    assert np.array_equal(np.sort(p.ravel()), np.arange(32 * d))


# ---- refusals (made-up device addresses: a refused call touches none of them)

DEV = 1 << 20


def _cfg(d=128, hq=8, hkv=2):
    return b.tq_byte_config(d, hq, hkv)


def _pt(table=DEV, mb=4, pages=8):
    return b.tq_page_table(table, mb, pages)


def _h(heads, data=DEV, d=128, n=3, s=None):
    s = s or (n * heads * d, heads * d, d)
    return b.tq_heads(data, s[0], s[1], s[2], heads)


def _rot(table=DEV, dim=128, inter=0, axes=1):
    return b.tq_rotary(table, dim, inter, axes)


def _append(cfg=None, pool=DEV, pt=None, batch=2, n=3, dt=b.TQ_BF16, k=None, v=None, start=DEV, count=None, wk=None,
            eps=1e-6, rot=None, pos=None, q=None, wq=None, qo=None, err=None):
    return b.tq_byte_append_paged(cfg or _cfg(), pool, pt or _pt(), batch, n, dt, k or _h(2), v or _h(2), start, count,
                                  wk, eps, rot, pos, q, wq, qo, err, None)


def _attend(cfg=None, pool=DEV, pt=None, batch=2, nq=1, dt=b.TQ_BF16, q=None, seq=DEV, count=None, scale=0.1, out=2 * DEV,
            ws=DEV, bytes_=1 << 40, err=None):
    return b.tq_byte_attention_paged(cfg or _cfg(), pool, pt or _pt(), batch, nq, dt, q or _h(8, n=nq), seq, count, scale,
                                     out, ws, bytes_, err, None)


def _rotate(d=128, dt=b.TQ_BF16, odt=b.TQ_BF16, batch=2, n=3, q=True, wq=None, qo=2 * DEV, k=None, wk=None, ko=None,
            eps=1e-6, rot=None, pos=None, start=None):
    return b.tq_norm_rotate(d, dt, odt, batch, n, _h(8) if q is True else q, wq, qo, k, wk, ko, eps, rot, pos, start,
                            None)


BAD_POOL = [dict(pool=None), dict(pool=DEV + 16), dict(pt=_pt(table=None)), dict(pt=_pt(table=DEV + 2)),
            dict(pt=_pt(mb=0)), dict(pt=_pt(pages=0)), dict(pt=_pt(mb=1 << 28)), dict(err=DEV + 2),
            dict(cfg=_cfg(hq=7)), dict(cfg=_cfg(hkv=0)), dict(batch=0), dict(batch=513), dict(dt=3)]


@pytest.mark.parametrize("kw", BAD_POOL + [
    dict(n=-1), dict(n=1 << 30), dict(k=_h(3)), dict(k=_h(2, data=None)), dict(k=_h(2, data=DEV + 8)),
    dict(v=_h(2, s=(768, 256, 4))), dict(v=_h(2, s=(-768, 256, 128))), dict(start=None), dict(start=DEV + 1),
    dict(count=DEV + 1), dict(pos=DEV + 2), dict(wk=DEV + 8), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
    dict(q=_h(8)), dict(q=_h(4), qo=DEV), dict(q=_h(8), qo=DEV + 8), dict(q=_h(8), qo=DEV, wq=DEV + 4),
    dict(rot=_rot(dim=8)), dict(rot=_rot(dim=24)), dict(rot=_rot(dim=256)), dict(rot=_rot(inter=2)),
    dict(rot=_rot(axes=0)), dict(rot=_rot(axes=5)), dict(rot=_rot(table=DEV + 4)),
    dict(q=_h(8, data=2 * DEV), qo=2 * DEV + 256), dict(q=_h(8, data=2 * DEV), qo=DEV),
])
def test_append_refusals(kw):
    assert _append(**kw) == b.TQ_ERR_INVALID_ARG
    assert b.tq_last_error()


@pytest.mark.parametrize("kw", BAD_POOL + [
    dict(nq=0), dict(nq=1 << 30), dict(q=_h(4)), dict(q=_h(8, data=DEV + 4)), dict(seq=None), dict(seq=DEV + 2),
    dict(count=DEV + 2), dict(out=None), dict(out=DEV + 8), dict(out=DEV), dict(ws=None), dict(ws=DEV + 128),
    dict(scale=math.inf),
    dict(scale=math.nan),
])
def test_attention_refusals(kw):
    assert _attend(**kw) == b.TQ_ERR_INVALID_ARG
    assert b.tq_last_error()


@pytest.mark.parametrize("kw", [
    dict(dt=3), dict(odt=b.TQ_F16), dict(q=None), dict(qo=None), dict(k=_h(2)), dict(batch=0), dict(batch=513),
    dict(n=-1), dict(n=1 << 30), dict(q=_h(0)), dict(q=_h(8, s=(1025, 1024, 128))), dict(qo=DEV + 4),
    dict(wq=DEV + 4), dict(pos=DEV + 1), dict(start=DEV + 1), dict(eps=-1.0), dict(rot=_rot(dim=144)),
    # outputs over inputs: shifted, in another type, in another layout, over the other tensor
    dict(qo=DEV + 1024), dict(qo=DEV, dt=b.TQ_BF16, odt=b.TQ_F32), dict(qo=DEV, q=_h(8, s=(6144, 2048, 128))),
    dict(k=_h(2, data=2 * DEV), ko=3 * DEV),
])
def test_norm_rotate_refusals(kw):
    assert _rotate(**kw) == b.TQ_ERR_INVALID_ARG
    assert b.tq_last_error()


def test_unbuilt_sizes():
    assert _append(cfg=_cfg(d=96)) == b.TQ_ERR_UNSUPPORTED
    assert _attend(cfg=_cfg(d=512)) == b.TQ_ERR_UNSUPPORTED
    assert _rotate(d=96) == b.TQ_ERR_UNSUPPORTED
    assert b.tq_byte_pool_bytes(_cfg(d=96), 4) == 0
    assert b.tq_byte_pool_bytes(_cfg(), 0) == 0
    assert b.tq_byte_pool_bytes(_cfg(), 5) == 6 * 2 * (32 * 128 + 32)


def test_workspace_is_checked():
    need = b.tq_byte_attention_workspace_bytes(_cfg(), _pt(), 2, 1, b.TQ_BF16)
    assert need > 0
    assert _attend(bytes_=need - 1) == b.TQ_ERR_WORKSPACE
    assert b.tq_byte_attention_workspace_bytes(_cfg(), _pt(), 0, 1, b.TQ_BF16) == 0


def test_empty_calls_launch_nothing():
    # (there is no GPU here: a launch would fail)
    assert _append(n=0) == b.TQ_OK
    assert _rotate(n=0) == b.TQ_OK


def test_dequantize_refusals():
    def f(b_=0, h=0, t0=0, t1=4, k=DEV, v=DEV):
        return b.tq_byte_dequantize(_cfg(), DEV, _pt(), 2, b_, h, t0, t1, k, v, None)
    for kw in (dict(b_=2), dict(h=2), dict(h=-1), dict(t0=-1), dict(t0=5), dict(k=None), dict(v=DEV + 2)):
        assert f(**kw) == b.TQ_ERR_INVALID_ARG
    assert f(t1=65) == b.TQ_ERR_CAPACITY
    assert f(t0=4) == b.TQ_OK


def test_python_refusals():
    torch = pytest.importorskip("torch")
    from turboquant_quantized_kv_tq_gb300 import PagedByteCache, Rotary, TQError, norm_rotate
    with pytest.raises(ValueError):
        Rotary(64, sections=[16, 17], device="cpu")
    with pytest.raises(ValueError):
        Rotary(64, freqs=[1.0] * 31, device="cpu")
    with pytest.raises(TQError):
        Rotary(24, device="cpu")
    assert Rotary(64, sections=[16, 8, 8], device="cpu").num_axes == 3
    with pytest.raises(ValueError):
        norm_rotate()
    with pytest.raises(ValueError):
        norm_rotate(out_dtype=torch.float16)
    with pytest.raises(ValueError):
        norm_rotate(torch.zeros(1, 1, 2, 64))
    with pytest.raises(TQError):
        PagedByteCache(96, 4, 4, 8, 4, device="cpu")
    c = PagedByteCache(64, 4, 2, 8, 4, device="cpu")
    table = torch.zeros(2, 4, dtype=torch.int32)
    seq = torch.zeros(2, dtype=torch.int32)
    for q in (torch.zeros(2, 4, 64, dtype=torch.float64), torch.zeros(2, 3, 64), torch.zeros(3, 4, 64),
              torch.zeros(2, 4, 128)[..., ::2]):
        with pytest.raises(ValueError):
            c.attention(q, seq, table)
    with pytest.raises(ValueError):
        c.attention(torch.zeros(2, 4, 64), seq.long(), table)
    with pytest.raises(ValueError):
        c.attention(torch.zeros(2, 4, 64), seq, table[:, :3])
    k = torch.zeros(2, 2, 3, 64)
    with pytest.raises(ValueError):
        c.append(k, k[:, :, :2], seq, table)
    with pytest.raises(ValueError):
        c.append(k, k, None, table)
    with pytest.raises(ValueError):
        c.append(k, k, seq, table, k_weight=torch.zeros(32))


def test_struct_sizes():
    assert ctypes.sizeof(b.tq_heads) == 40 and ctypes.sizeof(b.tq_rotary) == 24
