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


def _ends(rows, d, dtype, seed):
    """Rows of unlike magnitude, row i of size 2^e(i): from those whose squares pass fp32's largest value down to
    those whose squares are below its smallest (as far as the type goes)."""
    lo, hi = {"f32": (-140, 125), "bf16": (-125, 125), "f16": (-12, 13)}[dtype]
    e = np.linspace(lo, hi, rows).round()
    x = np.random.RandomState(seed).randn(rows, d).clip(-3.5, 3.5) * 2.0 ** e[:, None]
    return torch.from_numpy(x).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d,r", [(64, 32), (128, 0), (256, 256), (512, 64)])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-6])
def test_norm_of_any_magnitude(dtype, d, r, eps):
    """x / sqrt(mean(x^2) + eps) * w is an ordinary number wherever x and w are.

    The factor is off by at most 2^-20: sums of squares of one sign, 16 additions or less deep (2^-24 each, halved
    by the root: 2^-21), the division by d and the root's own rounding (2^-22 together), two products (2^-23).
    Cosines are off by 2^-22; a rotated value adds two products and a sum (2^-23).  Below 2^-126 an output and a
    factor of it are subnormal: steps of 2^-149, and the products' own (weights are at most 2)."""
    tq = _api()
    rows = 90
    x = _ends(rows, d, dtype, d).view(1, rows, 1, d)
    w = (1 + 0.2 * torch.randn(d, device="cuda").clamp(-3, 3)).to(DT[dtype])
    rot = tq.Rotary(r) if r else None
    freqs = [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]
    y, _ = tq.norm_rotate(x, rotary=rot, q_weight=w, eps=eps, out_dtype=torch.float32)
    # (eps enters as fp32)
    want, size = ref.norm_rotate(_np(x[0, :, 0]), _np(w), float(np.float32(eps)), freqs if r else None, [0] * (r // 2), False,
                                 np.arange(rows)[None])
    tol = (2.0 ** -20 + 2.0 ** -22 + 2.0 ** -23) * size + 2.0 ** -146
    got = _np(y[0, :, 0])
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - want) <= tol), np.max(np.abs(got - want) / tol)


def test_norm_of_infinities_and_zeros():
    """mean(x^2) is infinite: finite coordinates become 0 and the infinite one NaN; a NaN takes its whole row; a row
    of zeros without eps is 0 / 0.  Other rows stay as they are."""
    tq = _api()
    x = torch.randn(1, 6, 1, 128, device="cuda")
    w = torch.ones(128, device="cuda")
    clean, _ = tq.norm_rotate(x, q_weight=w, eps=0.0)
    x[0, 1, 0, 5], x[0, 2, 0, 7], x[0, 4] = float("inf"), float("nan"), 0.0
    y = tq.norm_rotate(x, q_weight=w, eps=0.0)[0][0, :, 0]
    assert torch.isnan(y[1, 5]) and not y[1, :5].any() and not y[1, 6:].any()
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    for i in (0, 3, 5):
        assert torch.equal(y[i], clean[0, i, 0])
    assert not tq.norm_rotate(x, q_weight=w)[0][0, 4].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_norms_large_keys(dtype):
    """Finite keys are finite codes after the norm, whatever their size, and nothing is recorded."""
    tq = _api()
    d, H, n = 128, 2, 37
    k = _ends(n, d, dtype, 3).view(1, 1, n, d).expand(1, H, n, d).contiguous()
    w = torch.ones(d, device="cuda", dtype=DT[dtype])
    c = tq.PagedByteCache(d, H, H, 8, 4)
    table = _i32([[3, 1, 7, 0]])
    c.append(k, torch.zeros_like(k), _i32([0]), table, k_weight=w, eps=0.0)
    assert c.device_error() == 0
    pool = ref.Pool(c.pool.cpu().numpy(), H, d)
    want, _ = ref.norm_rotate(_np(k[0, 0]), np.ones(d), 0.0, None, [], False, None)
    for h in range(H):
        got = pool.read(0, h, table[0].tolist(), n)
        size = np.array([pool.scale(int(table[0, t // 16]), h, 0) for t in range(n)])[:, None]
        # half a step of e4m3, normal or subnormal, and the norm's own 2^-20
        assert np.all(np.abs(got - want) <= np.maximum(2.0 ** -4 * np.abs(want), 2.0 ** -10 * size) * (1 + 2.0 ** -10) +
                      2.0 ** -20 * np.abs(want))


def test_norm_fp32_error():
    """The 2-norm of the error in fp32.  Roundings are independent and each at most 2^-24 (rms 2^-24 / sqrt 3): half the
    sum of squares' (16 deep: 1.15 units of 2^-24), division, eps and root 0.8, two products 0.8, cosines 1 to the pair, a
    rotated pair 0.8; together 2.1 units, 1.3e-7.  Twice that is allowed."""
    tq = _api()
    q = torch.randn(1, 600, 8, 128, device="cuda")
    w = 1 + 0.2 * torch.randn(128, device="cuda")
    y, _ = tq.norm_rotate(q, rotary=tq.Rotary(128), q_weight=w)
    freqs = [10000.0 ** (-2.0 * i / 128) for i in range(64)]
    want, _ = ref.norm_rotate(_np(q[0].transpose(0, 1)), _np(w), 1e-6, freqs, [0] * 64, False, np.arange(600)[None])
    assert np.linalg.norm(_np(y[0].transpose(0, 1)) - want) <= 2.6e-7 * np.linalg.norm(want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_any_magnitude_in_place(dtype):
    """Rows that are taken a second time, from a buffer that their neighbours' results already replace."""
    tq = _api()
    d, H, n = 128, 37, 50
    q = _ends(n * H, d, dtype, 5).view(1, n, H, d)
    q = q[:, torch.randperm(n, generator=torch.Generator().manual_seed(0)).cuda()]
    k = q.transpose(1, 2).contiguous()
    w = torch.linspace(0.5, 2.0, d, device="cuda").to(DT[dtype])
    want = tq.norm_rotate(q, k, rotary=tq.Rotary(d), q_weight=w, k_weight=w, eps=0.0)
    got = tq.norm_rotate(q, k, rotary=tq.Rotary(d), q_weight=w, k_weight=w, eps=0.0, q_out=q, k_out=k)
    assert got[0] is q and got[1] is k
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.isfinite(q).all()
    assert torch.equal(k, q.transpose(1, 2))
