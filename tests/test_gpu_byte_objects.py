"""The byte cache's and the rotation's objects beside the calls: what they own on other streams, the error word, errors."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def _api():
    import turboquant_quantized_kv_tq_gb300 as tq
    return tq


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _busy(s):
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # some 50 ms: the call below waits behind it


def test_dropped_rotary_lives_until_its_call_ran():
    tq = _api()
    q = torch.randn(2, 5, 4, 128, device="cuda")
    start = _i32([7, 100000])
    want = tq.norm_rotate(q, rotary=tq.Rotary(128), start=start)[0]
    s = torch.cuda.Stream()
    _busy(s)
    got = tq.norm_rotate(q, rotary=tq.Rotary(128), start=start, stream=s)[0]
    other = [torch.full((64,), 3, dtype=torch.int64, device="cuda") for _ in range(2000)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    del other


def test_dropped_cache_lives_until_its_call_ran():
    tq = _api()
    x = torch.randn(2, 1, 2, 40, 128, device="cuda")
    q, seq, start, table = torch.randn(1, 1, 4, 128, device="cuda"), _i32([40]), _i32([0]), _i32([[2, 0, 1]])

    def filled():
        c = tq.PagedByteCache(128, 4, 2, 3, 3)
        c.append(x[0], x[1], start, table)
        return c

    want = filled().attention(q, seq, table)
    s = torch.cuda.Stream()
    c = filled()
    size = c.pool.numel()
    _busy(s)
    got = c.attention(q, seq, table, stream=s)
    del c
    other = [torch.full((size,), 126, dtype=torch.uint8, device="cuda") for _ in range(200)]
    words = [torch.full((1,), 77, dtype=torch.int32, device="cuda") for _ in range(2000)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(int(w) == 77 for w in words[:50])
    del other


def test_device_error_waits_for_every_stream():
    tq = _api()
    c = tq.PagedByteCache(64, 2, 2, 4, 2)
    x, start, bad = torch.randn(1, 2, 3, 64, device="cuda"), _i32([0]), _i32([[9, 9]])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(50_000_000)  # some 25 ms
    c.append(x, x, start, bad, stream=s)
    assert c.device_error() == tq.binding.TQ_DEVERR_BAD_PAGE
    # cleared before the call returned: a later call's code, on any stream, is not lost
    c.append(x, x, start, bad, stream=s)
    s.synchronize()
    assert c.device_error() == tq.binding.TQ_DEVERR_BAD_PAGE
    assert c.device_error() == 0


def test_out_of_memory_is_torchs():
    """An output or a workspace that torch cannot allocate is its OutOfMemoryError, as from any torch call."""
    tq = _api()
    q = torch.zeros(1, 1 << 18, 8, 128, device="cuda", dtype=torch.bfloat16)  # 512 MB
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (64 << 20)) / total)
    try:
        with pytest.raises(torch.OutOfMemoryError):
            tq.norm_rotate(q)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    tq.norm_rotate(q)


def test_norm_rotate_refuses_inputs_that_require_a_gradient():
    tq = _api()
    x, w = torch.randn(1, 3, 2, 64, device="cuda"), torch.ones(64, device="cuda")
    want = tq.norm_rotate(x, q_weight=w)[0]
    x.requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        tq.norm_rotate(x, q_weight=w)
    with pytest.raises(ValueError, match="gradient"):
        tq.norm_rotate(None, x.transpose(1, 2))
    with pytest.raises(ValueError, match="gradient"):
        tq.norm_rotate(x.detach(), q_weight=w.requires_grad_())
    with torch.no_grad():
        assert torch.equal(tq.norm_rotate(x, q_weight=w)[0], want)
    with torch.inference_mode():
        assert torch.equal(tq.norm_rotate(x, q_weight=w)[0], want)


def test_captured_calls_with_a_stream():
    """Calls given the capturing stream, in two graphs of the same objects, which go once the graphs are done."""
    tq = _api()
    rot, c = tq.Rotary(128), tq.PagedByteCache(128, 4, 2, 3, 3)
    x = torch.randn(1, 1, 8, 128, device="cuda")
    start, seq, table = _i32([0]), _i32([1]), _i32([[2, 0, 1]])

    def step(stream=None):
        q = c.append(x[:, :, 4:6].transpose(1, 2), x[:, :, 6:].transpose(1, 2), start, table, rotary=rot, q=x[:, :, :4], stream=stream)
        return c.attention(q, seq, table, stream=stream)

    want = step()
    c.pool.zero_()
    graphs = []
    torch.cuda.synchronize()
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(torch.cuda.current_stream())
        graphs.append((g, out))
    for g, out in graphs:
        g.replay()
        assert torch.equal(out, want)
    assert c.device_error() == 0
    graphs[0][0].replay()
    torch.cuda.synchronize()
    del c, rot, graphs
    assert torch.ones(8, device="cuda").sum() == 8


def test_copied_objects_stand_alone():
    import copy
    tq = _api()
    rot, c = tq.Rotary(128), tq.PagedByteCache(128, 4, 2, 3, 3)
    x = torch.randn(2, 1, 2, 20, 128, device="cuda")
    q, table = torch.randn(1, 1, 4, 128, device="cuda"), _i32([[2, 0, 1]])
    c.append(x[0], x[1], _i32([0]), table, rotary=rot)
    want = c.attention(q, _i32([20]), table)
    r2, c2 = copy.deepcopy(rot), copy.deepcopy(c)
    before = c.pool.clone()
    c2.append(x[1, :, :, :5], x[0, :, :, :5], _i32([20]), table, rotary=r2)
    assert torch.equal(c.pool, before)
    c.append(x[1, :, :, :5], x[0, :, :, :5], _i32([20]), table, rotary=rot)
    assert torch.equal(c.pool, c2.pool)
    del c, rot
    junk = torch.full((1 << 20,), 3, dtype=torch.uint8, device="cuda")
    assert torch.equal(c2.attention(q, _i32([20]), table), want)
    c2.append(x[0], x[1], _i32([0]), _i32([[99, 99, 99]]), rotary=r2)
    assert c2.device_error() == tq.binding.TQ_DEVERR_BAD_PAGE
    del junk
