"""Timed cases of the operators around the 8-bit paged KV cache: head norms with the position rotation
(``norm_rotate``), the append of keys and values (``PagedByteCache.append``) and the attention that reads
the pool (``PagedByteCache.attention``).

A case is a dict of plain values.  ``run`` computes it in plain torch operations where ``own`` is false, and
through the package where it is true; ``exact`` computes it again in 64 bits from the definitions alone.

Definitions.
  norm      y = x / sqrt(mean(x^2) + eps) * w, per head row
  rotation  rotary pair i of r / 2 turns by pos[axis(i)] * freq(i); its members are y[i], y[i + r/2]
            ("halves") or y[2i], y[2i + 1] ("interleaved"); coordinates past r stay
  code      a block of 16 tokens of one KV head and side has the scale 2^e, e the smallest integer in
            [-30, 30] with max |x| <= 448 2^e, and codes e4m3(x / 2^e).  A block that already holds tokens
            takes the larger of its e and the one the new tokens need; held codes are rounded to it.
  block     K codes of 16 tokens in 128-byte rows (64 at head dim 64) whose 16-byte chunks are exchanged by
            the row's index, V codes transposed to [d][16] with tokens 2t, 2t+1, 2t+8, 2t+9 side by side,
            then the scales of K and V (fp32) and 24 bytes of padding.  Block (page, head) is page * heads + head.
"""

import math
import random

import numpy as np
import torch

own = False

TILE = 16
TOP = 448.0  # the largest e4m3 value
E_MIN, E_MAX = -30, 30
EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decode step's new tokens of a batch of 8, keys and queries out of a fused projection
        dict(name="rotate step", op="rotate", B=8, n=1, Hq=32, Hkv=8, d=128, dtype="bf16", out="bf16",
             norm=True, r=128, interleaved=False, axes=1, far=32768),
        # a prefill chunk of the long-context configuration
        dict(name="rotate chunk", op="rotate", B=1, n=4096, Hq=64, Hkv=8, d=128, dtype="bf16", out="bf16",
             norm=True, r=128, interleaved=False, axes=1, far=126976),
        # patches of two images or short clips, positions in time, height and width, fp32 for the packed caches
        dict(name="rotate axes", op="rotate", B=2, n=1369, Hq=16, Hkv=16, d=64, dtype="f16", out="f32",
             norm=False, r=64, interleaved=True, axes=3, far=0),
        # the same decode step, written straight into the cache
        dict(name="append step", op="append", B=8, n=1, Hq=32, Hkv=8, d=128, dtype="bf16", norm=True, r=128,
             interleaved=False, far=32768, start=1000, ragged=False),
        # the prefill chunk of 4096 tokens, beginning inside a block
        dict(name="append chunk", op="append", B=1, n=4096, Hq=64, Hkv=8, d=128, dtype="bf16", norm=True, r=128,
             interleaved=False, far=126976, start=1003, ragged=False),
        # a batch of short prompts of different lengths
        dict(name="append ragged", op="append", B=48, n=37, Hq=16, Hkv=2, d=64, dtype="f16", norm=False, r=32,
             interleaved=True, far=0, start=300, ragged=True),
        # one short sequence, one token: latency
        dict(name="attention short", op="attention", B=1, nq=1, T=1024, Hq=32, Hkv=8, d=128, dtype="f32", ragged=False),
        # the headline decode: 8 sequences of 32768 tokens
        dict(name="attention step", op="attention", B=8, nq=1, T=32768, Hq=32, Hkv=8, d=128, dtype="bf16", ragged=False),
        # one long sequence
        dict(name="attention long", op="attention", B=1, nq=1, T=131072, Hq=64, Hkv=8, d=128, dtype="bf16", ragged=False),
        # a serving batch of unlike lengths, some of them empty, seven queries to a KV head
        dict(name="attention ragged", op="attention", B=64, nq=1, T=9001, Hq=28, Hkv=4, d=128, dtype="f16", ragged=True),
        # four draft tokens a sequence
        dict(name="attention drafts", op="attention", B=16, nq=4, T=16384, Hq=32, Hkv=8, d=128, dtype="bf16", ragged=False),
        # a prefill chunk of 512 queries over a long cache
        dict(name="attention chunk", op="attention", B=4, nq=512, T=32768, Hq=32, Hkv=8, d=128, dtype="bf16", ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["rotate", "append", "attention", "attention"])
    d = rng.choice([64, 128, 128, 128, 256])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 8), (16, 2), (28, 4), (12, 4), (6, 1), (5, 5)])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "attention":
        nq = rng.choice([1, 1, 1, _log(rng, 2, 700)])
        T = _log(rng, max(16, nq), 131072)
        B = _log(rng, 1, 64)
        while B > 1 and (B * T * Hkv * d > 1 << 28 or B * T * Hq * nq > 1 << 30):
            B //= 2
        while T > nq and B * T * Hq * nq > 1 << 30:
            T = max(nq, T // 2)
        return dict(op=op, B=B, nq=nq, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, ragged=rng.random() < 0.5)
    n = rng.choice([1, _log(rng, 2, 4096)])
    B = _log(rng, 1, 64)
    while B > 1 and B * n * (Hq + 2 * Hkv) * d > 1 << 25:
        B //= 2
    while B * n * (Hq + 2 * Hkv) * d > 1 << 25:
        n //= 2
    r = rng.choice([d, d, d // 2])
    c = dict(op=op, B=B, n=n, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype, norm=rng.random() < 0.6, r=r,
             interleaved=rng.random() < 0.4, far=_log(rng, 1, 1000000))
    if op == "rotate":
        return dict(c, out=rng.choice([dtype, "f32"]), axes=rng.choice([1, 1, 2, 3]))
    return dict(c, start=rng.randrange(0, 700), ragged=rng.random() < 0.4)


def _lengths(c):
    """Host lists: tokens of each sequence after the step, and how many of them are the step's own."""
    r = random.Random(c["B"] * 1000003 + c.get("T", 0) * 17 + c.get("nq", c.get("n", 0)))
    n = c["nq"] if c["op"] == "attention" else c["n"]
    if c["op"] == "append":
        start = [r.randrange(0, c["start"] + 1) if c["ragged"] else c["start"] for _ in range(c["B"])]
        return start, [r.randrange(0, n + 1) if c["ragged"] and n > 1 else n for _ in range(c["B"])]
    if not c["ragged"]:
        return [c["T"]] * c["B"], [n] * c["B"]
    seq = [0 if r.random() < 0.08 else _log(r, 1, c["T"]) for _ in range(c["B"])]
    return seq, [min(s, r.randrange(1, n + 1)) if n > 1 else min(s, 1) for s in seq]


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "rotate":
        e = c["B"] * c["n"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": e * (size[c["dtype"]] + size[c["out"]]), "flops": e * (7 if c["norm"] else 3)}
    start, count = _lengths(c)
    if c["op"] == "append":
        new = sum(count) * c["Hkv"] * c["d"]
        q = c["B"] * c["n"] * c["Hq"] * c["d"]
        return {"bytes": 2 * new * (size[c["dtype"]] + 1) + 2 * q * size[c["dtype"]],
                "flops": (new + q) * (7 if c["norm"] else 3) + 4 * new}
    rows = sum(sum(max(0, s - k + 1 + i) for i in range(k)) for s, k in zip(start, count))
    pool = sum(start) * c["Hkv"] * (2 * c["d"] + 8 / TILE)
    return {"bytes": pool + 2 * c["B"] * c["nq"] * c["Hq"] * c["d"] * size[c["dtype"]],
            "flops": 4 * c["d"] * c["Hq"] * rows}


# ---------------------------------------------------------------- the block's layout

def _k_places(d, device):
    """Byte of K code [token][coordinate] in its block."""
    t = torch.arange(TILE, device=device)[:, None]
    x = torch.arange(d, device=device)[None]
    c = x // 16
    if d == 64:
        return t * 64 + (c ^ ((t // 2) % 4)) * 16 + x % 16
    return (c // 8) * 2048 + t * 128 + ((c % 8) ^ (t % 8)) * 16 + x % 16


def _v_places(d, device):
    """Byte of V code [token][coordinate] in its block."""
    t = torch.arange(TILE, device=device)[:, None]
    x = torch.arange(d, device=device)[None]
    return 16 * d + x * 16 + ((t % 8) // 2) * 4 + (t // 8) * 2 + t % 2


def _encode(x):
    return x.clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(codes):
    return codes.view(torch.float8_e4m3fn).to(torch.float32)


def _need(amax):
    """Smallest e with amax <= 448 2^e = 0.875 2^(e + 9), within its range."""
    m, x = torch.frexp(amax)
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


# ---------------------------------------------------------------- inputs

def _freqs(r):
    return [10000.0 ** (-2.0 * i / r) for i in range(r // 2)]


def _sections(r, axes):
    """Rotary pairs of each axis."""
    first = r // 2 // axes
    return [r // 2 - first * (axes - 1)] + [first] * (axes - 1)


def _axis_of(r, axes):
    return [a for a, k in enumerate(_sections(r, axes)) for _ in range(k)]


def _table(c, blocks, gen, device):
    """A block table of `blocks` entries a sequence out of a shuffled pool, and the pool's pages."""
    pages = c["B"] * blocks + 3
    order = torch.randperm(pages, generator=gen, device=device)[: c["B"] * blocks]
    return order.view(c["B"], blocks).to(torch.int32).contiguous(), pages


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 13)
    dt, d, B, Hq, Hkv = DTYPES[c["dtype"]], c["d"], c["B"], c["Hq"], c["Hkv"]
    s = {"c": c}

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    if c["op"] in ("rotate", "append"):
        n = c["n"]
        # a fused projection's output: [B][n] rows of queries, keys and values
        qkv = (normal(B, n, Hq + 2 * Hkv, d) * torch.exp(0.5 * normal(Hq + 2 * Hkv, d))).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv].transpose(1, 2), qkv[:, :, Hq + Hkv:].transpose(1, 2)
        s["wq"] = (1 + 0.1 * normal(d)).to(dt) if c["norm"] else None
        s["wk"] = (1 + 0.1 * normal(d)).to(dt) if c["norm"] else None
        axes = c.get("axes", 1)
        s["freq"] = torch.tensor(_freqs(c["r"]), dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(_axis_of(c["r"], axes), device=dev)
        if axes > 1:  # a grid of patches: time, height, width
            side = max(1, math.isqrt(n - 1) + 1)
            j = torch.arange(n, device=dev)
            grid = [j // max(1, n // 3), j // side, j % side][:axes]
            s["pos"] = (torch.stack(grid)[:, None].expand(axes, B, n) + c["far"]).to(torch.int32).contiguous()
        else:
            first = torch.randint(0, 64, (B, 1), generator=gen, device=dev) + c["far"]
            s["pos"] = (first + torch.arange(n, device=dev)).to(torch.int32)[None].contiguous()
        if own:
            from turboquant_quantized_kv_tq_gb300 import Rotary
            s["rotary"] = Rotary(c["r"], sections=_sections(c["r"], axes), interleaved=c["interleaved"])
    if c["op"] == "rotate":
        return s

    start, count = _lengths(c)
    if c["op"] == "append":
        blocks = max(1, max(-(-(a + k) // TILE) for a, k in zip(start, count)))
        s["table"], pages = _table(c, blocks, gen, dev)
        s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["count"] = torch.tensor(count, dtype=torch.int32, device=dev) if c["ragged"] else None
        # pages in use: finite codes of earlier tokens at scales around the new tokens'
        pool = torch.randint(0, 256, ((pages + 1) * Hkv, 32 * d + 32), generator=gen, device=dev, dtype=torch.uint8)
        pool[pool % 128 == 127] = 126
        scale = torch.exp2(torch.randint(-8, -5, (pool.shape[0], 2), generator=gen, device=dev).float())
        pool[:, 32 * d:] = 0
        pool[:, 32 * d:32 * d + 8] = scale.view(torch.uint8)
    else:
        blocks = max(1, -(-c["T"] // TILE))
        s["table"], pages = _table(c, blocks, gen, dev)
        s["seq"] = torch.tensor(start, dtype=torch.int32, device=dev)
        s["count"] = torch.tensor(count, dtype=torch.int32, device=dev) if c["ragged"] and c["nq"] > 1 else None
        s["q"] = normal(B, c["nq"], Hq, d).to(dt)
        # keys and values with channels of unlike spread, quantized block by block
        pool = torch.zeros((pages + 1) * Hkv, 32 * d + 32, dtype=torch.uint8, device=dev)
        spread = torch.exp(0.7 * normal(2, Hkv, d))
        part = max(1, (1 << 27) // (Hkv * TILE * d))  # pages at a time
        for at in range(0, pages + 1, part):
            m = min(part, pages + 1 - at)
            for side, places in ((0, _k_places(d, dev)), (1, _v_places(d, dev))):
                x = normal(m, Hkv, TILE, d) * spread[side][None, :, None] * (0.6 if side == 0 else 1.0)
                e = _need(x.abs().amax((-1, -2)))
                rows = pool[at * Hkv:(at + m) * Hkv]
                rows[:, places.reshape(-1)] = _encode(torch.ldexp(x, -e[..., None, None])).view(m * Hkv, TILE * d)
                rows[:, 32 * d + 4 * side:32 * d + 4 * side + 4] = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e).view(-1, 1).view(torch.uint8)
        # what lies behind a sequence's last token is anything, NaN codes among it
        seq = s["seq"].long()
        last = s["table"].long().gather(1, ((seq - 1).clamp(min=0) // TILE)[:, None])[:, 0]
        rows = (last[:, None] * Hkv + torch.arange(Hkv, device=dev)).reshape(-1)
        behind = torch.arange(TILE, device=dev)[None] >= ((seq - 1) % TILE + 1)[:, None]
        behind = behind.repeat_interleave(Hkv, 0)[:, :, None].expand(-1, -1, d).reshape(len(rows), -1)
        for places in (_k_places(d, dev), _v_places(d, dev)):
            p = places.reshape(-1)
            pool[rows[:, None], p[None]] = torch.where(behind, torch.full_like(pool[:1, :1], 127), pool[rows[:, None], p[None]])
    s["pool"], s["pages"] = pool, pages
    if own:
        from turboquant_quantized_kv_tq_gb300 import PagedByteCache
        s["cache"] = PagedByteCache(d, Hq, Hkv, pages, blocks)
        s["cache"].pool.copy_(pool.view(-1))
        s["pool"] = s["cache"].pool.view(pool.shape)
    return s


# ---------------------------------------------------------------- the plain forms

def _norm_rotate(s, x, w, token_dim):
    """fp32 rows of x (any leading dims) after norm and rotation; the token axis is `token_dim` (1 or 2)."""
    c = s["c"]
    x = x.to(torch.float32)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.to(torch.float32)
    angle = s["pos"].to(torch.float64)[s["axis"]].permute(1, 2, 0) * s["freq"]  # [B][n][r/2]
    angle = angle.unsqueeze(2 if token_dim == 1 else 1)
    cos, sin = torch.cos(angle).to(torch.float32), torch.sin(angle).to(torch.float32)
    r = c["r"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = x[..., : r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((y, x[..., r:]), -1)


def _append(s):
    c, dev = s["c"], s["k"].device
    d, n, B, H = c["d"], c["n"], c["B"], c["Hkv"]
    q = _norm_rotate(s, s["q"], s["wq"], 1).to(s["q"].dtype)
    start = s["start"].long()
    count = s["count"].long() if s["count"] is not None else torch.full_like(start, n)
    held = start % TILE
    nb = (TILE - 1 + n + TILE - 1) // TILE
    place = torch.arange(nb * TILE, device=dev)
    j = place[None] - held[:, None]                                   # the new token at each place
    new = (j >= 0) & (j < count[:, None])
    old = (place[None] < held[:, None])
    live = new.view(B, nb, TILE).any(-1)                              # blocks that get a token
    at = (start // TILE)[:, None] + torch.arange(nb, device=dev)
    page = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    page = torch.where(live, page, torch.full_like(page, s["pages"]))
    rows = (page[:, None] * H + torch.arange(H, device=dev)[None, :, None]).reshape(-1)   # [B][H][nb]
    block = s["pool"][rows]
    scales = block[:, 32 * d:32 * d + 8].contiguous().view(torch.float32).view(B, H, nb, 2)
    fresh = []
    for side, x, places in ((0, _norm_rotate(s, s["k"], s["wk"], 2), _k_places(d, dev)), (1, s["v"].to(torch.float32), _v_places(d, dev))):
        p = places.reshape(-1)
        x = x.gather(2, j.clamp(0, n - 1)[:, None, :, None].expand(B, H, nb * TILE, d)).view(B, H, nb, TILE, d)
        is_new, is_old = (m.view(B, 1, nb, TILE, 1) for m in (new, old))
        x = torch.where(is_new, x, torch.zeros_like(x))
        e = _need(x.abs().amax((-1, -2)))
        e_old = torch.frexp(scales[..., side])[1] - 1
        e = torch.where(is_old.any(3)[..., 0], torch.maximum(e, e_old), e)
        was = block[:, p].view(B, H, nb, TILE, d)
        codes = _encode(torch.ldexp(x, -e[..., None, None]))
        kept = _encode(torch.ldexp(torch.where(is_old, _decode(was), torch.zeros_like(x)), (e_old - e)[..., None, None]))
        codes = torch.where(is_new, codes, torch.where(is_old, kept, was))
        block[:, p] = torch.where(live.view(B, 1, nb, 1, 1), codes, was).view(-1, TILE * d)
        one = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
        fresh.append(torch.where(live.view(B, 1, nb), one, scales[..., side]))
    block[:, 32 * d:32 * d + 8] = torch.stack(fresh, -1).view(-1, 2).view(torch.uint8)
    s["pool"][rows] = block
    return q


def _attention(s):
    c, dev = s["c"], s["q"].device
    d, nq, B, H, G = c["d"], c["nq"], c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    seq = s["seq"].long()
    count = s["count"].long() if s["count"] is not None else torch.full_like(seq, nq)
    blocks = s["table"].shape[1]
    rows = (s["table"].long()[:, None] * H + torch.arange(H, device=dev)[None, :, None]).reshape(-1)
    valid = torch.arange(blocks * TILE, device=dev)[None] < seq[:, None]
    scales = s["pool"][:, 32 * d:32 * d + 8].contiguous().view(torch.float32)[rows].view(B, H, blocks, 1, 1, 2)

    def side(places, k):
        x = _decode(s["pool"][rows[:, None], places.reshape(-1)[None]]).view(B, H, blocks, TILE, d)
        x = (x * scales[..., k]).view(B, H, blocks * TILE, d)
        return x.masked_fill_(~valid[:, None, :, None], 0.0)

    q = s["q"].to(torch.float32).view(B, nq, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, d)
    score = torch.matmul(q, side(_k_places(d, dev), 0).transpose(-1, -2)).mul_(d ** -0.5)
    i = torch.arange(nq, device=dev)
    limit = torch.where(i[None] < count[:, None], seq[:, None] - count[:, None] + 1 + i[None], torch.zeros_like(seq)[:, None])
    limit = limit.repeat_interleave(G, 1)                                # [B][nq G]
    score.masked_fill_((torch.arange(blocks * TILE, device=dev) >= limit[..., None])[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, side(_v_places(d, dev), 1)) / total.masked_fill(total == 0, 1.0)
    return o.view(B, H, nq, G, d).permute(0, 2, 1, 3, 4).reshape(B, nq, H * G, d).to(s["q"].dtype)


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "rotate":
        out = DTYPES[c["out"]]
        if own:
            from turboquant_quantized_kv_tq_gb300 import norm_rotate
            q, k = norm_rotate(s["q"], s["k"], rotary=s["rotary"], positions=s["pos"], q_weight=s["wq"],
                               k_weight=s["wk"], eps=EPS, out_dtype=out)
        else:
            q, k = (_norm_rotate(s, x, w, t).to(out).contiguous() for x, w, t in ((s["q"], s["wq"], 1), (s["k"], s["wk"], 2)))
        return {"q": q, "k": k}
    if c["op"] == "append":
        if own:
            q = s["cache"].append(s["k"], s["v"], s["start"], s["table"], count=s["count"], rotary=s["rotary"],
                                  positions=s["pos"], k_weight=s["wk"], q=s["q"], q_weight=s["wq"], eps=EPS)
        else:
            q = _append(s)
        d = c["d"]
        return {"q": q, "codes": s["pool"][:, : 32 * d].view(torch.float8_e4m3fn),
                "scales": s["pool"][:, 32 * d:32 * d + 8].view(torch.float32)}
    if own:
        return s["cache"].attention(s["q"], s["seq"], s["table"], count=s["count"])
    return _attention(s)


# ---------------------------------------------------------------- 64 bits, from the definitions

def _exact_row(c, x, w, pos):
    """x [..., n, d] in 64 bits with tokens next to last; pos [axes][n]."""
    x = x.double()
    if w is not None:
        x = x * w.double() / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + EPS)
    y = x.clone()
    r = c["r"]
    for i, (f, a) in enumerate(zip(_freqs(r), _axis_of(r, pos.shape[0]))):
        t = pos[a].double() * f
        m, k = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
        y[..., m] = x[..., m] * torch.cos(t) - x[..., k] * torch.sin(t)
        y[..., k] = x[..., m] * torch.sin(t) + x[..., k] * torch.cos(t)
    return y


def _values64():
    """The value of each e4m3 byte."""
    got = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = math.ldexp(m, -9) if e == 0 else math.ldexp(8 + m, e - 10)
        got.append(math.nan if b & 127 == 127 else -v if b & 128 else v)
    return np.array(got)


def _round64(x):
    """The nearest e4m3 value, ties to the even one, as the value."""
    x = x.clamp(-448.0, 448.0)
    step = torch.exp2(torch.clamp(torch.frexp(x)[1] - 1, min=-6).double() - 3)
    return torch.round(x / step) * step


def _places64(d):
    """Numpy [2][16][d]: byte of each K and V code, one by one."""
    at = np.zeros((2, TILE, d), dtype=np.int64)
    order = [0, 1, 8, 9, 2, 3, 10, 11, 4, 5, 12, 13, 6, 7, 14, 15]  # tokens in the order of V's bytes
    for t in range(TILE):
        for x in range(d):
            if d == 64:
                at[0, t, x] = 64 * t + 16 * ((x // 16) ^ (t // 2 % 4)) + x % 16
            else:
                at[0, t, x] = 2048 * (x // 128) + 128 * t + 16 * ((x % 128 // 16) ^ (t % 8)) + x % 16
            at[1, t, x] = 16 * d + 16 * x + order.index(t)
    return at


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    B, H, d = c["B"], c["Hkv"], c["d"]
    if c["op"] in ("rotate", "append"):
        q = torch.stack([_exact_row(c, s["q"][b].transpose(0, 1), s["wq"], s["pos"][:, b]).transpose(0, 1) for b in range(B)])
        k = torch.stack([_exact_row(c, s["k"][b], s["wk"], s["pos"][:, b]) for b in range(B)])
        if c["op"] == "rotate":
            return {"q": q, "k": k}
        value = torch.from_numpy(_values64()).to(q.device)
        pool = s["pool"].clone()
        codes = value[pool[:, : 32 * d].long()]
        scales = pool[:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
        places = torch.from_numpy(_places64(d)).to(q.device)
        start, count = _lengths(c)
        table = s["table"].cpu().tolist()
        for b in range(B):
            for t0 in range(start[b] // TILE * TILE, start[b] + count[b], TILE):
                lo, hi = max(start[b], t0), min(start[b] + count[b], t0 + TILE)
                if hi <= lo:
                    continue
                row = table[b][t0 // TILE] * H
                for side, x in ((0, k), (1, s["v"])):
                    x = x[b, :, lo - start[b]:hi - start[b]].double()                  # [H][m][d]
                    e = torch.tensor([min(E_MAX, max(E_MIN, math.ceil(math.log2(a / 448)) if a > 0 else E_MIN))
                                      for a in x.abs().amax((1, 2)).tolist()], device=q.device, dtype=torch.float64)
                    if lo > t0:
                        was = torch.log2(scales[row:row + H, side]).round()
                        e = torch.maximum(e, was)
                        p = places[side, : lo - t0].reshape(-1)
                        codes[row:row + H, p] = _round64(codes[row:row + H, p] * torch.exp2(was - e)[:, None])
                    p = places[side, lo - t0:hi - t0].reshape(-1)
                    codes[row:row + H, p] = _round64(x.reshape(H, -1) * torch.exp2(-e)[:, None])
                    scales[row:row + H, side] = torch.exp2(e)
        return {"q": q, "codes": codes, "scales": scales}
    value = torch.from_numpy(_values64()).to(s["q"].device)
    places = torch.from_numpy(_places64(d)).to(s["q"].device)
    G, nq = c["Hq"] // H, c["nq"]
    start, count = _lengths(c)
    out = torch.zeros(B, nq, H * G, d, dtype=torch.float64, device=s["q"].device)
    for b in range(B):
        T, k = start[b], count[b]
        if T == 0 or k == 0:
            continue
        pages = s["table"][b, : -(-T // TILE)].long()
        limit = torch.arange(T - k + 1, T + 1, device=out.device).repeat_interleave(G)
        for h in range(H):
            block = s["pool"][pages * H + h]
            scale = block[:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
            K, V = (value[block[:, places[i]].long()].mul_(scale[:, i, None, None]).reshape(-1, d)[:T] for i in (0, 1))
            p = (s["q"][b, :k, h * G:(h + 1) * G].reshape(k * G, d).double() @ K.T).div_(math.sqrt(d))
            p.masked_fill_(torch.arange(T, device=out.device)[None] >= limit[:, None], -math.inf)
            p = p.sub_(p.amax(-1, keepdim=True)).exp_()
            out[b, :k, h * G:(h + 1) * G] = ((p @ V) / p.sum(-1, keepdim=True)).view(k, G, d)
    return out
