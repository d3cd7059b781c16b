"""Timed cases of verifying trees of drafted tokens over the 8-bit paged KV cache, and of reading that cache
back: the ancestor masks and positions of a tree (``draft_tree``), the attention of its drafts
(``PagedByteCache.attention`` with ``tree``), the move of the accepted ones to where a plain decode would have
put them (``PagedByteCache.keep``), and the values of whole batches (``PagedByteCache.read``).

A case is a dict of plain values.  ``run`` computes it in plain torch operations where ``own`` is false, and
through the package where it is true; ``exact`` computes it again in 64 bits from the definitions alone.

Definitions.
  tree      draft i of an entry has a parent in [-1, i); -1 is the sequence before the drafts.  Bit j of its
            mask (32 to a word) is set where j is i or one of its ancestors; its position is start + the number
            of its ancestors.  Drafts past the entry's count have no bits and the position start.
  attention the c drafts of an entry are the last c tokens of its sequence: draft i attends to the first
            len - c tokens and to those of the last c whose bit is set.  Rows past c, and rows that attend to
            nothing, are zeros.
  keep      the token at start + path[j] moves to start + j, for j < count.  The scale exponent of a block
            becomes the largest among those of the blocks that its 16 tokens come from, and every code is
            rounded to it.
  read      token j of an entry is the one at start + j; rows past the entry's count are zeros.
  block     16 tokens of one KV head and side have e4m3 codes and a scale 2^e.  K codes in 128-byte rows (64 at
            head dim 64) whose 16-byte chunks are exchanged by the row's index, V codes transposed to [d][16]
            with tokens 2t, 2t+1, 2t+8, 2t+9 side by side, then the scales of K and V (fp32) and 24 bytes of
            padding.  Block (page, head) is page * heads + head.
"""

import math
import random

import numpy as np
import torch

own = False

TILE = 16
TOP = 448.0  # the largest e4m3 value
E_MIN, E_MAX = -30, 30
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one sequence's small tree, made anew each step: latency
        dict(name="tree of one", op="tree", B=1, n=8, reach=4, ragged=False),
        # a full serving batch with wide trees of unlike sizes
        dict(name="tree batch", op="tree", B=256, n=250, reach=40, ragged=True),
        # eight drafts after a short prompt: latency
        dict(name="attention short", op="attention", B=1, n=8, T=1024, Hq=32, Hkv=8, d=128, dtype="bf16", reach=4, ragged=False),
        # the headline batch of 8 sequences with trees of 16 drafts
        dict(name="attention step", op="attention", B=8, n=16, T=32768, Hq=32, Hkv=8, d=128, dtype="bf16", reach=8, ragged=False),
        # one long sequence, a wide tree, eight queries to a KV head
        dict(name="attention long", op="attention", B=1, n=32, T=131072, Hq=64, Hkv=8, d=128, dtype="bf16", reach=12, ragged=False),
        # a serving batch of unlike lengths and trees, some of them empty, seven queries to a KV head
        dict(name="attention ragged", op="attention", B=64, n=13, T=9001, Hq=28, Hkv=4, d=128, dtype="f16", reach=5, ragged=True),
        # small heads, a tree of 24
        dict(name="attention small heads", op="attention", B=16, n=24, T=16384, Hq=16, Hkv=2, d=64, dtype="bf16", reach=6, ragged=False),
        # fp32 queries, three drafts a sequence
        dict(name="attention fp32", op="attention", B=8, n=3, T=8192, Hq=32, Hkv=8, d=128, dtype="f32", reach=2, ragged=False),
        # the accepted path of each sequence of the headline batch
        dict(name="keep step", op="keep", B=8, n=16, m=5, Hkv=8, d=128, start=1000, ragged=True),
        # a large batch with long accepted paths
        dict(name="keep batch", op="keep", B=256, n=64, m=20, Hkv=8, d=128, start=1000, ragged=True),
        # a block or two of each of a few sequences: what a check of the stored values reads
        dict(name="read short", op="read", B=4, n=21, Hkv=2, d=64, dtype="f32", start=37, ragged=True),
        # whole prompts on their way to another cache
        dict(name="read prompts", op="read", B=8, n=32768, Hkv=8, d=128, dtype="bf16", start=0, ragged=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.999)))))))


def draw(rng):
    op = rng.choice(["tree", "attention", "attention", "attention", "keep", "read"])
    Hq, Hkv = rng.choice([(32, 8), (64, 8), (8, 8), (16, 2), (28, 4), (12, 4), (6, 1), (5, 5)])
    d = rng.choice([64, 128, 128, 128, 256])
    B, ragged = _log(rng, 1, 64), rng.random() < 0.5
    if op == "tree":
        return dict(op=op, B=_log(rng, 1, 256), n=_log(rng, 1, 250), reach=_log(rng, 1, 40), ragged=ragged)
    if op == "attention":
        n, T = _log(rng, 1, 64), _log(rng, 64, 131072)
        while B > 1 and (B * T * Hkv * d > 1 << 28 or B * T * Hq * n > 1 << 28):
            B //= 2
        while T > 64 and (B * T * Hkv * d > 1 << 28 or B * T * Hq * n > 1 << 28):
            T = max(64, T // 2)
        return dict(op=op, B=B, n=n, T=T, Hq=Hq, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]),
                    reach=_log(rng, 1, 16), ragged=ragged)
    if op == "keep":
        n = _log(rng, 1, 64)
        return dict(op=op, B=B, n=n, m=rng.randint(1, max(1, n // 3)), Hkv=Hkv, d=d, start=rng.randrange(0, 2000), ragged=ragged)
    n = _log(rng, 1, 32768)
    while B > 1 and B * n * Hkv * d > 1 << 28:
        B //= 2
    return dict(op=op, B=B, n=n, Hkv=Hkv, d=d, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), start=rng.randrange(0, 700),
                ragged=ragged)


def _counts(c):
    """Host lists: (lengths or starts, counts) of the entries."""
    r = random.Random(c["B"] * 1000003 + c.get("T", 0) * 17 + c["n"])
    B, n = c["B"], c["n"]
    if c["op"] == "attention":
        if not c["ragged"]:
            return [c["T"]] * B, [n] * B
        seq = [0 if r.random() < 0.08 else _log(r, 1, c["T"]) for _ in range(B)]
        return seq, [min(s, r.randrange(1, n + 1)) for s in seq]
    first = [c.get("start", 100) + (r.randrange(0, 64) if c["ragged"] else 0) for _ in range(B)]
    if c["op"] == "keep":
        return first, [r.randrange(1, c["m"] + 1) if c["ragged"] else c["m"] for _ in range(B)]
    return first, [r.randrange(0, n + 1) if c["ragged"] else n for _ in range(B)]


def _parents(c, seed):
    """Host [B][n]: a draft's parent is one of the `reach` before it; the first has none."""
    r = np.random.RandomState(int(seed) % (1 << 31))
    back = r.randint(1, c["reach"] + 1, (c["B"], c["n"]))
    return np.maximum(np.arange(c["n"])[None] - back, np.where(np.arange(c["n"]) == 0, -1, 0)[None]).astype(np.int32)


def _path(c, seed):
    """Host [B][m]: the accepted drafts.  Those that move come from behind every place that receives one (and,
    where the places are in several blocks, from blocks behind those), as from a tree whose first levels are
    wider than the path is long: a pass that is made again finds its tokens where they were."""
    r = np.random.RandomState(int(seed) % (1 << 31))
    first, m = _counts(c)[0], c["m"]
    got = np.zeros((c["B"], m), dtype=np.int32)
    for b in range(c["B"]):
        j = np.arange(c["n"])
        lo, hi = first[b] // TILE, (first[b] + m - 1) // TILE
        free = j[(j >= m) & ((first[b] + j) // TILE > hi)] if hi > lo else j[m:]
        stay = max(m - len(free), r.randint(0, m + 1))
        got[b, :stay] = np.arange(stay)
        got[b, stay:] = np.sort(r.permutation(free)[:m - stay])
    return got


def work(case):
    c = case
    first, count = _counts(c)
    if c["op"] == "tree":
        return {"bytes": 4 * c["B"] * c["n"] * (2 + (c["n"] + 31) // 32) + 8 * c["B"], "flops": 0}
    if c["op"] == "keep":
        return {"bytes": 2 * sum(count) * c["Hkv"] * 2 * c["d"] + 4 * c["B"] * (c["m"] + 3), "flops": 0}
    if c["op"] == "read":
        return {"bytes": 2 * c["Hkv"] * c["d"] * (sum(count) + c["B"] * c["n"] * SIZE[c["dtype"]]),
                "flops": 2 * sum(count) * c["Hkv"] * c["d"]}
    rows = sum((s - k) * k + k for s, k in zip(first, count))  # (a draft sees itself at least)
    pool = sum(first) * c["Hkv"] * (2 * c["d"] + 8 / TILE)
    return {"bytes": pool + 2 * c["B"] * c["n"] * c["Hq"] * c["d"] * SIZE[c["dtype"]] + 4 * c["B"] * c["n"] * ((c["n"] + 31) // 32),
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

def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 29)
    B, n = c["B"], c["n"]
    s = {"c": c}
    first, count = _counts(c)
    ints = {"dtype": torch.int32, "device": dev}
    s["count"] = torch.tensor(count, **ints)
    if c["op"] == "tree":
        s["parents"] = torch.from_numpy(_parents(c, seed)).to(dev)
        s["start"] = torch.randint(0, 32768, (B,), generator=gen, device=dev, dtype=torch.int32)
        return s

    d, Hkv = c["d"], c["Hkv"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    last = c["T"] if c["op"] == "attention" else max(first) + n  # tokens of the longest sequence
    blocks = max(1, -(-last // TILE))
    pages = B * blocks + 3
    order = torch.randperm(pages, generator=gen, device=dev)[: B * blocks]
    s["table"] = order.view(B, blocks).to(torch.int32).contiguous()
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
    if c["op"] == "attention":
        s["seq"] = torch.tensor(first, **ints)
        s["q"] = normal(B, n, c["Hq"], d).to(DTYPES[c["dtype"]])
        s["parents"] = torch.from_numpy(_parents(c, seed)).to(dev)
        s["tree"] = _tree(s["parents"], s["count"], torch.zeros_like(s["count"]))[0]
        # what lies behind a sequence's last token is anything, NaN codes among it
        seq = s["seq"].long()
        page = s["table"].long().gather(1, ((seq - 1).clamp(min=0) // TILE)[:, None])[:, 0]
        rows = (page[:, None] * Hkv + torch.arange(Hkv, device=dev)).reshape(-1)
        behind = torch.arange(TILE, device=dev)[None] >= ((seq - 1) % TILE + 1)[:, None]
        behind = behind.repeat_interleave(Hkv, 0)[:, :, None].expand(-1, -1, d).reshape(len(rows), -1)
        for places in (_k_places(d, dev), _v_places(d, dev)):
            p = places.reshape(-1)
            pool[rows[:, None], p[None]] = torch.where(behind, torch.full_like(pool[:1, :1], 127), pool[rows[:, None], p[None]])
    else:
        s["start"] = torch.tensor(first, **ints)
    if c["op"] == "keep":
        s["path"] = torch.from_numpy(_path(c, seed)).to(dev)
        # blocks that drafts have raised: scales of unlike size next to each other
        up = torch.exp2(torch.randint(0, 4, (pool.shape[0], 2), generator=gen, device=dev).float())
        scale = pool[:, 32 * d:32 * d + 8].contiguous().view(torch.float32)
        pool[:, 32 * d:32 * d + 8] = (scale * up).view(torch.uint8)
    s["pool"], s["pages"] = pool, pages
    if own:
        from turboquant_quantized_kv_tq_gb300 import PagedByteCache
        s["cache"] = PagedByteCache(d, c.get("Hq", Hkv), Hkv, pages, blocks)
        s["cache"].pool.copy_(pool.view(-1))
        s["pool"] = s["cache"].pool.view(pool.shape)
    return s


# ---------------------------------------------------------------- the plain forms

def _tree(parents, count, start):
    """int32 masks [B][n][words] and positions [1][B][n]."""
    B, n = parents.shape
    dev = parents.device
    i = torch.arange(n, device=dev)
    live = i[None] < count[:, None]
    reach = (parents[:, :, None] == i) | torch.eye(n, dtype=torch.bool, device=dev)
    for _ in range((n - 1).bit_length()):  # ancestors of ancestors
        reach = torch.matmul(reach.float(), reach.float()) > 0
    reach &= live[:, :, None]
    words = (n + 31) // 32
    bits = torch.zeros(B, n, 32 * words, dtype=torch.int64, device=dev)
    bits[:, :, :n] = reach
    masks = (bits.view(B, n, words, 32) << torch.arange(32, device=dev)).sum(-1)
    masks = torch.where(masks >= 1 << 31, masks - (1 << 32), masks).to(torch.int32)
    depth = (reach.sum(-1) - 1).clamp(min=0)
    return masks, (start[:, None] + depth).to(torch.int32)[None]


def _attention(s):
    c, dev = s["c"], s["q"].device
    d, n, B, H, G = c["d"], c["n"], c["B"], c["Hkv"], c["Hq"] // c["Hkv"]
    seq, count = s["seq"].long(), s["count"].long()
    blocks = s["table"].shape[1]
    rows = (s["table"].long()[:, None] * H + torch.arange(H, device=dev)[None, :, None]).reshape(-1)
    valid = torch.arange(blocks * TILE, device=dev)[None] < seq[:, None]
    scales = s["pool"][:, 32 * d:32 * d + 8].contiguous().view(torch.float32)[rows].view(B, H, blocks, 1, 1, 2)

    def side(places, k):
        x = _decode(s["pool"][rows[:, None], places.reshape(-1)[None]]).view(B, H, blocks, TILE, d)
        x = (x * scales[..., k]).view(B, H, blocks * TILE, d)
        return x.masked_fill_(~valid[:, None, :, None], 0.0)

    q = s["q"].to(torch.float32).view(B, n, H, G, d).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, d)
    score = torch.matmul(q, side(_k_places(d, dev), 0).transpose(-1, -2)).mul_(d ** -0.5)
    # draft j of each token (negative: a token before the drafts), and whether draft i attends to it
    j = torch.arange(blocks * TILE, device=dev)[None] - (seq - count)[:, None]
    at = j.clamp(0, n - 1)
    word = s["tree"].long().gather(2, (at // 32)[:, None].expand(B, n, -1))
    sees = (j < 0)[:, None] | ((word >> (at % 32)[:, None]) & 1).bool()
    sees &= (torch.arange(n, device=dev)[None] < count[:, None])[:, :, None] & valid[:, None]
    score.masked_fill_(~sees.repeat_interleave(G, 1)[:, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    p = score.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, side(_v_places(d, dev), 1)) / total.masked_fill(total == 0, 1.0)
    return o.view(B, H, n, G, d).permute(0, 2, 1, 3, 4).reshape(B, n, H * G, d).to(s["q"].dtype)


def _keep(s):
    c, dev = s["c"], s["path"].device
    d, m, B, H = c["d"], c["m"], c["B"], c["Hkv"]
    start, count, path = s["start"].long(), s["count"].long(), s["path"].long()
    nb = (TILE - 1 + c["n"] + TILE - 1) // TILE                       # blocks that the drafts touch, at most
    at = (start // TILE)[:, None] + torch.arange(nb, device=dev)
    page = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    page = torch.where(at < s["table"].shape[1], page, torch.full_like(page, s["pages"]))
    rows = (page[:, None] * H + torch.arange(H, device=dev)[None, :, None]).reshape(-1)   # [B][H][nb]
    block = s["pool"][rows]
    e = torch.frexp(block[:, 32 * d:32 * d + 8].contiguous().view(torch.float32))[1].view(B, H, nb, 2) - 1
    place = torch.arange(nb * TILE, device=dev)[None]
    j = place - (start % TILE)[:, None]
    kept = (j >= 0) & (j < count[:, None])
    source = torch.where(kept, (start % TILE)[:, None] + path.gather(1, j.clamp(0, m - 1)), place)   # [B][nb 16]
    gets = kept.view(B, 1, nb, TILE).any(-1)
    for side, places in ((0, _k_places(d, dev)), (1, _v_places(d, dev))):
        p = places.reshape(-1)
        was = block[:, p].view(B, H, nb * TILE, d)
        codes = was.gather(2, source[:, None, :, None].expand(B, H, nb * TILE, d))
        from_e = e[..., side].gather(2, (source // TILE)[:, None].expand(B, H, nb * TILE)).view(B, H, nb, TILE)
        top = from_e.amax(-1)
        moved = _encode(torch.ldexp(_decode(codes).view(B, H, nb, TILE, d), (from_e - top[..., None])[..., None]))
        block[:, p] = torch.where(gets[..., None, None], moved, was.view(B, H, nb, TILE, d)).view(-1, TILE * d)
        block[:, 32 * d + 4 * side:32 * d + 4 * side + 4] = torch.ldexp(torch.ones_like(top, dtype=torch.float32), top).view(-1, 1).view(torch.uint8)
    s["pool"][rows] = block
    return (start + count).to(torch.int32)


def _read(s):
    c, dev = s["c"], s["start"].device
    d, n, B, H, out = c["d"], c["n"], c["B"], c["Hkv"], DTYPES[c["dtype"]]
    nb = (TILE - 1 + n + TILE - 1) // TILE
    at = (s["start"].long() // TILE)[:, None] + torch.arange(nb, device=dev)
    page = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    rows = (page[:, None] * H + torch.arange(H, device=dev)[None, :, None]).reshape(-1)   # [B][H][nb]
    scales = s["pool"][:, 32 * d:32 * d + 8].contiguous().view(torch.float32)[rows].view(B, H, nb, 1, 1, 2)
    place = (s["start"].long() % TILE)[:, None] + torch.arange(n, device=dev)
    live = torch.arange(n, device=dev)[None] < s["count"][:, None]

    def side(places, k):
        x = _decode(s["pool"][rows[:, None], places.reshape(-1)[None]]).view(B, H, nb, TILE, d)
        x = (x * scales[..., k]).view(B, H, nb * TILE, d).gather(2, place[:, None, :, None].expand(B, H, n, d))
        return x.masked_fill_(~live[:, None, :, None], 0.0).to(out)

    return side(_k_places(d, dev), 0), side(_v_places(d, dev), 1)


def run(state):
    s = state
    c = s["c"]
    if c["op"] == "tree":
        if own:
            from turboquant_quantized_kv_tq_gb300 import draft_tree
            masks, positions = draft_tree(s["parents"], start=s["start"], count=s["count"])
        else:
            masks, positions = _tree(s["parents"], s["count"], s["start"])
        return {"masks": masks, "positions": positions}
    if c["op"] == "attention":
        if own:
            return s["cache"].attention(s["q"], s["seq"], s["table"], count=s["count"], tree=s["tree"])
        return _attention(s)
    if c["op"] == "keep":
        if own:
            length = s["cache"].keep(s["path"], s["start"], s["table"], count=s["count"])
        else:
            length = _keep(s)
        d = c["d"]
        return {"length": length, "codes": s["pool"][:, : 32 * d].view(torch.float8_e4m3fn),
                "scales": s["pool"][:, 32 * d:32 * d + 8].view(torch.float32)}
    if own:
        k, v = s["cache"].read(s["start"], s["table"], c["n"], count=s["count"], dtype=DTYPES[c["dtype"]])
    else:
        k, v = _read(s)
    return {"k": k, "v": v}


# ---------------------------------------------------------------- 64 bits, from the definitions

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
    B, n = c["B"], c["n"]
    if c["op"] == "tree":
        parents, count, start = (s[k].cpu().tolist() for k in ("parents", "count", "start"))
        masks = np.zeros((B, n, (n + 31) // 32), dtype=np.uint32)
        positions = np.repeat(np.array(start, dtype=np.int32)[:, None], n, 1)[None]
        for b in range(B):
            for i in range(count[b]):
                up = parents[b][i]
                if up >= 0:
                    masks[b, i] = masks[b, up]
                    positions[0, b, i] = positions[0, b, up] + 1
                masks[b, i, i // 32] |= np.uint32(1 << (i % 32))
        return {"masks": masks.view(np.int32), "positions": positions}
    H, d = c["Hkv"], c["d"]
    first, count = _counts(c)
    dev = s["pool"].device
    value = torch.from_numpy(_values64()).to(dev)
    places = torch.from_numpy(_places64(d)).to(dev)
    table = s["table"].cpu().tolist()
    if c["op"] == "keep":
        codes = value[s["pool"][:, : 32 * d].long()]
        scales = s["pool"][:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
        path = s["path"].cpu().tolist()
        for b in range(B):
            for t0 in range(first[b] // TILE * TILE, first[b] + count[b], TILE):
                taken = [t - first[b] for t in range(t0, t0 + TILE)]
                taken = [first[b] + path[b][j] if 0 <= j < count[b] else first[b] + j for j in taken]
                # [H][16]: the blocks that the tokens come from
                rows = torch.tensor([[table[b][t // TILE] * H + h for t in taken] for h in range(H)], device=dev)
                row = table[b][t0 // TILE] * H
                slot = torch.tensor(taken, device=dev) % TILE
                for side in (0, 1):
                    size = scales[rows, side]
                    top = size.amax(1)
                    x = codes[rows[:, :, None], places[side, slot][None]] * (size / top[:, None])[:, :, None]
                    codes[row:row + H, places[side].reshape(-1)] = _round64(x).view(H, TILE * d)
                    scales[row:row + H, side] = top
        return {"length": np.array([a + k for a, k in zip(first, count)], dtype=np.int32), "codes": codes, "scales": scales}
    if c["op"] == "read":
        out = torch.zeros(2, B, H, n, d, dtype=torch.float64, device=dev)
        scales = s["pool"][:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
        for b in range(B):
            t = torch.arange(first[b], first[b] + count[b], device=dev)
            pages = s["table"][b].long()[t // TILE]
            for h in range(H):
                rows = pages * H + h
                for side in (0, 1):
                    out[side, b, h, :count[b]] = value[s["pool"][rows[:, None], places[side, t % TILE]].long()] * scales[rows, side][:, None]
        return {"k": out[0], "v": out[1]}
    G = c["Hq"] // H
    parents = s["parents"].cpu().tolist()
    out = torch.zeros(B, n, H * G, d, dtype=torch.float64, device=dev)
    for b in range(B):
        T, k = first[b], count[b]
        if T == 0 or k == 0:
            continue
        sees = np.ones((k, T), dtype=bool)
        sees[:, T - k:] = False
        for i in range(k):
            up = i
            while up >= 0:
                sees[i, T - k + up] = True
                up = parents[b][up]
        blind = torch.from_numpy(~sees).to(dev).repeat_interleave(G, 0)
        pages = s["table"][b, : -(-T // TILE)].long()
        for h in range(H):
            block = s["pool"][pages * H + h]
            scale = block[:, 32 * d:32 * d + 8].contiguous().view(torch.float32).double()
            K, V = (value[block[:, places[i]].long()].mul_(scale[:, i, None, None]).reshape(-1, d)[:T] for i in (0, 1))
            p = (s["q"][b, :k, h * G:(h + 1) * G].reshape(k * G, d).double() @ K.T).div_(math.sqrt(d))
            p.masked_fill_(blind, -math.inf)
            p = p.sub_(p.amax(-1, keepdim=True)).exp_()
            out[b, :k, h * G:(h + 1) * G] = ((p @ V) / p.sum(-1, keepdim=True)).view(k, G, d)
    return out
