"""Plain float64 forms of the byte cache, the head norms and the position rotation (numpy; shares no
code with the package): block layout, e4m3 rounding, appends with block scales, attention."""

import numpy as np

TILE = 16


def e4m3_values():
    """Value of each byte (NaN for 0x7f, 0xff)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where(b & 128, -v, v)
    v[[127, 255]] = np.nan
    return v


VALUES = e4m3_values()


def e4m3_encode(x):
    """Nearest e4m3 byte of float64 x (ties to even, saturating; NaN gives 0)."""
    x = np.asarray(x, dtype=np.float64)
    pos = VALUES[:127]
    a = np.minimum(np.abs(np.nan_to_num(x, nan=0.0, posinf=448.0, neginf=-448.0)), 448.0)
    hi = np.clip(np.searchsorted(pos, a, side="left"), 1, 126)
    lo = hi - 1
    up = (a - pos[lo] > pos[hi] - a) | ((a - pos[lo] == pos[hi] - a) & (hi % 2 == 0))
    code = np.where(up, hi, lo)
    return np.where(np.signbit(x) & ~np.isnan(x), code | 128, code).astype(np.uint8)


def need(amax):
    """Smallest e in [-30, 30] with amax <= 448 2^e."""
    for e in range(-30, 31):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return 30


def places(d):
    """[2][16][d]: byte of the K and V code of each token and coordinate of a block."""
    t, x = np.meshgrid(np.arange(TILE), np.arange(d), indexing="ij")
    c = x // 16
    if d == 64:
        k = 64 * t + 16 * (c ^ ((t // 2) % 4)) + x % 16
    else:
        k = 2048 * (c // 8) + 128 * t + 16 * ((c % 8) ^ (t % 8)) + x % 16
    v = 16 * d + 16 * x + 4 * ((t % 8) // 2) + 2 * (t // 8) + t % 2
    return np.stack([k, v])


class Pool:
    """The pool's bytes as [pages + 1][heads][block]."""

    def __init__(self, raw, heads, d):
        self.heads, self.d, self.at = heads, d, places(d)
        self.blocks = np.array(raw, dtype=np.uint8).reshape(-1, heads, 32 * d + 32)

    def scale(self, page, h, side):
        s = 32 * self.d + 4 * side
        return self.blocks[page, h, s:s + 4].copy().view(np.float32)[0]

    def set_scale(self, page, h, side, e):
        s = 32 * self.d + 4 * side
        self.blocks[page, h, s:s + 4] = np.array([2.0 ** e], dtype=np.float32).view(np.uint8)

    def append(self, side, x, start, table, count=None):
        """x: float64 [B][heads][n][d]."""
        B, H, n, d = x.shape
        for b in range(B):
            m = n if count is None else min(n, max(0, count[b]))
            for t0 in range(start[b] // TILE * TILE, start[b] + m, TILE):
                lo, hi = max(start[b], t0), min(start[b] + m, t0 + TILE)
                if hi <= lo:
                    continue
                page = table[b][t0 // TILE]
                for h in range(H):
                    new = x[b, h, lo - start[b]:hi - start[b]]
                    fin = np.abs(new[np.isfinite(new)])
                    e = need(fin.max() if fin.size else 0.0)
                    blk = self.blocks[page, h]
                    if lo > t0:
                        was = int(round(np.log2(self.scale(page, h, side))))
                        if was > e:
                            e = was
                        p = self.at[side, :lo - t0]
                        blk[p] = e4m3_encode(VALUES[blk[p]] * 2.0 ** (was - e))
                    blk[self.at[side, lo - t0:hi - t0]] = e4m3_encode(new * 2.0 ** -e)
                    self.set_scale(page, h, side, e)

    def read(self, side, h, pages, n):
        """Float64 [n][d]: the first n tokens of a sequence."""
        out = [VALUES[self.blocks[p, h][self.at[side]]] * float(self.scale(p, h, side)) for p in pages]
        return np.concatenate(out)[:n] if out else np.zeros((0, self.d))


def norm_rotate(x, w, eps, freqs, axis_of, interleaved, pos):
    """x: float64 [..., n, d] with pos [axes][n] -> (y, bound): bound[i] >= |a| + |b| of y_i's pair after the norm."""
    if w is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    y, size = x.copy(), np.abs(x)
    r = 2 * len(freqs) if freqs is not None else 0
    for i in range(r // 2):
        t = pos[axis_of[i]].astype(np.float64) * freqs[i]
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        y[..., a] = x[..., a] * np.cos(t) - x[..., b] * np.sin(t)
        y[..., b] = x[..., a] * np.sin(t) + x[..., b] * np.cos(t)
        size[..., a] = size[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, size


def attention(q, pool, seq, cnt, table, scale):
    """q: float64 [B][nq][Hq][d] -> (out, spread, reach): spread = sum p |v| / sum p per coordinate,
    reach [B][nq][Hq] = scale * the largest sum |q||k| of the row."""
    B, nq, Hq, d = q.shape
    G = Hq // pool.heads
    out, spread, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3])
    for b in range(B):
        pages = table[b][:(seq[b] + TILE - 1) // TILE]
        for h in range(pool.heads):
            K, V = pool.read(0, h, pages, seq[b]), pool.read(1, h, pages, seq[b])
            for i in range(min(nq, max(0, cnt[b]))):
                m = seq[b] - cnt[b] + 1 + i
                if m <= 0:
                    continue
                x = q[b, i, h * G:(h + 1) * G]
                s = scale * (x @ K[:m].T)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[b, i, h * G:(h + 1) * G] = p @ V[:m]
                spread[b, i, h * G:(h + 1) * G] = p @ np.abs(V[:m])
                reach[b, i, h * G:(h + 1) * G] = abs(scale) * (np.abs(x) @ np.abs(K[:m]).T).max(-1)
    return out, spread, reach


def attention_least(q, pool, seq, cnt, table, scale, step):
    """[B][nq][Hq][d]: what attention may lose where its weights are stored with a smallest step.

    A token of a value block with scale 2^e enters as w = p 2^e times its code.  Stored to half a step of
    step * (the row's largest w), a w is off by at most that, and by no more than w itself where it becomes
    zero: sum over the tokens of min(step / 2 * max w, w) |code|."""
    B, nq, Hq, d = q.shape
    G = Hq // pool.heads
    least = np.zeros(q.shape)
    for b in range(B):
        pages = table[b][:(seq[b] + TILE - 1) // TILE]
        for h in range(pool.heads):
            K, V = pool.read(0, h, pages, seq[b]), pool.read(1, h, pages, seq[b])
            size = np.repeat([float(pool.scale(p, h, 1)) for p in pages], TILE)[:seq[b]]
            for i in range(min(nq, max(0, cnt[b]))):
                m = seq[b] - cnt[b] + 1 + i
                if m <= 0:
                    continue
                s = scale * (q[b, i, h * G:(h + 1) * G] @ K[:m].T)
                p = np.exp(s - s.max(-1, keepdims=True))
                w = p / p.sum(-1, keepdims=True) * size[:m]
                off = np.minimum(step / 2 * w.max(-1, keepdims=True), w)
                least[b, i, h * G:(h + 1) * G] = off @ (np.abs(V[:m]) / size[:m, None])
    return least
