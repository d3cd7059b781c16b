"""Plain forms of drafted trees over the byte cache (numpy, float64; shares no code with the package)."""

import numpy as np

import byte_reference as ref

TILE = ref.TILE


def masks_positions(parents, count, start):
    """([B][n][n] bool, [B][n]) of parents [B][n]: which drafts each sees, and its position."""
    B, n = parents.shape
    sees, pos = np.zeros((B, n, n), dtype=bool), np.repeat(np.asarray(start)[:, None], n, 1).astype(np.int64)
    for b in range(B):
        for i in range(min(n, max(0, count[b]))):
            up, chain = i, []
            while up >= 0:
                chain.append(up)
                p = int(parents[b, up])
                if p < -1 or p >= up:
                    break
                up = p
            if up == -1:
                sees[b, i, chain] = True
                pos[b, i] += len(chain) - 1
    return sees, pos


def pack(sees):
    """int32 [B][n][words] of bool [B][n][n]."""
    B, n, _ = sees.shape
    words = (n + 31) // 32
    bits = np.zeros((B, n, 32 * words), dtype=np.uint64)
    bits[:, :, :n] = sees
    w = (bits.reshape(B, n, words, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def attention(q, pool, seq, cnt, table, scale, sees, step=0.0):
    """q: float64 [B][nq][Hq][d] -> (out, spread, reach, least) as byte_reference.attention's and attention_least's: what
    attention may lose where its weights have a smallest step of `step` times the row's largest."""
    B, nq, Hq, d = q.shape
    G = Hq // pool.heads
    out, spread, reach, least = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3]), np.zeros(q.shape)
    for b in range(B):
        pages = table[b][:(seq[b] + TILE - 1) // TILE]
        c = min(nq, max(0, cnt[b]))
        who = np.zeros((c, seq[b]), dtype=bool)
        for t in range(seq[b]):
            j = t - (seq[b] - c)
            who[:, t] = True if j < 0 else sees[b, :c, j]
        for h in range(pool.heads):
            K, V = pool.read(0, h, pages, seq[b]), pool.read(1, h, pages, seq[b])
            size = np.repeat([float(pool.scale(p, h, 1)) for p in pages], TILE)[:seq[b]]
            for i in range(c):
                if not who[i].any():
                    continue
                k, v = K[who[i]], V[who[i]]
                x = q[b, i, h * G:(h + 1) * G]
                s = scale * (x @ k.T)
                p = np.exp(s - s.max(-1, keepdims=True))
                p /= p.sum(-1, keepdims=True)
                out[b, i, h * G:(h + 1) * G] = p @ v
                spread[b, i, h * G:(h + 1) * G] = p @ np.abs(v)
                reach[b, i, h * G:(h + 1) * G] = abs(scale) * (np.abs(x) @ np.abs(k).T).max(-1)
                w = p * size[who[i]]
                off = np.minimum(step / 2 * w.max(-1, keepdims=True), w)
                least[b, i, h * G:(h + 1) * G] = off @ (np.abs(v) / size[who[i], None])
    return out, spread, reach, least


def keep(pool, path, start, cnt, table):
    """Moves the tokens in `pool` (byte_reference.Pool); an entry whose path does not rise stays."""
    was = pool.blocks.copy()
    old = ref.Pool(was, pool.heads, pool.d)
    n = path.shape[1]
    for b in range(path.shape[0]):
        c = min(n, max(0, cnt[b]))
        way = [int(x) for x in path[b, :c]]
        if c and (start[b] < 0 or way[0] < 0 or any(y <= x for x, y in zip(way, way[1:]))):
            continue
        for t0 in range(start[b] // TILE * TILE, start[b] + c, TILE):
            src = [start[b] + way[t - start[b]] if 0 <= t - start[b] < c else t for t in range(t0, t0 + TILE)]
            if src == list(range(t0, t0 + TILE)):
                continue
            page = table[b][t0 // TILE]
            for h in range(pool.heads):
                for side in (0, 1):
                    e = [int(round(np.log2(old.scale(table[b][t // TILE], h, side)))) for t in src]
                    top = max(e)
                    for s, t in enumerate(src):
                        codes = old.blocks[table[b][t // TILE], h][old.at[side, t % TILE]]
                        if e[s] != top:
                            codes = ref.e4m3_encode(ref.VALUES[codes] * 2.0 ** (e[s] - top))
                        pool.blocks[page, h, pool.at[side, s]] = codes
                    pool.set_scale(page, h, side, top)


def read(pool, start, cnt, n, table):
    """float64 (k, v) [B][heads][n][d]."""
    B = len(start)
    out = np.zeros((2, B, pool.heads, n, pool.d))
    for b in range(B):
        for j in range(min(n, max(0, cnt[b]))):
            t = start[b] + j
            page = table[b][t // TILE]
            for h in range(pool.heads):
                for side in (0, 1):
                    out[side, b, h, j] = ref.VALUES[pool.blocks[page, h][pool.at[side, t % TILE]]] * float(pool.scale(page, h, side))
    return out[0], out[1]
