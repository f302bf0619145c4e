"""The 8-bit key/value cache from its definition, in numpy: appending in f32 with every operation
rounded (the cache's bytes are defined bit by bit), attention in 64 bits.  A sequence at a time,
a block at a time."""
import numpy as np

BLOCK = 32


def rec_bytes(dim):
    return 64 * dim + 16


def split(rec, dim):
    """Views of one record (uint8 [64 * dim + 16]): key codes, value codes, f32 scales [2]."""
    kc = rec[:32 * dim].view(np.int8).reshape(BLOCK, dim)
    vc = rec[32 * dim:64 * dim].view(np.int8).reshape(BLOCK, dim)
    return kc, vc, rec[64 * dim:64 * dim + 8].view(np.float32)


def record(data, table, b, blk, h):
    """The record of block blk of sequence b, head h (data: [pages, heads, blocks, bytes])."""
    nb = data.shape[2]
    return data[table[b, blk // nb], h, blk % nb]


def rotate(x, pos, cos, sin, interleaved):
    """x f32 [dim] at position pos; cos, sin f32 [positions, rotary / 2]."""
    r = 2 * cos.shape[1]
    y = x.copy()
    i = np.arange(r // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
    c, s = cos[pos], sin[pos]
    y[a] = x[a] * c - x[b] * s
    y[b] = x[b] * c + x[a] * s
    return y


def _codes(x, d):
    if d == 0:
        return np.zeros(x.shape, np.int8)
    return np.clip(np.rint(x / d), -127, 127).astype(np.int8)


def append(data, starts, lens, table, k, v, dim, rope=None):
    """In place.  k, v: f32 [tokens, heads, dim]; rope: (cos, sin, interleaved) or None."""
    for b in range(len(lens)):
        n = starts[b + 1] - starts[b]
        first = lens[b] - n
        for blk in range(max(first, 0) // BLOCK, -(-lens[b] // BLOCK)):
            old = max(0, max(first, 0) - blk * BLOCK)
            at = range(blk * BLOCK + old, min(lens[b], (blk + 1) * BLOCK))
            if len(at) == 0:
                continue
            for h in range(data.shape[1]):
                kc, vc, d = split(record(data, table, b, blk, h), dim)
                rows = [starts[b] + p - first for p in at]
                new_k = np.stack([rotate(k[r, h], p, *rope) if rope else k[r, h] for r, p in zip(rows, at)])
                for w, (codes, x) in enumerate(((kc, new_k), (vc, v[rows, h]))):
                    scale = np.float32(np.abs(x).max() / np.float32(127))
                    if old:
                        scale = max(scale, d[w])
                    if scale < np.float32(2.0 ** -100):
                        scale = np.float32(0)
                    if old and scale != d[w]:
                        ratio = d[w] / scale if scale else np.float32(0)
                        codes[:old] = np.clip(np.rint(codes[:old].astype(np.float32) * ratio), -127, 127).astype(np.int8)
                    codes[old:old + len(at)] = _codes(x, scale)
                    d[w] = scale


def values(data, table, b, n, dim, which, dtype=np.float64):
    """Keys (0) or values (1) of sequence b's first n tokens, [n, heads, dim]."""
    out = np.zeros((n, data.shape[1], dim), dtype)
    for blk in range(-(-n // BLOCK)):
        m = min(BLOCK, n - blk * BLOCK)
        for h in range(data.shape[1]):
            r = split(record(data, table, b, blk, h), dim)
            out[blk * BLOCK:blk * BLOCK + m, h] = r[which][:m].astype(dtype) * dtype(r[2][which])
    return out


def attend(data, starts, lens, table, q, dim, scale, window=0):
    """(out, lse, bound terms) in 64 bits: out [tokens, heads, dim], lse [tokens, heads], the sums
    of |w v| [tokens, heads, dim] and the largest sum of |q k| * scale [tokens, heads] that error
    bounds need.  Rows of no sequence stay NaN."""
    T, H, _ = q.shape
    out, absum = np.full((T, H, dim), np.nan), np.zeros((T, H, dim))
    lse, big = np.full((T, H), np.nan), np.zeros((T, H))
    q = q.astype(np.float64)
    for b in range(len(lens)):
        n = int(starts[b + 1] - starts[b])
        if n == 0:
            continue
        k, v = values(data, table, b, lens[b], dim, 0), values(data, table, b, lens[b], dim, 1)
        G = H // k.shape[1]
        for t in range(n):
            p, row = lens[b] - n + t, starts[b] + t
            lo = max(0, p - window + 1) if window else 0
            for h in range(H):
                if p < 0:
                    out[row, h], lse[row, h] = 0, -np.inf
                    continue
                kk, vv = k[lo:p + 1, h // G], v[lo:p + 1, h // G]
                s = kk @ q[row, h] * scale
                m = s.max()
                w = np.exp(s - m)
                out[row, h], absum[row, h] = w @ vv / w.sum(), w @ np.abs(vv) / w.sum()
                lse[row, h] = m + np.log(w.sum())
                big[row, h] = (np.abs(kk) @ np.abs(q[row, h])).max() * scale
    return out, lse, absum, big
