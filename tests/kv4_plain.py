"""Plain 64-bit forms of the 4-bit K/V cache operators for the GPU tests: the
oracle's scalar C rows on a cache held as plain arrays, and the page layout
written out from the specification (section 16), item by item."""
import numpy as np

import oracle

XMAX = 1785


def rshr(x, s):
    x = np.asarray(x, np.int64)
    return x if s == 0 else (x + (np.int64(1) << (s - 1))) >> s


def sat32(x):
    return np.clip(x, -(2 ** 31 - 1), 2 ** 31 - 1)


def k_place(c):
    """(byte, high nibble) of channel c in a token's K row."""
    return c // 8 * 4 + c % 4, c // 4 % 2


def v_place(c, j):
    """(byte, high nibble) of channel c and key j in a V page."""
    return c // 16 * 512 + c % 8 * 64 + j // 16 * 16 + c // 8 % 2 * 8 + j // 8 % 2 * 4 + j % 4, j // 4 % 2


class Pages:
    """A paged cache as arrays of values, and its packed bytes."""

    def __init__(self, n_blocks, n_kv, d, rng):
        self.n_blocks, self.n_kv, self.d = n_blocks, n_kv, d
        self.k = rng.integers(-7, 8, (n_blocks, n_kv, 64, d)).astype(np.int8)
        self.v = rng.integers(-7, 8, (n_blocks, n_kv, 64, d)).astype(np.int8)
        self.ck = rng.integers(1, 256, (n_blocks, n_kv, 64)).astype(np.uint8)
        self.cv = rng.integers(1, 256, (n_blocks, n_kv, 64)).astype(np.uint8)

    def packed(self):
        d = self.d
        k = np.zeros((self.n_blocks, self.n_kv, 64, d // 2), np.uint8)
        v = np.zeros((self.n_blocks, self.n_kv, 32 * d), np.uint8)
        for c in range(d):
            byte, hi = k_place(c)
            k[..., byte] |= (self.k[..., c] + 8).astype(np.uint8) << (4 * hi)
        c, j = np.meshgrid(np.arange(d), np.arange(64), indexing="ij")
        byte, hi = v_place(c, j)
        for h in (0, 1):
            m = hi == h
            v[:, :, byte[m]] |= (self.v[:, :, j[m], c[m]] + 8).astype(np.uint8) << (4 * h)
        return k, v.reshape(k.shape)


def rope(y, cos, sin, inter):
    """Rotate the first 2 len(cos) channels of one row (saturating to 32 bits)."""
    y = np.asarray(y, np.int64).copy()
    r2 = len(cos)
    a, b = (slice(0, 2 * r2, 2), slice(1, 2 * r2, 2)) if inter else (slice(0, r2), slice(r2, 2 * r2))
    x0, x1, c, s = y[a].copy(), y[b].copy(), np.asarray(cos, np.int64), np.asarray(sin, np.int64)
    y[a], y[b] = rshr(x0 * c - x1 * s, 14), rshr(x1 * c + x0 * s, 14)
    return sat32(y)


def append(pages, table, prm, n_q, cos, sin, inter, gammas, eps, qkv, seq, pos):
    """Appends to `pages` in place; (q8, mq, kq, k_val, v_val)."""
    n_kv, d = pages.n_kv, pages.d
    T = len(pos)
    q8 = np.zeros((T, n_q, d), np.int8)
    mq, kq = np.zeros((T, n_q), np.int32), np.zeros((T, n_q), np.int32)
    kv, vv = np.zeros((T, n_kv, d), np.int16), np.zeros((T, n_kv, d), np.int16)
    max_pos = len(cos)
    for t in range(T):
        if not 0 <= pos[t] < max_pos:
            continue
        rows = qkv[t].reshape(-1, d)

        def head(x, gamma):
            y = oracle.qknorm(x, gamma, eps)[0] if gamma is not None else sat32(np.asarray(x, np.int64) * 4)
            return rope(y, cos[pos[t]], sin[pos[t]], inter)

        for h in range(n_q):
            e = prm[h // (n_q // n_kv), 8:].astype(np.int64)
            y = sat32(head(rows[h], gammas[0]) << (e.max() - e))
            q8[t, h], mq[t, h], kq[t, h] = (a[0] for a in oracle.actquant(y, 14))
        blk = -1
        if 0 <= seq[t] < table.shape[0] and pos[t] // 64 < table.shape[1]:
            blk = table[seq[t], pos[t] // 64]
        if not 0 <= blk < pages.n_blocks:
            continue
        for g in range(n_kv):
            p = prm[g].astype(np.int64)
            xk = np.clip(rshr((head(rows[n_q + g], gammas[1]) << p[8:]) * p[0], p[1]), -XMAX, XMAX)
            xv = np.clip(rshr(rows[n_q + n_kv + g].astype(np.int64) * p[2], p[3]), -XMAX, XMAX)
            for x, codes, scale, val in ((xk, pages.k, pages.ck, kv), (xv, pages.v, pages.cv, vv)):
                q, c = oracle.quant4(x)
                codes[blk, g, pos[t] % 64], scale[blk, g, pos[t] % 64] = q[0], c[0]
                val[t, g] = q[0].astype(np.int16) * c[0]
    return q8, mq, kq, kv, vv


def attention(pages, table, prm, n_q, q8, mq, kq, seq, pos, window=0, max_len=1 << 30, rows=None):
    """int32 rows [T, n_q d]; keys of pages outside the pool are left out."""
    T, d, n_kv = len(pos), pages.d, pages.n_kv
    out = np.zeros((T, n_q, d), np.int32)
    for t in range(T) if rows is None else rows:
        if not 0 <= pos[t] < max_len or not 0 <= seq[t] < table.shape[0] or pos[t] // 64 >= table.shape[1]:
            continue
        j = np.arange(max(0, pos[t] + 1 - window) if window else 0, pos[t] + 1)
        blk = table[seq[t], j // 64]
        j, blk = j[(blk >= 0) & (blk < pages.n_blocks)], blk[(blk >= 0) & (blk < pages.n_blocks)]
        if not len(j):
            continue
        for g in range(n_kv):
            K, V = pages.k[blk, g, j % 64], pages.v[blk, g, j % 64]
            ck, cv = pages.ck[blk, g, j % 64], pages.cv[blk, g, j % 64]
            for h in range(g * (n_q // n_kv), (g + 1) * (n_q // n_kv)):
                out[t, h], _ = oracle.attention4_row(q8[t, h], mq[t, h], kq[t, h], K, ck, V, cv, prm[g])
    return out.reshape(T, n_q * d)


def params(n_kv, d, rng, inter=False, units=400.0):
    """[n_kv, 8 + d] parameters of a head with unit-variance keys and values."""
    def dy(x):
        k = 14 - int(np.floor(np.log2(x)))
        return int(round(x * 2.0 ** k)), k
    p = np.zeros((n_kv, 8 + d), np.int32)
    for g in range(n_kv):
        u = 1.0 / (units + 9 * g)
        p[g, :8] = [*dy(1 / (u * 4 * 2 ** 14)), *dy(1 / (u * 2 ** 12)), *dy(128 * u), *dy(u * 2.3 / np.sqrt(d))]
        e = rng.integers(0, 4, d // 2)
        p[g, 8:] = np.repeat(e, 2) if inter else np.tile(e, 2)
    return p


def table(lens, max_blocks, n_blocks, rng, fill=-1):
    """A block table whose sequences own distinct pages in random order."""
    order = rng.permutation(n_blocks).astype(np.int32)
    t = np.full((len(lens), max_blocks), fill, np.int32)
    at = 0
    for i, n in enumerate(lens):
        need = -(-n // 64)
        t[i, :need] = order[at:at + need]
        at += need
    assert at <= n_blocks
    return t


def queries(T, n_q, d, rng):
    return (np.clip(np.rint(rng.normal(0, 40, (T, n_q, d))), -127, 127).astype(np.int8),
            rng.integers(1 << 14, 1 << 15, (T, n_q)).astype(np.int32), rng.integers(18, 22, (T, n_q)).astype(np.int32))
