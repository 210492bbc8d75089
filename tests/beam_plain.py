"""Plain forms of beam search, of the cached keys' weights and of eviction (the
arithmetic specification, sections 17 to 19) in numpy int64 and Python integers,
for the tests."""
import numpy as np

MASKED = -(1 << 31)
DEAD = -(1 << 63)
LIVE = -(1 << 62)


def rshr(x, s):
    return x if s == 0 else (x + (1 << (s - 1))) >> s


def octave(f):
    return 32768 + rshr(f * (22787 + rshr(f * (7419 + rshr(2562 * f, 10)), 10)), 10)


def lse(row):
    """Log of the sum of exponentials (Q16) of unmasked int64 logits."""
    m = int(row.max())
    delta = rshr(np.maximum(row - m, -(1 << 22)) * 47274, 21)
    ip, p = -(delta >> 10), octave(delta & 1023) << 15
    e = np.where(ip >= 31, 0, (p + ((np.int64(1) << np.minimum(ip, 40)) >> 1)) >> np.minimum(ip, 40))
    total = int(e.sum())
    b = total.bit_length()
    y = total << (32 - b) if b <= 32 else total >> (b - 32)
    lg = b - 31
    for _ in range(20):
        z = y * y
        c = z >> 63
        y, lg = z >> (31 + c), 2 * lg + c
    return m + rshr(lg * 726817, 24)


def select(logits, scores, n_out, done=None, end_id=-1):
    """(parent, token, score, done) [groups][n_out] of logits [groups * beams][n]."""
    groups, beams = scores.shape
    out = [np.full((groups, n_out), x, t) for x, t in ((-1, np.int32), (-1, np.int32), (DEAD, np.int64), (0, np.int32))]
    for g in range(groups):
        found = []
        for b in range(beams):
            s = int(scores[g, b])
            if s < LIVE:
                continue
            s = min(s, -LIVE)
            if done is not None and done[g, b]:
                found.append((-s, b, end_id, 1))
                continue
            row = logits[g * beams + b].astype(np.int64)
            ids = np.flatnonzero(row != MASKED)
            if not len(ids):
                continue
            base = s - lse(row[ids])
            for i in ids[np.lexsort((ids, -row[ids]))[:n_out]]:
                found.append((-(base + int(row[i])), b, int(i), int(i == end_id)))
        for k, (s, b, i, e) in enumerate(sorted(found)[:n_out]):
            out[0][g, k], out[1][g, k], out[2][g, k], out[3][g, k] = b, i, -s, e
    return out


def reorder(table, parent, lens):
    """(new table, src, dst)."""
    groups, beams = parent.shape
    new, src, dst = table.copy(), np.full(parent.shape, -1, np.int32), np.full(parent.shape, -1, np.int32)
    for g in range(groups):
        old, full = table[g * beams:(g + 1) * beams], int(lens[g]) // 64
        grows = lens[g] % 64 and full < table.shape[1]
        ok = [0 <= p < beams for p in parent[g]]
        spare = [q for q in range(beams) if q not in parent[g].tolist()]
        seen = set()
        for b in range(beams):
            p, row = int(parent[g, b]), new[g * beams + b]
            if ok[b]:
                row[:full] = old[p, :full]
            if not grows:
                continue
            if ok[b] and p not in seen:
                seen.add(p)
                row[full] = old[p, full]
            else:
                row[full] = old[spare.pop(0), full]
                if ok[b]:
                    src[g, b], dst[g, b] = old[p, full], row[full]
    return new, src, dst


def probabilities(q8, mq, kq, k4, ck, prm):
    """p (Q24) of one query row over its keys (values k4 [n][d], scale codes ck)."""
    t = (k4.astype(np.int64) @ q8.astype(np.int64)) * ck.astype(np.int64)
    sh = min(62, max(0, int(kq) + int(prm[7]) - 10))
    delta = np.maximum(rshr((t - t.max()) * (int(mq) * int(prm[6])), sh), -40 * 1024)
    ip = -(delta >> 10)
    e = np.where(ip >= 24, 0, (octave(delta & 1023) + ((np.int64(1) << np.minimum(ip, 40)) >> 1)) >> np.minimum(ip, 40))
    e = np.minimum(e, 32767)
    total = int(e.sum())
    bl = total.bit_length()
    return rshr(e * ((1 << (bl + 23)) // total), bl - 1)


def weigh(pages, weight, table, prm, n_q, q8, mq, kq, seq, pos, window=0, max_len=1 << 30):
    """Adds to weight [n_blocks][n_kv][64]."""
    n_kv = pages.n_kv
    for t in range(len(pos)):
        if not 0 <= pos[t] < max_len or not 0 <= seq[t] < table.shape[0] or pos[t] // 64 >= table.shape[1]:
            continue
        j = np.arange(max(0, pos[t] + 1 - window) if window else 0, pos[t] + 1)
        blk = table[seq[t], j // 64]
        j, blk = j[(blk >= 0) & (blk < pages.n_blocks)], blk[(blk >= 0) & (blk < pages.n_blocks)]
        if not len(j):
            continue
        for h in range(n_q):
            g = h // (n_q // n_kv)
            p = probabilities(q8[t, h], mq[t, h], kq[t, h], pages.k[blk, g, j % 64], pages.ck[blk, g, j % 64], prm[g])
            np.add.at(weight, (blk, g, j % 64), p)


def evict(pages, weight, table, seq, lens, keep, sinks, recent, new_table, max_len=1 << 30):
    """Moves in `pages` and `weight`; the kept places [n][n_kv][keep]."""
    kept = np.full((len(seq), pages.n_kv, keep), -1, np.int32)
    moves = []
    for i, (s, n) in enumerate(zip(seq, lens)):
        if not 0 <= s < table.shape[0] or not 0 <= n <= min(max_len, table.shape[1] * 64):
            continue
        j = np.arange(n)
        blk = table[s, j // 64]
        inside = (blk >= 0) & (blk < pages.n_blocks)
        for g in range(pages.n_kv):
            at = j
            if n > keep:
                w = np.where(inside, weight[np.where(inside, blk, 0), g, j % 64], 0)
                mid = j[sinks:n - recent]
                best = mid[np.lexsort((mid, ~w[sinks:n - recent]))[:keep - sinks - recent]]
                at = np.sort(np.concatenate([j[:sinks], best, j[n - recent:]]))
            kept[i, g, :len(at)] = at
            to = new_table[i, np.arange(len(at)) // 64]
            for x, (a, b) in enumerate(zip(at, to)):
                if not 0 <= b < pages.n_blocks:
                    continue
                if inside[a]:
                    f = (blk[a], g, a % 64)
                    moves.append(((b, g, x % 64), (pages.k[f].copy(), pages.v[f].copy(), pages.ck[f], pages.cv[f], weight[f])))
                else:
                    moves.append(((b, g, x % 64), (0, 0, 1, 1, 0)))
    for to, v in moves:
        pages.k[to], pages.v[to], pages.ck[to], pages.cv[to], weight[to] = v
    return kept
