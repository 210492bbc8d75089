"""Append with rotary positions of their own, the cached keys' weights and
eviction on the GPU against the plain forms, bit for bit."""
import numpy as np
import pytest

import beam_plain as bp
import kv4_plain as kp
from test_gpu_kv4 import Dev, cuda, ragged, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


# ------------------------------------------------------------------- axes
def append_axes_plain(pages, tab, prm, n_q, cos, sin, inter, gammas, eps, qkv, seq, pos, rp, axis):
    """kv4_plain.append token by token, each with a table of one row made of the rows that its pairs take."""
    T, r2 = len(pos), cos.shape[1]
    outs = [np.zeros((T, n_q, pages.d), np.int8), np.zeros((T, n_q), np.int32), np.zeros((T, n_q), np.int32),
            np.zeros((T, pages.n_kv, pages.d), np.int16), np.zeros((T, pages.n_kv, pages.d), np.int16)]
    for t in range(T):
        rows = rp[:, t]
        if pos[t] < 0 or (rows < 0).any() or (rows >= len(cos)).any():
            continue
        pick = rows[np.minimum(axis, len(rp) - 1)]
        c, s = cos[pick, np.arange(r2)], sin[pick, np.arange(r2)]
        # (the place chooses the row of a table that holds the same row everywhere)
        row = np.broadcast_to(c, (int(pos[t]) + 1, r2)), np.broadcast_to(s, (int(pos[t]) + 1, r2))
        got = kp.append(pages, tab, prm, n_q, *row, inter, gammas, eps, qkv[t:t + 1], seq[t:t + 1], pos[t:t + 1])
        for o, g in zip(outs, got):
            o[t] = g[0]
    return outs


AXES = [
    # n_q, n_kv, d, rot, interleaved, norm, axes, woven, runs (sequence, first place, tokens)
    (4, 2, 64, 64, False, True, 1, False, [(0, 0, 1)]),
    (1, 1, 128, 128, False, False, 3, False, [(0, 63, 1), (1, 64, 1)]),
    (3, 1, 64, 32, True, False, 3, True, [(1, 5, 7), (0, 62, 5)]),
    (6, 2, 128, 64, True, True, 4, False, [(0, 3, 66), (1, 0, 1), (2, 127, 2)]),
    (8, 8, 64, 16, False, True, 2, True, [(0, 60, 9), (2, 0, 130)]),
    (5, 1, 128, 0, False, False, 1, False, [(0, 1, 40)]),
    (10, 2, 64, 8, True, True, 4, True, [(0, 0, 3), (1, 7, 2), (2, 120, 17)]),
    (7, 7, 64, 48, False, False, 3, True, [(0, 9, 33)]),
    (2, 1, 128, 128, False, True, 3, True, [(0, 5, 300), (1, 0, 1), (2, 64, 271)]),
    (2, 1, 64, 64, False, True, 4, False, [(0, 1, 1400), (1, 11, 700)]),
]


@pytest.mark.parametrize("n_q,n_kv,d,rot,inter,norm,axes,woven,runs", AXES)
def test_append_axes(torch, n_q, n_kv, d, rot, inter, norm, axes, woven, runs):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(n_q * d + rot)
    lens = [max([p + n for s, p, n in runs if s == i], default=1) for i in range(3)]
    blocks = -(-max(lens) // 64) + 1
    tab = kp.table(lens, blocks, 3 * blocks, rng)
    prm = kp.params(n_kv, d, rng, inter)
    pages = kp.Pages(3 * blocks, n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged(runs)
    T, far = len(pos), 5000
    rp = rng.integers(0, far, (axes, T)).astype(np.int32)
    pos[rng.random(T) < 0.1] = -1 - (T > 5)              # padding, whatever its rows
    if T > 5:
        rp[:, pos < 0] = -9
    r2 = rot // 2
    axis = (np.arange(r2) % axes if woven else np.arange(r2) * axes // max(r2, 1)).astype(np.uint8)
    if r2 > 8 and axes > 1:
        axis[3] = 200                                    # an axis that is not there counts as the last
    cos, sin = tables(rot, far)
    gq, gk = (rng.integers(-(1 << 13), 1 << 13, d).astype(np.int16) for _ in range(2)) if norm else (None, None)
    qkv = np.rint(rng.normal(0, 4096, (T, (n_q + 2 * n_kv) * d))).astype(np.int32)
    want = append_axes_plain(pages, tab, prm, n_q, cos, sin, inter, (gq, gk), 17 if norm else 0, qkv, seq, pos, rp, axis)
    gam = dict(q_gamma=cuda(torch, gq), k_gamma=cuda(torch, gk), eps=17) if norm else {}
    rope = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin), interleaved=inter, **gam) if rot else pkg.RopeNorm(None, None, max_pos=far)
    outs = [torch.full((T + 2,) + w.shape[1:], 99, dtype=dt, device="cuda")
            for w, dt in zip(want, (torch.int8, torch.int32, torch.int32, torch.int16, torch.int16))]
    pkg.detint_kv4_append_axes(dev.cache, rope, cuda(torch, qkv), cuda(torch, seq), cuda(torch, pos), cuda(torch, rp),
                               cuda(torch, axis) if axes > 1 else None, q8=outs[0], mq=outs[1], kq=outs[2], k_val=outs[3], v_val=outs[4])
    for o, w in zip(outs, want):
        o = o.cpu().numpy()
        assert np.array_equal(o[:T], w) and (o[T:] == 99).all()
    dev.holds(pages)
    assert not dev.status.any()


def test_append_axes_out_of_range_positions_are_padding(torch):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(2)
    pages = kp.Pages(4, 2, 64, rng)
    tab, prm = kp.table([64], 1, 4, rng), kp.params(2, 64, rng)
    cos, sin = tables(64, 100)
    axis = (np.arange(32) % 2).astype(np.uint8)
    for bad in (-1, 100, (1 << 31) - 1, -(1 << 31)):
        for n in (3, 700):                               # rows one by one, and chunks of them
            dev = Dev(torch, pages, tab, prm, 4)
            pos = np.concatenate([np.arange(3), np.full(n - 3, -1)]).astype(np.int32)
            rp = rng.integers(0, 100, (2, n)).astype(np.int32)
            rp[1, 1] = bad
            qkv = rng.integers(-9999, 9999, (n, 8 * 64)).astype(np.int32)
            want = append_axes_plain(pages, tab, prm, 4, cos, sin, False, (None, None), 0, qkv, np.zeros(n, np.int32), pos, rp, axis)
            rope = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin))
            q = pkg.detint_kv4_append_axes(dev.cache, rope, cuda(torch, qkv), cuda(torch, np.zeros(n, np.int32)), cuda(torch, pos),
                                           cuda(torch, rp), cuda(torch, axis))
            assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip(q, want))
            dev.holds(pages)
            assert dev.status[1] == 1


def test_one_axis_with_the_place_is_the_plain_append(torch):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(7)
    pages = kp.Pages(20, 2, 128, rng)
    tab, prm = kp.table([600, 500], 10, 20, rng), kp.params(2, 128, rng)
    cos, sin = tables(128, 700)
    seq, pos = ragged([(0, 0, 600), (1, 3, 497)])
    x = cuda(torch, rng.integers(-9999, 9999, (len(pos), 8 * 128)).astype(np.int32))
    rope = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin))
    a, b = (Dev(torch, pages, tab, prm, 4) for _ in range(2))
    seq, pos = cuda(torch, seq), cuda(torch, pos)
    p = pkg.detint_kv4_append(a.cache, rope, x, seq, pos)
    q = pkg.detint_kv4_append_axes(b.cache, rope, x, seq, pos, pos)
    assert all(torch.equal(u, v) for u, v in zip(p, q))
    assert all(torch.equal(u, v) for u, v in ((a.k, b.k), (a.v, b.v), (a.ck, b.ck), (a.cv, b.cv)))


# ------------------------------------------------------------------ weigh
WEIGHS = [
    # n_q, n_kv, d, window, runs (sequence, first place, tokens)
    (2, 1, 64, 0, [(0, 0, 1)]),
    (4, 2, 128, 0, [(0, 63, 1), (1, 64, 1), (2, 0, 1)]),
    (1, 1, 128, 0, [(0, 700, 1)]),
    (6, 2, 64, 100, [(0, 5, 40), (1, 300, 3), (2, 99, 1)]),
    (10, 2, 64, 0, [(2, 500, 2), (0, 127, 66)]),
    (5, 1, 128, 65, [(0, 0, 130)]),
    (16, 1, 64, 0, [(0, 250, 5), (1, 0, 3)]),
    (34, 2, 64, 0, [(0, 70, 2), (1, 9, 1)]),
    (64, 1, 128, 1, [(0, 70, 3)]),
    (8, 8, 128, 0, [(0, 1000, 33), (1, 31, 2)]),
    (32, 8, 64, 0, [(i, 37 * i, 1) for i in range(40)]),
]


def crowd(block, seq, pos, q8, mq, kq):
    """For the form of blocks: padding behind the tokens, so that there are too
    many for one wave of single tokens, which it would hand them to."""
    if not block:
        return seq, pos, q8, mq, kq
    more = lambda x, v: np.concatenate([x, np.full((1000,) + x.shape[1:], v, x.dtype)])  # noqa: E731
    return more(seq, 0), more(pos, -1), more(q8, 3), more(mq, 20000), more(kq, 20)


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("n_q,n_kv,d,window,runs", WEIGHS)
def test_weigh(torch, n_q, n_kv, d, window, runs, block):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(n_q * d + window)
    n = max(s for s, _, _ in runs) + 1
    lens = [max([p + m for s, p, m in runs if s == i], default=1) for i in range(n)]
    blocks = -(-max(lens) // 64) + 1
    pool = sum(-(-x // 64) for x in lens) + 2
    tab, prm = kp.table(lens, blocks, pool, rng), kp.params(n_kv, d, rng, units=90.0)
    pages = kp.Pages(pool, n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged(runs)
    q8, mq, kq = kp.queries(len(pos), n_q, d, rng)
    w = rng.integers(0, 1 << 40, (pool, n_kv, 64))       # added to, not set
    wt = cuda(torch, w)
    bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos, window)
    seq, pos, q8, mq, kq = crowd(block, seq, pos, q8, mq, kq)
    f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
    got = f(dev.cache, *(cuda(torch, x) for x in (q8, mq, kq, seq, pos)), max(lens), wt, window=window)
    assert got is wt and np.array_equal(wt.cpu().numpy(), w)
    dev.holds(pages)
    assert not dev.status.any()


@pytest.mark.parametrize("block", [False, True])
def test_weigh_shared_pages_padding_and_bad_pages(torch, block):
    """Sequences that share pages meet in the same sums; padding and tokens past
    max_len or the table add nothing; keys of a page outside the pool are masked."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(11)
    n_q, n_kv, d = 6, 2, 128
    pages = kp.Pages(12, n_kv, d, rng)
    tab = np.array([[0, 1, 2, 3], [0, 1, 2, 4], [0, 1, 5, -1], [6, 99, 7, 8], [-3, -3, -3, -3]], np.int32)
    prm = kp.params(n_kv, d, rng, units=90.0)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq = np.array([0, 1, 2, 3, 0, 4, 1, 9, -1, 2, 2, 3, 3, 3, 1, 1], np.int32)
    pos = np.array([255, 250, 191, 200, -1, 100, 252, 5, 5, 253, 256, 70, 64, 63, 254, -7], np.int32)
    q8, mq, kq = kp.queries(len(pos), n_q, d, rng)
    for max_len, window in ((256, 0), (255, 0), (256, 64), (256, 3)):
        w = np.zeros((12, n_kv, 64), np.int64)
        wt = cuda(torch, w)
        bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos, window, max_len)
        f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
        s_, p_, *q_ = crowd(block, seq, pos, q8, mq, kq)
        f(dev.cache, *(cuda(torch, x) for x in (*q_, s_, p_)), max_len, wt, window=window)
        assert np.array_equal(wt.cpu().numpy(), w)
    assert dev.status[1] == 1 and not dev.status[6]


@pytest.mark.parametrize("block", [False, True])
@pytest.mark.parametrize("window", [0, 1, 10, 64, 200])
def test_weigh_tokens_in_any_order(torch, window, block):
    """Neighbouring tokens of a sequence far apart from each other, forwards and
    back, the same one twice: a block's pages are not next to each other."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(window)
    n_q, n_kv, d, n = 4, 2, 64, 4000
    pages = kp.Pages(64, n_kv, d, rng)
    tab, prm = rng.permutation(63).astype(np.int32)[None], kp.params(n_kv, d, rng, units=90.0)
    dev = Dev(torch, pages, tab, prm, n_q)
    pos = np.array([0, 3999, 1, 2000, 2000, 63, 64, -1, 3000, 10, 3998, 700, 701, 702, 5, 1500, 1400, 1300, 3999], np.int32)
    seq = np.zeros(len(pos), np.int32)
    q8, mq, kq = kp.queries(len(pos), n_q, d, rng)
    w = np.zeros((64, n_kv, 64), np.int64)
    wt = cuda(torch, w)
    bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos, window)
    seq, pos, q8, mq, kq = crowd(block, seq, pos, q8, mq, kq)
    f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
    f(dev.cache, *(cuda(torch, x) for x in (q8, mq, kq, seq, pos)), n, wt, window=window)
    assert np.array_equal(wt.cpu().numpy(), w) and not dev.status.any()


@pytest.mark.parametrize("block", [False, True])
def test_weigh_extreme_queries(torch, block):
    """Scales at the ends of their range, zero queries, the largest codes: one key
    takes everything, or all of them the same."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(3)
    n_q, n_kv, d = 8, 2, 64
    pages = kp.Pages(6, n_kv, d, rng)
    pages.k[0], pages.ck[0], pages.k[1], pages.ck[1] = 7, 255, -7, 255
    tab, prm = np.arange(6, dtype=np.int32)[None], kp.params(n_kv, d, rng)
    q8, mq, kq = kp.queries(33, n_q, d, rng)
    q8[:9], q8[9:12] = 127, 0
    mq[12:14], kq[12:14] = 0, 0
    kq[14:18], kq[18:22] = -40, 90
    mq[22:25] = 32768
    pos = rng.integers(0, 384, 33).astype(np.int32)
    w = np.zeros((6, n_kv, 64), np.int64)
    wt, dev = cuda(torch, w), Dev(torch, pages, tab, prm, n_q)
    seq = np.zeros(33, np.int32)
    bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos)
    seq, pos, q8, mq, kq = crowd(block, seq, pos, q8, mq, kq)
    f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
    f(dev.cache, *(cuda(torch, x) for x in (q8, mq, kq, seq, pos)), 384, wt)
    assert np.array_equal(wt.cpu().numpy(), w)


@pytest.mark.parametrize("n_q,n_kv,d,n,new,window", [
    (8, 1, 128, 120000, 1, 0), (2, 1, 64, 300000, 2, 0), (16, 1, 64, 40000, 3, 0), (3, 1, 128, 20000, 40, 0),
    (4, 1, 64, 50000, 20, 30000), (1, 1, 64, 524288, 1, 0), (4, 1, 128, 33000, 17, 0)])
@pytest.mark.parametrize("block", [False, True])
def test_weigh_long_contexts(torch, n_q, n_kv, d, n, new, window, block):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(n)
    blocks = -(-n // 64)
    pages = kp.Pages(blocks, n_kv, d, rng)
    tab, prm = rng.permutation(blocks).astype(np.int32)[None], kp.params(n_kv, d, rng, units=60.0)
    dev = Dev(torch, pages, tab, prm, n_q)
    pos = np.arange(n - new, n).astype(np.int32)
    q8, mq, kq = kp.queries(new, n_q, d, rng)
    w = np.zeros((blocks, n_kv, 64), np.int64)
    wt, seq = cuda(torch, w), np.zeros(new, np.int32)
    bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos, window)
    seq, pos, q8, mq, kq = crowd(block, seq, pos, q8, mq, kq)
    f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
    f(dev.cache, *(cuda(torch, x) for x in (q8, mq, kq, seq, pos)), n, wt, window=window)
    assert np.array_equal(wt.cpu().numpy(), w) and not dev.status.any()


# ------------------------------------------------------------------ evict
def check_evict(torch, pages, weight, tab, seq, lens, keep, sinks, recent, new, max_len, clean=True):
    import deterministic_integer_only_gb300 as pkg
    dev = Dev(torch, pages, tab, kp.params(pages.n_kv, pages.d, np.random.default_rng(0)), pages.n_kv)
    wt = cuda(torch, weight)
    want = bp.evict(pages, weight, tab, seq, lens, keep, sinks, recent, new, max_len)
    n = len(seq)
    kept = torch.full((n * pages.n_kv * keep + 5,), 77, dtype=torch.int32, device="cuda")
    pkg.detint_kv4_evict(dev.cache, wt, cuda(torch, seq), cuda(torch, lens), max_len, keep, cuda(torch, new), sinks, recent, kept)
    kept = kept.cpu().numpy()
    assert np.array_equal(kept[:-5].reshape(want.shape), want) and (kept[-5:] == 77).all()
    assert np.array_equal(wt.cpu().numpy(), weight)
    dev.holds(pages)
    assert bool(dev.status[1]) != clean
    return want


def setup(rng, lens, keep, n_kv, d):
    n, room = len(lens), -(-keep // 64)
    pool = sum(-(-x // 64) for x in lens) + n * room + 2
    pages = kp.Pages(pool, n_kv, d, rng)
    tab = kp.table(lens, max(-(-max(lens) // 64), 1), pool, rng)
    free = np.setdiff1d(np.arange(pool), tab[tab >= 0])
    return pages, tab, rng.permutation(free)[:n * room].astype(np.int32).reshape(n, room)


@pytest.mark.parametrize("n_kv,d,lens,keep,sinks,recent", [
    (1, 64, [1], 1, 0, 0), (2, 128, [2, 1, 65], 1, 0, 0), (1, 128, [64, 63, 65], 64, 4, 8), (3, 64, [200, 0, 131], 70, 0, 0),
    (2, 64, [500, 400], 129, 129, 0), (2, 128, [500, 400], 129, 0, 129), (1, 64, [777], 100, 60, 40), (2, 128, [3000], 1000, 4, 64),
    (1, 128, [5000, 17, 4097], 63, 1, 1), (8, 64, [1025] * 5, 512, 16, 32), (1, 64, [20000, 33001], 4099, 4, 100),
    (1, 128, [70000], 300, 0, 0), (1, 64, [2000], 1999, 3, 3)])
def test_evict(torch, n_kv, d, lens, keep, sinks, recent):
    rng = np.random.default_rng(sum(lens) + keep)
    pages, tab, new = setup(rng, lens, keep, n_kv, d)
    w = np.rint(np.exp(rng.normal(12, 4, (pages.n_blocks, n_kv, 64)))).astype(np.int64)
    check_evict(torch, pages, w, tab, np.arange(len(lens), dtype=np.int32), np.array(lens, np.int32), keep, sinks, recent, new, max(lens))


@pytest.mark.parametrize("lens,keep", [([3000, 17, 900], 200), ([400001], 700)])
def test_evict_under_the_largest_bound(torch, lens, keep):
    """max_len 524288, where the keys of a CTA's share do not fit its shared memory."""
    rng = np.random.default_rng(keep)
    pages, tab, new = setup(rng, lens, keep, 1, 64)
    w = np.rint(np.exp(rng.normal(8, 4, (pages.n_blocks, 1, 64)))).astype(np.int64)
    check_evict(torch, pages, w, tab, np.arange(len(lens), dtype=np.int32), np.array(lens, np.int32), keep, 4, 9, new, 524288)


WEIGHTS = {
    "zeros": lambda rng, s: np.zeros(s, np.int64),
    "few values": lambda rng, s: rng.integers(0, 3, s),
    "extremes": lambda rng, s: rng.choice([-(1 << 63), (1 << 63) - 1, 0, -1, 1], s),
    "wide": lambda rng, s: rng.integers(-(1 << 63), (1 << 63) - 1, s),
    "one large": lambda rng, s: (rng.random(s) < 0.01) * (np.int64(1) << 50),
    "close": lambda rng, s: (np.int64(1) << 40) + rng.integers(0, 4000, s),
    "bit edge": lambda rng, s: (np.int64(1) << 33) - rng.integers(0, 2, s) * rng.integers(0, 2049, s),
}


@pytest.mark.parametrize("kind", WEIGHTS)
@pytest.mark.parametrize("lens,keep,sinks,recent", [([900, 64, 333], 257, 3, 5), ([40000], 1000, 0, 0), ([5000, 4500], 4400, 10, 10)])
def test_evict_values(torch, kind, lens, keep, sinks, recent):
    """Ties go to the lower place; negative weights order as numbers do."""
    rng = np.random.default_rng(len(kind))
    pages, tab, new = setup(rng, lens, keep, 2, 64)
    w = np.asarray(WEIGHTS[kind](rng, (pages.n_blocks, 2, 64)), np.int64)
    check_evict(torch, pages, w, tab, np.arange(len(lens), dtype=np.int32), np.array(lens, np.int32), keep, sinks, recent, new, max(lens))


@pytest.mark.parametrize("kind", WEIGHTS)
@pytest.mark.parametrize("n,n_kv,most,keep", [(50, 8, 700, 190), (20, 4, 8192, 300)])
def test_evict_many_sequences(torch, kind, n, n_kv, most, keep):
    """More CTAs than the GPU holds at two per SM, by themselves and in clusters."""
    rng = np.random.default_rng(n + len(kind))
    lens = rng.integers(0, 500, n)
    lens[[3, n - 2]] = most, most - 1
    pages, tab, new = setup(rng, list(lens), keep, n_kv, 64)
    w = np.asarray(WEIGHTS[kind](rng, (pages.n_blocks, n_kv, 64)), np.int64)
    check_evict(torch, pages, w, tab, np.arange(n, dtype=np.int32), lens.astype(np.int32), keep, 2, 7, new, most)


def test_evict_rows_of_the_table_and_bad_entries(torch):
    """Any rows in any order, the same one twice; lengths and sequences out of
    range move nothing; a page outside the pool moves as zeros of weight 0."""
    rng = np.random.default_rng(5)
    lens = [300, 200, 260, 100]
    pages, tab, new = setup(rng, lens, 128, 2, 128)
    w = rng.integers(-5, 1 << 30, (pages.n_blocks, 2, 64))
    new = np.concatenate([new, np.full((1, 2), -1, np.int32)])
    check_evict(torch, pages, w, tab, np.array([2, 0, 2], np.int32), np.array([260, 300, 130], np.int32), 128, 4, 4, new[:3], 300)
    tab[1, 1], tab[1, 2] = -1, pages.n_blocks
    check_evict(torch, pages, w, tab, np.array([1, 4, -1, 0], np.int32), np.array([200, 10, 10, 301], np.int32), 128, 4, 4, new[:4], 300,
                clean=False)
    check_evict(torch, pages, w, tab, np.array([0, 3], np.int32), np.array([300, 100], np.int32), 128, 4, 4, new[3:], 300, clean=False)


def test_evict_lengths_change_under_a_captured_graph(torch):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(8)
    pages, tab, new = setup(rng, [900, 900], 200, 2, 64)
    dev = Dev(torch, pages, tab, kp.params(2, 64, rng), 2)
    w = rng.integers(0, 1 << 30, (pages.n_blocks, 2, 64))
    wt, seq, lens = cuda(torch, w), cuda(torch, np.arange(2, dtype=np.int32)), cuda(torch, np.array([900, 900], np.int32))
    nt, kept = cuda(torch, new), torch.empty(2, 2, 200, dtype=torch.int32, device="cuda")
    st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=st):
        pkg.detint_kv4_evict(dev.cache, wt, seq, lens, 900, 200, nt, 4, 9, kept, stream=st)
    for ln in ([900, 201], [150, 899], [0, 900]):
        lens.copy_(cuda(torch, np.array(ln, np.int32)))
        g.replay()
        torch.cuda.synchronize()
        want = bp.evict(pages, w, tab, np.arange(2), np.array(ln), 200, 4, 9, new, 900)
        assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(wt.cpu().numpy(), w)
        dev.holds(pages)


# ------------------------------------- together: a context with a budget
def test_a_context_with_a_budget(torch):
    """Prefill, weigh with the last tokens, evict, then decode on with rotary
    positions apart from the places, weigh every step and evict again."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(6)
    n_q, n_kv, d, n, keep, seen = 4, 2, 64, 300, 130, 16
    pages = kp.Pages(16, n_kv, d, rng)
    prm = kp.params(n_kv, d, rng, units=90.0)
    cos, sin = tables(d, 600)
    tab = np.full((1, 6), -1, np.int32)
    tab[0, :5] = [3, 9, 1, 12, 7]
    dev = Dev(torch, pages, tab, prm, n_q)
    rope = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin))
    w = np.zeros((16, n_kv, 64), np.int64)
    wt = cuda(torch, w)
    axis = np.zeros(d // 2, np.uint8)

    def go(places, positions):
        qkv = np.rint(rng.normal(0, 9000, (len(places), (n_q + 2 * n_kv) * d))).astype(np.int32)
        seq, rp = np.zeros(len(places), np.int32), np.asarray(positions, np.int32)[None]
        pos = np.asarray(places, np.int32)
        want = append_axes_plain(pages, tab, prm, n_q, cos, sin, False, (None, None), 0, qkv, seq, pos, rp, axis)
        q = pkg.detint_kv4_append_axes(dev.cache, rope, cuda(torch, qkv), cuda(torch, seq), cuda(torch, pos), cuda(torch, rp))
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(q, want))
        o = (pkg.detint_kv4_prefill if len(pos) > 1 else pkg.detint_kv4_decode)(dev.cache, *q, cuda(torch, seq), cuda(torch, pos), 384)
        rows = list(range(max(0, len(pos) - seen), len(pos)))
        assert np.array_equal(o.cpu().numpy()[rows], kp.attention(pages, tab, prm, n_q, *want[:3], seq, pos, rows=rows)[rows])
        cut = [x[rows[0]:].contiguous() for x in (*q, cuda(torch, seq), cuda(torch, pos))]
        (pkg.detint_kv4_weigh_block if len(rows) > 1 else pkg.detint_kv4_weigh)(dev.cache, *cut, 384, wt)
        bp.weigh(pages, w, tab, prm, n_q, *(x[rows[0]:] for x in want[:3]), seq[rows[0]:], pos[rows[0]:])
        assert np.array_equal(wt.cpu().numpy(), w)

    go(np.arange(n), np.arange(n))
    at, held = n, n
    for new in ([0, 2, 4], [5, 6, 8]):
        new = np.array([new], np.int32)
        want = bp.evict(pages, w, tab, [0], [held], keep, 4, 8, new)
        kept = pkg.detint_kv4_evict(dev.cache, wt, cuda(torch, np.zeros(1, np.int32)), cuda(torch, np.array([held], np.int32)), 384,
                                    keep, cuda(torch, new), 4, 8)
        assert np.array_equal(kept.cpu().numpy(), want) and np.array_equal(wt.cpu().numpy(), w)
        dev.holds(pages)
        tab[0] = -1
        tab[0, :3] = new[0]
        dev.table.copy_(cuda(torch, tab))
        held = keep
        for _ in range(30):
            go([held], [at])
            held, at = held + 1, at + 1
    dev.holds(pages)
    assert not dev.status.any()
