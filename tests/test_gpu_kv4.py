"""The 4-bit paged K/V cache operators on the GPU against plain 64-bit forms
(kv4_plain: the oracle's scalar rows on plain arrays), bit for bit: every
output, every byte of the pages and everything that must stay as it was."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

import kv4_plain as kp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


def cuda(torch, a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Dev:
    """Pages, table and parameters on the device."""

    def __init__(self, torch, pages, table, prm, n_q):
        import deterministic_integer_only_gb300 as pkg
        k, v = pages.packed()
        self.k, self.v = cuda(torch, k), cuda(torch, v)
        self.ck, self.cv = cuda(torch, pages.ck), cuda(torch, pages.cv)
        self.table, self.prm = cuda(torch, table), cuda(torch, prm)
        self.status = torch.zeros(8, dtype=torch.int32, device="cuda")
        self.cache = pkg.KV4Cache(self.k, self.v, self.ck, self.cv, self.table, self.prm, n_q, status=self.status)

    def holds(self, pages):
        k, v = pages.packed()
        assert np.array_equal(self.k.cpu().numpy(), k) and np.array_equal(self.v.cpu().numpy(), v)
        assert np.array_equal(self.ck.cpu().numpy(), pages.ck) and np.array_equal(self.cv.cpu().numpy(), pages.cv)


def ragged(spec):
    """(seq, pos) of runs (sequence, first position, tokens)."""
    seq = np.concatenate([np.full(n, s) for s, _, n in spec]).astype(np.int32)
    pos = np.concatenate([np.arange(p, p + n) for _, p, n in spec]).astype(np.int32)
    return seq, pos


def tables(rot, max_pos, stretch=1.0):
    a = np.arange(max_pos)[:, None] / stretch * 1e4 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))[None]
    return np.rint(np.cos(a) * 16384).astype(np.int16), np.rint(np.sin(a) * 16384).astype(np.int16)


def run_append(torch, pages, dev, prm, n_q, rot, inter, norm, qkv, seq, pos, max_pos, pad=0, tab=None, eps=17):
    """The GPU's outputs and the plain form's, after checking them and the pages."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(5)
    n_kv, d, T = pages.n_kv, pages.d, len(pos)
    cos, sin = tables(rot, max_pos)
    gq, gk = (rng.integers(-(1 << 13), 1 << 13, d).astype(np.int16) for _ in range(2)) if norm else (None, None)
    want = kp.append(pages, tab, prm, n_q, cos, sin, inter, (gq, gk), eps if norm else 0, qkv, seq, pos)
    gam = dict(q_gamma=cuda(torch, gq), k_gamma=cuda(torch, gk), eps=eps) if norm else {}
    r = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin), interleaved=inter, **gam) if rot else \
        pkg.RopeNorm(None, None, max_pos=max_pos, **gam)
    width = qkv.shape[1]
    buf = torch.full((T, width + pad), 123456789, dtype=torch.int32, device="cuda")
    buf[:, :width] = cuda(torch, qkv)
    outs = [torch.full((T + 2,) + s, 99, dtype=dt, device="cuda") for s, dt in
            (((n_q, d), torch.int8), ((n_q,), torch.int32), ((n_q,), torch.int32), ((n_kv, d), torch.int16), ((n_kv, d), torch.int16))]
    pkg.detint_kv4_append(dev.cache, r, buf[:, :width], cuda(torch, seq), cuda(torch, pos), q8=outs[0], mq=outs[1], kq=outs[2],
                          k_val=outs[3], v_val=outs[4])
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        o = o.cpu().numpy()
        assert np.array_equal(o[:T], w)
        assert (o[T:] == 99).all()                      # rows behind the last token are left as they were
    dev.holds(pages)
    return want


APPENDS = [
    # n_q, n_kv, d, rot, interleaved, norm, runs (sequence, first position, tokens)
    (4, 2, 64, 64, False, True, [(0, 0, 1)]),
    (1, 1, 128, 128, False, False, [(0, 63, 1), (1, 64, 1)]),
    (3, 1, 64, 32, True, False, [(1, 5, 7), (0, 62, 5)]),
    (6, 2, 128, 64, True, True, [(0, 3, 66), (1, 0, 1), (2, 127, 2)]),
    (8, 8, 64, 16, False, True, [(0, 60, 9), (2, 0, 130)]),
    (5, 1, 128, 0, False, False, [(0, 1, 40)]),
    (10, 2, 64, 8, True, True, [(0, 0, 3), (1, 7, 2), (2, 120, 17)]),
    (7, 7, 64, 48, False, False, [(0, 9, 33)]),
]


@pytest.mark.parametrize("n_q,n_kv,d,rot,inter,norm,runs", APPENDS)
def test_append(torch, n_q, n_kv, d, rot, inter, norm, runs):
    rng = np.random.default_rng(n_q * d + rot)
    lens = [max([p + n for s, p, n in runs if s == i], default=1) for i in range(3)]
    tab = kp.table(lens, 4, 12, rng)
    prm = kp.params(n_kv, d, rng, inter)
    pages = kp.Pages(12, n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged(runs)
    qkv = np.rint(rng.normal(0, 4096, (len(pos), (n_q + 2 * n_kv) * d))).astype(np.int32)
    qkv[:, ::37] *= 7
    run_append(torch, pages, dev, prm, n_q, rot, inter, norm, qkv, seq, pos, 200, pad=4 * (n_q % 3), tab=tab)
    assert not dev.status.any()


@pytest.mark.parametrize("d,norm,inter", [(64, True, False), (128, False, True), (128, True, False), (64, False, False)])
def test_append_chunks_of_rows(torch, d, norm, inter):
    """Enough tokens that a CTA takes whole chunks of rows, with odd run ends."""
    rng = np.random.default_rng(d + norm)
    n_q, n_kv = 2, 1
    runs = [(0, 5, 1003), (1, 0, 1), (2, 64, 1130), (3, 1, 63), (1, 1, 1200)]
    lens = [1008, 1201, 1194, 64]
    tab = kp.table(lens, 19, 60, rng)
    prm = kp.params(n_kv, d, rng, inter)
    pages = kp.Pages(60, n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged(runs)
    pos = np.concatenate([pos, [-1, -1, -5]]).astype(np.int32)     # padding at the end
    seq = np.concatenate([seq, [0, 9, -1]]).astype(np.int32)
    qkv = np.rint(rng.normal(0, 4096, (len(pos), (n_q + 2 * n_kv) * d))).astype(np.int32)
    run_append(torch, pages, dev, prm, n_q, d // 2, inter, norm, qkv, seq, pos, 1300, tab=tab)
    assert not dev.status.any()


@pytest.mark.parametrize("T", [171, 333, 700, 1403, 3001])
@pytest.mark.parametrize("d,norm,inter", [(64, False, True), (128, True, False)])
def test_append_tiles_of_every_size(torch, d, norm, inter, T):
    """Tiles of 2 to 32 tokens on a GPU of 152 SMs, the last one cut short."""
    rng = np.random.default_rng(T + d)
    n_q, n_kv = 16, 8
    lens = [T // 3 + 5, T - T // 3 - 1]
    tab = kp.table(lens, 40, 70, rng)
    prm = kp.params(n_kv, d, rng, inter)
    pages = kp.Pages(70, n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged([(0, 5, T // 3), (1, 0, T - T // 3 - 1)])
    pos = np.concatenate([pos, [-1]]).astype(np.int32)
    seq = np.concatenate([seq, [0]]).astype(np.int32)
    qkv = np.rint(rng.normal(0, 4096, (T, (n_q + 2 * n_kv) * d))).astype(np.int32)
    run_append(torch, pages, dev, prm, n_q, d, inter, norm, qkv, seq, pos, 2100, tab=tab)
    assert not dev.status.any()


@pytest.mark.parametrize("norm", [True, False])
def test_append_extreme_rows(torch, norm):
    """Zero rows, single spikes, the largest magnitudes, every exponent."""
    rng = np.random.default_rng(3)
    n_q, n_kv, d = 4, 2, 128
    pages = kp.Pages(4, n_kv, d, rng)
    tab = kp.table([64], 1, 4, rng)
    prm = kp.params(n_kv, d, rng)
    width = (n_q + 2 * n_kv) * d
    rows = [np.zeros(width), np.eye(width)[5], np.eye(width)[5] * -(2 ** 31 - 1), np.full(width, 2 ** 31 - 1), np.full(width, -(2 ** 31 - 1)),
            np.tile([2 ** 31 - 1, -(2 ** 31 - 1)], width // 2), np.full(width, 1), np.full(width, -1)]
    rows += [np.rint(rng.normal(0, 2.0 ** b, width)).clip(-(2 ** 31 - 1), 2 ** 31 - 1) for b in range(0, 31)]
    rows += [np.full(width, 2 ** 29 - 1), np.full(width, 2 ** 29), np.full(width, -2 ** 29), np.full(width, 2 ** 24), np.full(width, 2 ** 24 - 1)]
    qkv = np.array(rows).astype(np.int32)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged([(0, 2, len(qkv))])
    run_append(torch, pages, dev, prm, n_q, 128, False, norm, qkv, seq, pos, 64, tab=tab, eps=32767)


def test_append_leaves_out_padding_and_bad_places(torch):
    rng = np.random.default_rng(8)
    n_q, n_kv, d = 4, 2, 64
    pages = kp.Pages(6, n_kv, d, rng)
    tab = kp.table([128, 70], 2, 6, rng)
    tab[1, 1] = 6                                       # outside the pool
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    # padding, a sequence and a position outside the table, past the rotation rows, a bad page
    seq = np.array([0, -1, 2, 0, 0, 1, 1, 0], np.int32)
    pos = np.array([-1, 3, 3, 130, 128, 64, 10, 127], np.int32)
    qkv = np.rint(rng.normal(0, 4096, (8, 8 * d))).astype(np.int32)
    run_append(torch, pages, dev, prm, n_q, d, False, False, qkv, seq, pos, 130, tab=tab)
    assert dev.status.cpu().tolist() == [0, 1, 0, 0, 0, 0, 0, 0]


def run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, max_len, window, which, rows=None, want=None, pad=0):
    """which: "decode"; "prefill", which hands few tokens to the single-token
    form; "blocks": the tokens repeated until they are too many for that."""
    import deterministic_integer_only_gb300 as pkg
    T, width = len(pos), n_q * pages.d
    if want is None:
        want = kp.attention(pages, tab, prm, n_q, *q, seq, pos, window, max_len, rows)
    if which == "blocks":
        assert rows is None
        n = 2 * torch.cuda.get_device_properties(0).multi_processor_count // (T * pages.n_kv) + 1
        q, seq, pos, want = [np.concatenate([a] * n) for a in q], np.tile(seq, n), np.tile(pos, n), np.tile(want, (n, 1))
        T *= n
    buf = torch.full((T + 2, width + pad), -77, dtype=torch.int32, device="cuda")
    out = buf[:T, :width] if pad else buf[:T]
    args = [cuda(torch, a) for a in q] + [cuda(torch, seq), cuda(torch, pos)]
    fn = pkg.detint_kv4_decode if which == "decode" else pkg.detint_kv4_prefill
    fn(dev.cache, *args, max_len, window=window, out=out)
    torch.cuda.synchronize()
    got = buf.cpu().numpy()
    assert (got[T:] == -77).all() and (got[:, width:] == -77).all()
    got = got[:T, :width]
    if rows is not None:
        got_r, want = got[rows], want[rows]
    else:
        got_r = got
    assert np.array_equal(got_r, want), np.argwhere(got_r != want)[:4]
    return got


HEADS = [(1, 1, 64), (2, 1, 128), (3, 1, 64), (8, 2, 128), (5, 1, 128), (16, 2, 64), (12, 1, 64), (4, 4, 128), (10, 5, 64)]


@pytest.mark.parametrize("which", ["decode", "prefill", "blocks"])
@pytest.mark.parametrize("n_q,n_kv,d", HEADS)
def test_attention_of_ragged_tokens(torch, which, n_q, n_kv, d):
    """Every head layout, lengths around page ends, several tokens of a sequence,
    padding and empty rows among them."""
    rng = np.random.default_rng(n_q * 7 + d)
    lens = [1, 2, 63, 64, 65, 128, 200, 333]
    tab = kp.table(lens, 7, 24, rng)
    pages = kp.Pages(24, n_kv, d, rng)
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq = np.concatenate([np.arange(8), [7, 7, 3, 0, 6, 6]]).astype(np.int32)
    pos = np.concatenate([np.array(lens) - 1, [0, 300, 5, -1, -9, 199]]).astype(np.int32)
    q = kp.queries(len(pos), n_q, d, rng)
    for window in (0, 1, 7, 64, 130):
        run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, 400, window, which, pad=2 * (window % 3))
    assert not dev.status.any()


@pytest.mark.parametrize("n_q,n_kv,d", [(4, 2, 64), (2, 1, 128), (6, 1, 128), (16, 1, 64), (40, 1, 64), (64, 1, 128)])
def test_prefill_blocks(torch, n_q, n_kv, d):
    """Runs of one sequence that start and end inside a block of query rows."""
    rng = np.random.default_rng(n_q + d)
    runs = [(0, 0, 70), (1, 17, 1), (2, 60, 33), (1, 100, 90), (3, 0, 5), (0, 70, 3), (4, 3, 280)]
    lens = [73, 190, 93, 5, 283]
    tab = kp.table(lens, 5, 16, rng)
    pages = kp.Pages(16, n_kv, d, rng)
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    seq, pos = ragged(runs)
    q = kp.queries(len(pos), n_q, d, rng)
    for window in (0, 3, 50):
        a = run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, 283, window, "prefill")
        run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, 283, window, "decode", want=a)
    # any order of the same tokens gives the same rows
    o = rng.permutation(len(pos))
    run_attention(torch, dev, pages, prm, tab, n_q, [x[o] for x in q], seq[o], pos[o], 283, 0, "prefill",
                  want=run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, 283, 0, "prefill")[o])


@pytest.mark.parametrize("which", ["decode", "prefill", "blocks"])
def test_attention_extremes(torch, which):
    """The largest scores of both signs, all keys alike, underflow of all but
    one key, zero queries, shifts at their ends."""
    rng = np.random.default_rng(2)
    n_q, n_kv, d = 8, 1, 128
    pages = kp.Pages(4, n_kv, d, rng)
    tab = kp.table([250], 4, 4, rng)
    pages.k[tab[0, 0], 0, :20], pages.ck[tab[0, 0], 0, :20] = 7, 255
    pages.k[tab[0, 1], 0, :20], pages.ck[tab[0, 1], 0, :20] = -7, 255
    pages.v[tab[0, 2], 0], pages.cv[tab[0, 2], 0] = 7, 255
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    pos = np.array([249, 249, 100, 63, 0, 249, 20, 249, 249], np.int32)
    seq = np.zeros(len(pos), np.int32)
    q8, mq, kq = kp.queries(len(pos), n_q, d, rng)
    q8[0], q8[1] = 127, -127
    q8[2], mq[2], kq[2] = 0, 0, 0
    kq[3], kq[4] = -40, 90                              # shift clamped to 0; everything rounds to nothing
    mq[5], kq[6] = 1 << 15, 5
    kq[7], kq[8] = 14, 10 - prm[0, 7] + 2               # far below the maximum; a shift of 2
    run_attention(torch, dev, pages, prm, tab, n_q, (q8, mq, kq), seq, pos, 250, 0, which)
    # output scales that saturate 32 bits, and mantissas at their ends
    prm[0, 4:8] = [1 << 15, 0, 1 << 15, 1]
    dev = Dev(torch, pages, tab, prm, n_q)
    run_attention(torch, dev, pages, prm, tab, n_q, (q8, mq, kq), seq, pos, 250, 0, which)


@pytest.mark.parametrize("which", ["decode", "prefill", "blocks"])
def test_bad_pages_and_places_are_masked_and_recorded(torch, which):
    rng = np.random.default_rng(6)
    n_q, n_kv, d = 4, 2, 64
    pages = kp.Pages(8, n_kv, d, rng)
    tab = kp.table([200, 130, 64], 4, 8, rng)
    tab[0, 1], tab[1, 0], tab[1, 1], tab[1, 2] = -1, 8, -5, 1 << 30      # one page missing; every page missing
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    # the last four: sequences and positions outside the table, and past max_len
    seq = np.array([0, 0, 1, 2, 3, -1, 2, 0], np.int32)
    pos = np.array([199, 66, 129, 63, 10, 10, 256, 220], np.int32)
    q = kp.queries(len(pos), n_q, d, rng)
    run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, 210, 0, which)
    assert dev.status.cpu().tolist() == [0, 1, 0, 0, 0, 0, 0, 0]


@pytest.mark.parametrize("n_q,n_kv,d,hi", [(2, 1, 64, 600), (8, 2, 128, 1100), (4, 1, 128, 2500), (3, 1, 64, 4800), (16, 2, 64, 4500), (5, 1, 128, 4200)])
def test_decode_split_over_a_cluster(torch, n_q, n_kv, d, hi):
    """Few tokens of 600 to 4800 keys: 2 to 16 CTAs share one, some without a page."""
    rng = np.random.default_rng(hi)
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, 3, hi)
    q = kp.queries(3, n_q, d, rng)
    seq, pos = np.arange(3, dtype=np.int32), np.array([hi - 1, hi // 3, 64], np.int32)
    for window in (0, 65, 900):
        run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, hi, window, "decode")
    assert not dev.status.any()


@pytest.mark.parametrize("n_q,n_kv,d,hi", [(2, 1, 64, 34000), (3, 1, 128, 40001)])
def test_few_tokens_of_long_contexts(torch, n_q, n_kv, d, hi):
    """More than 32 pages for each of 16 CTAs: two launches with a workspace as
    single tokens, one where a block of few tokens, which has none, goes there."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(hi)
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, 2, hi)
    assert pkg.detint_kv4_workspace(dev.cache, 2, hi) > 0
    q = kp.queries(2, n_q, d, rng)
    seq, pos = np.arange(2, dtype=np.int32), np.array([hi - 1, hi // 2], np.int32)
    for window in (0, 33000):
        for which in ("decode", "prefill"):
            run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, hi, window, which)
    assert not dev.status.any()


@pytest.mark.parametrize("n_q,n_kv,d,T,hi", [(32, 8, 128, 40, 2600), (32, 4, 64, 40, 1900), (16, 2, 128, 64, 2500), (24, 8, 64, 40, 3000),
                                             (16, 8, 128, 40, 5200), (4, 4, 64, 80, 12000)])
def test_decode_in_two_launches(torch, n_q, n_kv, d, T, hi):
    """Batches whose decode takes the two-launch path: against the plain form on
    some rows and against the block form, bit for bit, on all; twice on one
    workspace, whose first contents do not matter."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(T)
    lens = [1 + (hi - 1) * ((i * 7) % T) // (T - 1) for i in range(T)]
    nb = sum(-(-n // 64) for n in lens)
    tab = kp.table(lens, -(-hi // 64), nb, rng)
    pages = kp.Pages(nb, n_kv, d, rng)
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    need = pkg.detint_kv4_workspace(dev.cache, T, hi)
    assert need > 0
    seq, pos = np.arange(T, dtype=np.int32), np.array(lens, np.int32) - 1
    pos[3] = -1
    q = kp.queries(T, n_q, d, rng)
    rows = [0, 1, 2, 3, T - 1]
    for window in (0, 700):
        got = run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, hi, window, "prefill", rows=rows)
        run_attention(torch, dev, pages, prm, tab, n_q, q, seq, pos, hi, window, "decode", want=got)
        ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
        dq = [cuda(torch, a) for a in q] + [cuda(torch, seq), cuda(torch, pos)]
        for _ in range(2):
            o = pkg.detint_kv4_decode(dev.cache, *dq, hi, window=window, workspace=ws)
            assert np.array_equal(o.cpu().numpy(), got)
    with pytest.raises(pkg.DetintError) as e:
        pkg.detint_kv4_decode(dev.cache, *dq, hi, workspace=ws[:need - 16])
    assert e.value.code == 1


@pytest.mark.parametrize("which", ["decode", "prefill", "blocks"])
def test_longest_context(torch, which):
    """524288 keys: sums past 32 bits, every page index used."""
    rng = np.random.default_rng(4)
    n_q, n_kv, d, n = 2, 1, 64, 1 << 19
    pages = kp.Pages(n // 64, n_kv, d, rng)
    pages.cv[:] = 255
    tab = kp.table([n], n // 64, n // 64, rng)
    prm = kp.params(n_kv, d, rng)
    dev = Dev(torch, pages, tab, prm, n_q)
    q8, mq, kq = kp.queries(3, n_q, d, rng)
    q8[0], mq[0], kq[0] = 0, 0, 0                       # all weights alike: the largest sums there are
    pos = np.array([n - 1, n - 1, n - 64], np.int32)
    run_attention(torch, dev, pages, prm, tab, n_q, (q8, mq, kq), np.zeros(3, np.int32), pos, n, 0, which)


def test_pages_past_32_bit_offsets(torch):
    """A pool of more than 4 GB for K and for V: pages at its far end are
    appended to and read at the right place."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(9)
    n_q, n_kv, d = 4, 2, 128
    nb = (1 << 32) // (n_kv * 64 * d // 2) + 70
    shape = (nb, n_kv, 64, d // 2)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((nb, n_kv, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    small = kp.Pages(3, n_kv, d, rng)
    far = np.array([nb - 1, nb - 68, 1], np.int32)
    pk, pv = small.packed()
    at = cuda(torch, far.astype(np.int64))
    k[at], v[at], ks[at], vs[at] = cuda(torch, pk), cuda(torch, pv), cuda(torch, small.ck), cuda(torch, small.cv)
    tab = np.array([[0, 1, 2]], np.int32)
    prm = kp.params(n_kv, d, rng)
    dt = cuda(torch, far[tab])
    cache = pkg.KV4Cache(k, v, ks, vs, dt, cuda(torch, prm), n_q)
    seq, pos = ragged([(0, 60, 9), (0, 130, 2)])
    cos, sin = tables(d, 200)
    qkv = np.rint(rng.normal(0, 4096, (len(pos), 8 * d))).astype(np.int32)
    want = kp.append(small, tab, prm, n_q, cos, sin, False, (None, None), 0, qkv, seq, pos)
    q = pkg.detint_kv4_append(cache, pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin)), cuda(torch, qkv), cuda(torch, seq), cuda(torch, pos))
    for a, b in zip(q, want):
        assert np.array_equal(a.cpu().numpy(), b)
    pk, pv = small.packed()
    for got, exp in ((k, pk), (v, pv), (ks, small.ck), (vs, small.cv)):
        assert np.array_equal(got[at].cpu().numpy(), exp)
    want = kp.attention(small, tab, prm, n_q, *want[:3], seq, pos)
    for fn in (pkg.detint_kv4_decode, pkg.detint_kv4_prefill):
        assert np.array_equal(fn(cache, *q, cuda(torch, seq), cuda(torch, pos), 192).cpu().numpy(), want)


def _step_setup(torch, rng, n_q, n_kv, d, n_seq, max_len):
    nb = n_seq * -(-max_len // 64)
    tab = kp.table([max_len] * n_seq, -(-max_len // 64), nb, rng)
    pages = kp.Pages(nb, n_kv, d, rng)
    prm = kp.params(n_kv, d, rng)
    return pages, tab, prm, Dev(torch, pages, tab, prm, n_q)


def test_append_then_attention_token_by_token_equals_one_prefill(torch):
    """The operators as a model uses them: a prompt appended and attended to in
    one call each, or a token at a time, leaves the same pages and rows."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(12)
    n_q, n_kv, d, n = 4, 2, 64, 75
    pages, tab, prm, a = _step_setup(torch, rng, n_q, n_kv, d, 2, 128)
    b = Dev(torch, pages, tab, prm, n_q)
    cos, sin = tables(d, 128)
    r = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin))
    qkv = cuda(torch, np.rint(rng.normal(0, 4096, (2 * n, 8 * d))).astype(np.int32))
    seq, pos = ragged([(0, 0, n), (1, 0, n)])
    ds, dp = cuda(torch, seq), cuda(torch, pos)
    q = pkg.detint_kv4_append(a.cache, r, qkv, ds, dp)
    whole = pkg.detint_kv4_prefill(a.cache, *q, ds, dp, n)
    for t in range(n):
        i = torch.tensor([t, n + t], device="cuda")
        q1 = pkg.detint_kv4_append(b.cache, r, qkv[i], ds[i], dp[i])
        step = pkg.detint_kv4_decode(b.cache, *q1, ds[i], dp[i], 128)
        assert torch.equal(step, whole[i]), t
    for x, y in ((a.k, b.k), (a.v, b.v), (a.ck, b.ck), (a.cv, b.cv)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("T,hi,n_q,n_kv", [(2, 300, 8, 4), (16, 4200, 32, 2)])
def test_captured_step_is_replayed_with_new_positions(torch, T, hi, n_q, n_kv):
    """Append and decode in a CUDA graph (both decode forms): the replay reads
    the positions that are in memory then."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(T)
    d, width = 64, (n_q + 2 * n_kv) * 64
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, T, hi)
    ref = Dev(torch, pages, tab, prm, n_q)
    cos, sin = tables(d, hi)
    r = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin), interleaved=True)
    qkv = torch.zeros((T, width), dtype=torch.int32, device="cuda")
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")
    need = pkg.detint_kv4_workspace(dev.cache, T, hi)
    assert (need > 0) == (T == 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    q8, out = torch.empty((T, n_q, d), dtype=torch.int8, device="cuda"), torch.empty((T, n_q * d), dtype=torch.int32, device="cuda")
    mq, kq = (torch.empty((T, n_q), dtype=torch.int32, device="cuda") for _ in range(2))

    def step():
        pkg.detint_kv4_append(dev.cache, r, qkv, seq, pos, q8=q8, mq=mq, kq=kq)
        pkg.detint_kv4_decode(dev.cache, q8, mq, kq, seq, pos, hi, out=out, workspace=ws)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for p in (0, 63, 64, 200, hi - 1):
        x = cuda(torch, np.rint(rng.normal(0, 4096, (T, width))).astype(np.int32))
        qkv.copy_(x)
        pos.fill_(p)
        pos[T - 1] = p // 2
        g.replay()
        q = pkg.detint_kv4_append(ref.cache, r, x, seq, pos)
        assert torch.equal(out, pkg.detint_kv4_prefill(ref.cache, *q, seq, pos, hi)), p


FIRST_CALL = """
import sys
sys.path[:0] = [%(root)r, %(tests)r]
import numpy as np, torch
import deterministic_integer_only_gb300 as pkg
import test_gpu_kv4 as t
rng = np.random.default_rng(2)
pages, tab, prm, dev = t._step_setup(torch, rng, 8, 2, 64, 3, 200)
q = [t.cuda(torch, a) for a in t.kp.queries(3, 8, 64, rng)]
seq, pos = torch.arange(3, dtype=torch.int32, device="cuda"), t.cuda(torch, np.array([199, 0, 64], np.int32))
out = torch.zeros((3, 512), dtype=torch.int32, device="cuda")
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pkg.detint_kv4_%(which)s(dev.cache, *q, seq, pos, 200, out=out)
g.replay()
torch.cuda.synchronize()
want = t.kp.attention(pages, tab, prm, 8, *[a.cpu().numpy() for a in q], seq.cpu().numpy(), pos.cpu().numpy())
assert np.array_equal(out.cpu().numpy(), want)
"""


@pytest.mark.parametrize("which", ["decode", "prefill"])
def test_first_call_of_a_process_may_be_captured(torch, which):
    here = os.path.dirname(os.path.abspath(__file__))
    code = FIRST_CALL % dict(root=os.path.dirname(here), tests=here, which=which)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_host_threads_at_once(torch):
    """Calls of two host threads, each on a stream of its own."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(31)
    n_q, n_kv, d, T, hi = 8, 2, 128, 6, 700
    sets = []
    for _ in range(2):
        pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, T, hi)
        q = kp.queries(T, n_q, d, rng)
        pos = rng.integers(0, hi, T).astype(np.int32)
        want = kp.attention(pages, tab, prm, n_q, *q, np.arange(T), pos)
        sets.append((dev, [cuda(torch, a) for a in q], cuda(torch, np.arange(T, dtype=np.int32)), cuda(torch, pos), want))
    torch.cuda.synchronize()

    def work(x):
        dev, q, seq, pos, want = x
        s = torch.cuda.Stream()
        got = [fn(dev.cache, *q, seq, pos, hi, stream=s) for _ in range(20) for fn in (pkg.detint_kv4_decode, pkg.detint_kv4_prefill)]
        s.synchronize()
        return all(np.array_equal(g.cpu().numpy(), want) for g in got)

    with ThreadPoolExecutor(2) as ex:
        assert all(ex.map(work, sets))


@pytest.mark.parametrize("n_q,d,hi", [(1, 64, 100), (8, 64, 1300)])
def test_more_tokens_than_a_launch_takes(torch, n_q, d, hi):
    """65600 tokens: past a launch's 65535 for the single-token form, in one
    launch of clusters and in two with a workspace."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(hi)
    T = 65600
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, 1, d, 3, hi)
    q = kp.queries(T, n_q, d, rng)
    seq = np.sort(rng.integers(0, 3, T)).astype(np.int32)
    pos = rng.integers(-2, hi, T).astype(np.int32)
    args = [cuda(torch, a) for a in (*q, seq, pos)]
    assert (pkg.detint_kv4_workspace(dev.cache, T, hi) > 0) == (hi > 1000)
    dec = pkg.detint_kv4_decode(dev.cache, *args, hi)
    pre = pkg.detint_kv4_prefill(dev.cache, *args, hi)
    assert torch.equal(dec, pre)
    rows = np.array([0, 1, 32767, 65533, 65534, 65535, 65536, 65537, T - 1])
    want = kp.attention(pages, tab, prm, n_q, *[a[rows] for a in q], seq[rows], pos[rows])
    assert np.array_equal(dec.cpu().numpy()[rows], want)
    assert not dev.status.any()


def test_one_row_of_a_wider_buffer(torch):
    """A single row's stride does not matter, whatever its buffer's width."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(14)
    pages, tab, prm, dev = _step_setup(torch, rng, 4, 2, 64, 1, 64)
    ref = Dev(torch, pages, tab, prm, 4)
    qkv = cuda(torch, np.rint(rng.normal(0, 4096, (1, 8 * 64 + 3))).astype(np.int32))
    rope = pkg.RopeNorm(*(cuda(torch, a) for a in tables(64, 64)))
    seq, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda")
    q = pkg.detint_kv4_append(dev.cache, rope, qkv, seq, pos)
    w = pkg.detint_kv4_append(ref.cache, rope, qkv[:, :512].contiguous(), seq, pos)
    assert all(torch.equal(a, b) for a, b in zip(q, w)) and torch.equal(dev.k, ref.k) and torch.equal(dev.v, ref.v)
    out = torch.full((1, 4 * 64 + 1), -5, dtype=torch.int32, device="cuda")
    pkg.detint_kv4_decode(dev.cache, *q, seq, pos, 64, out=out)
    assert torch.equal(out[:, :256], pkg.detint_kv4_decode(dev.cache, *q, seq, pos, 64)) and int(out[0, 256]) == -5


def test_two_streams_at_once(torch):
    """The same cache read by calls on two streams, each with its own outputs
    and workspace."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(21)
    n_q, n_kv, d, T, hi = 16, 4, 128, 20, 5000
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, T, hi)
    qs = [[cuda(torch, a) for a in kp.queries(T, n_q, d, rng)] for _ in range(2)]
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = cuda(torch, rng.integers(0, hi, T).astype(np.int32))
    want = [pkg.detint_kv4_prefill(dev.cache, *q, seq, pos, hi) for q in qs]
    assert pkg.detint_kv4_workspace(dev.cache, T, hi) > 0
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        got = [pkg.detint_kv4_decode(dev.cache, *q, seq, pos, hi, stream=s) for q, s in zip(qs, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refusals(torch):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(1)
    pages, tab, prm, dev = _step_setup(torch, rng, 4, 2, 64, 1, 64)
    q8, mq, kq = (cuda(torch, a) for a in kp.queries(3, 4, 64, rng))
    seq, pos = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")
    dec = pkg.detint_kv4_decode
    for bad in ((q8.cpu(), mq, kq, seq, pos), (q8.int(), mq, kq, seq, pos), (q8, mq[:2], kq, seq, pos), (q8, mq, kq.long(), seq, pos),
                (q8, mq, kq, seq.cpu(), pos), (q8, mq, kq, seq[:1], pos), (q8[:, :, ::2], mq, kq, seq, pos)):
        with pytest.raises(ValueError):
            dec(dev.cache, *bad, 64)
    with pytest.raises(ValueError):
        dec(dev.cache, q8, mq, kq, seq, pos, 64, out=torch.empty((3, 200), dtype=torch.int32, device="cuda"))
    for kw in (dict(max_len=0), dict(max_len=(1 << 19) + 1), dict(max_len=64, window=-1), dict(max_len=64, window=(1 << 32) + 1),
               dict(max_len=(1 << 32) + 64)):
        with pytest.raises(pkg.DetintError):
            dec(dev.cache, q8, mq, kq, seq, pos, **kw)
    cos, sin = (cuda(torch, a) for a in tables(64, 64))
    qkv = torch.zeros((3, 8 * 64), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pkg.detint_kv4_append(dev.cache, pkg.RopeNorm(cos, sin), qkv.long(), seq, pos)
    with pytest.raises(ValueError):
        pkg.detint_kv4_append(dev.cache, pkg.RopeNorm(cos, sin), qkv[:, :500], seq, pos)
    with pytest.raises(ValueError):                     # gammas of another head width
        g = torch.ones(128, dtype=torch.int16, device="cuda")
        pkg.detint_kv4_append(dev.cache, pkg.RopeNorm(cos, sin, q_gamma=g, k_gamma=g), qkv, seq, pos)
    with pytest.raises(pkg.DetintError):                # one gamma
        pkg.detint_kv4_append(dev.cache, pkg.RopeNorm(cos, sin, q_gamma=g[:64].contiguous()), qkv, seq, pos)


@pytest.mark.parametrize("n_q,n_kv,d,T,hi", [(16, 8, 128, 1, 300), (4, 1, 64, 3, 700), (32, 4, 64, 40, 1900)])
def test_windows_past_every_key(torch, n_q, n_kv, d, T, hi):
    """A window of max_len or more sees every key, up to the largest int: both
    forms give what no window gives, with the workspace that was asked for."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(hi + T)
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, T, hi)
    q = [cuda(torch, a) for a in kp.queries(T, n_q, d, rng)]
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = cuda(torch, rng.integers(hi // 2, hi, T).astype(np.int32))
    need = pkg.detint_kv4_workspace(dev.cache, T, hi)
    assert (need > 0) == (T == 40)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    want = pkg.detint_kv4_decode(dev.cache, *q, seq, pos, hi, workspace=ws)
    rows = np.array([0, T - 1])
    assert np.array_equal(want.cpu().numpy()[rows], kp.attention(pages, tab, prm, n_q, *[a.cpu().numpy()[rows] for a in q],
                                                                 rows, pos.cpu().numpy()[rows]))
    for window in (hi - 1, hi, hi + 1, (1 << 31) - 63, (1 << 31) - 1):
        got = pkg.detint_kv4_prefill(dev.cache, *q, seq, pos, hi, window=window)
        if window >= hi:
            assert torch.equal(got, want), window
        assert torch.equal(pkg.detint_kv4_decode(dev.cache, *q, seq, pos, hi, window=window, workspace=ws), got), window
    assert not dev.status.any()


@pytest.mark.parametrize("n_q,n_kv,d,T,hi", [(16, 8, 128, 100, 3000), (8, 8, 64, 160, 2300)])
def test_a_workspace_serves_smaller_calls(torch, n_q, n_kv, d, T, hi):
    """A buffer sized once, for the largest batch and context, is enough for
    every smaller call, also where the largest takes one launch and a smaller
    one two."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(hi)
    pages, tab, prm, dev = _step_setup(torch, rng, n_q, n_kv, d, T, hi)
    need = pkg.detint_kv4_workspace(dev.cache, T, hi)
    for n in [*range(1, T + 1), 2 * T, 5 * T]:
        smaller = [pkg.detint_kv4_workspace(dev.cache, n, m) for m in (1, 64, 700, 2100, hi)]
        assert smaller == sorted(smaller)
        assert smaller[-1] <= need if n <= T else smaller[-1] >= need
    buf = torch.full((need + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[:need]
    q = kp.queries(T, n_q, d, rng)
    pos = rng.integers(hi // 2, hi, T).astype(np.int32)
    dq, dp = [cuda(torch, a) for a in q], cuda(torch, pos)
    seq = torch.arange(T, dtype=torch.int32, device="cuda")
    want = pkg.detint_kv4_prefill(dev.cache, *dq, seq, dp, hi)
    row = kp.attention(pages, tab, prm, n_q, *[a[:1] for a in q], np.zeros(1, np.int32), pos[:1])
    assert np.array_equal(want[:1].cpu().numpy(), row)
    for n in (T, T // 2, 40, 38, 20, 7, 1):
        for window in (0, hi - 10, 2200):
            exp = want if not window else pkg.detint_kv4_prefill(dev.cache, *dq, seq, dp, hi, window=window)
            args = [a[:n] for a in dq] + [seq[:n], dp[:n]]
            got = pkg.detint_kv4_decode(dev.cache, *args, hi, window=window, workspace=ws if need else None)
            assert torch.equal(got, exp[:n]), (n, window)
    assert (buf[need:] == 0x5A).all()
    assert not dev.status.any()


REFUSED_LAUNCH = """
import ctypes, sys
sys.path[:0] = [%(root)r, %(tests)r]
import numpy as np, torch
import deterministic_integer_only_gb300 as pkg
import test_gpu_kv4 as t
rng = np.random.default_rng(17)
pages, tab, prm, dev = t._step_setup(torch, rng, 4, 2, 64, 1, 64)
ref = t.Dev(torch, pages, tab, prm, 4)
q = [t.cuda(torch, a) for a in t.kp.queries(1, 4, 64, rng)]
seq, pos = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 5, dtype=torch.int32, device="cuda")
qkv = t.cuda(torch, np.rint(rng.normal(0, 4096, (1, 8 * 64))).astype(np.int32))
rope = pkg.RopeNorm(*(t.cuda(torch, a) for a in t.tables(64, 64)))
out, q2 = torch.zeros((1, 256), dtype=torch.int32, device="cuda"), [torch.empty_like(a) for a in q]
want = pkg.detint_kv4_append(ref.cache, rope, qkv, seq, pos)
pkg.detint_kv4_decode(dev.cache, *q, seq, pos, 64, out=out)
torch.cuda.synchronize()
legacy, other, codes, raw = torch.cuda.default_stream(), torch.cuda.Stream(), [], ctypes.c_void_p()
torch.cuda.cudart().cudaStreamCreate(ctypes.addressof(raw))     # one that the legacy stream would wait for
calls = (lambda: pkg.detint_kv4_decode(dev.cache, *q, seq, pos, 64, out=out, stream=legacy),
         lambda: pkg.detint_kv4_append(dev.cache, rope, qkv, seq, pos, *q2, stream=other))
try:
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=torch.cuda.ExternalStream(raw.value)):
        for call in calls:
            try:
                call()
                codes.append(0)
            except pkg.DetintError as e:
                codes.append(e.code)
except RuntimeError:                # the refused launch ended the capture
    pass
other.synchronize()
assert codes == [7, 0], codes
assert all(torch.equal(a, b) for a, b in zip(q2, want)) and torch.equal(dev.k, ref.k) and torch.equal(dev.v, ref.v)
"""


def test_a_refused_launch_does_not_fail_the_next_call(torch):
    """A launch that CUDA refuses on the host (on the legacy stream while another
    is being captured) is that call's error and not the next one's."""
    here = os.path.dirname(os.path.abspath(__file__))
    code = REFUSED_LAUNCH % dict(root=os.path.dirname(here), tests=here)
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)
