"""Beam selection, beam reordering and page copies on the GPU against the plain
forms (beam_plain), whole numbers that have to be equal."""
import numpy as np
import pytest

import beam_plain as bp
import kv4_plain as kp
from test_gpu_kv4 import Dev, cuda, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


def check_select(torch, logits, scores, n_out, done=None, end_id=-1, pad=0, shift=0):
    """shift: elements by which the rows' start is off a 16-byte boundary."""
    import deterministic_integer_only_gb300 as pkg
    rows, n = logits.shape
    buf = torch.full((rows * (n + pad) + shift + 8,), (1 << 31) - 1, dtype=torch.int32, device="cuda")
    x = buf[shift:shift + rows * (n + pad)].view(rows, n + pad)[:, :n]
    x.copy_(cuda(torch, logits))
    want = bp.select(logits, scores, n_out, done, end_id)
    shape = want[0].shape
    outs = [torch.full((shape[0] * shape[1] + 3,), 99, dtype=torch.int64 if i == 2 else torch.int32, device="cuda") for i in range(4)]
    pkg.detint_beam_select(x, cuda(torch, scores), n_out, None if done is None else cuda(torch, done), end_id, out=outs)
    for o, w in zip(outs, want):
        o = o.cpu().numpy()
        assert np.array_equal(o[:-3].reshape(shape), w)
        assert (o[-3:] == 99).all()                      # behind the last group: left as it was
    return want


def normal(rng, rows, n, spread=2.0):
    return np.rint(rng.normal(0, spread * 65536, (rows, n))).astype(np.int32)


@pytest.mark.parametrize("groups,beams,n,n_out,pad,shift", [
    (1, 1, 1, 1, 0, 0), (1, 1, 5, 8, 0, 0), (2, 3, 63, 6, 1, 0), (1, 4, 151936, 4, 0, 0), (3, 5, 2051, 64, 0, 1),
    (1, 64, 300, 64, 0, 0), (40, 2, 33001, 3, 3, 2), (7, 1, 128256, 1, 64, 0), (1, 2, 400001, 5, 0, 0), (1, 1, 1500000, 7, 0, 0),
    (1, 3, 1 << 14, 64, 4, 0), (170, 2, 20000, 4, 0, 0), (5, 16, 5000, 32, 0, 3), (1, 1, 2048, 33, 0, 0), (1, 1, 2049, 17, 0, 0)])
def test_select_sizes(torch, groups, beams, n, n_out, pad, shift):
    rng = np.random.default_rng(groups * n + n_out)
    logits = normal(rng, groups * beams, n)
    scores = -rng.integers(0, 1 << 22, (groups, beams))
    check_select(torch, logits, scores, n_out, pad=pad, shift=shift)


KINDS = {
    "equal": lambda rng, n: np.full(n, 12345),
    "zeros and ones": lambda rng, n: rng.integers(0, 2, n),
    "few steps": lambda rng, n: rng.integers(0, 5, n) * 65536,
    "extremes": lambda rng, n: rng.choice([-(1 << 31) + 1, (1 << 31) - 1, 0, -1], n),
    "lowest": lambda rng, n: np.full(n, -(1 << 31) + 1),
    "all masked": lambda rng, n: np.full(n, bp.MASKED),
    "one": lambda rng, n: np.where(np.arange(n) == n * 2 // 3, 7, bp.MASKED),
    "ascending": lambda rng, n: np.arange(n) * 3,
    "descending": lambda rng, n: -np.arange(n) * 3,
    "half masked": lambda rng, n: np.where(rng.random(n) < 0.5, bp.MASKED, rng.integers(-90000, 90000, n)),
    "few allowed": lambda rng, n: np.where(rng.random(n) < 0.002, rng.integers(-90000, 90000, n), bp.MASKED),
    "a run allowed": lambda rng, n: np.where(np.arange(n) < 6000, rng.integers(-90000, 90000, n), bp.MASKED),
    "a run on top": lambda rng, n: np.where(np.arange(n) // 2048 % 16 == 3, 1 << 20, 0) + rng.integers(0, 1000, n),
    "flat tail": lambda rng, n: np.where(np.arange(n) == 5, 0, -18 * 45426 - rng.integers(0, 9, n)),
}


@pytest.mark.parametrize("n,n_out", [(97, 4), (3001, 64), (50000, 64), (151936, 5)])
@pytest.mark.parametrize("kind", KINDS)
def test_select_values(torch, kind, n, n_out):
    """Ties, extremes, masks that leave nothing, a few or one run of tokens, whose
    values all reach the bound and are too many to be ranked by counting."""
    rng = np.random.default_rng(n)
    logits = np.stack([KINDS[kind](rng, n) for _ in range(4)]).astype(np.int32)
    check_select(torch, logits, np.array([[0, -70000], [-5, -5]]), n_out)


def test_select_finished_missing_and_extreme_beams(torch):
    rng = np.random.default_rng(4)
    logits = normal(rng, 24, 1000)
    logits[3] = bp.MASKED
    logits[17, 5:] = bp.MASKED
    scores = -rng.integers(0, 1 << 20, (6, 4))
    done = (rng.random((6, 4)) < 0.3).astype(np.int32) * 7
    scores[0, 1:] = bp.DEAD
    scores[1] = bp.DEAD                                  # nothing at all
    scores[2, 0], scores[2, 1] = bp.LIVE, bp.LIVE - 1    # the last one there, the first one not
    scores[3, 2], scores[3, 3] = (1 << 62) + 5, (1 << 63) - 1
    done[4] = 1                                          # every beam finished
    for n_out in (1, 4, 9, 64):
        want = check_select(torch, logits, scores, n_out, done, 999)
        assert (want[0][1] == -1).all() and (want[2][1] == bp.DEAD).all()
    logits[:, 999] = bp.MASKED                           # a masked end token still is what a finished beam continues with
    check_select(torch, logits, scores, 4, done, 999)
    check_select(torch, logits, scores, 4, None, -1)


def test_select_feeds_itself_on_a_captured_graph(torch):
    """Steps whose scores and flags are the outputs of the step before, replayed
    with other logits; two graphs with workspaces of their own on two streams."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(9)
    G, W, n = 3, 4, 40001
    runs = []
    for i in range(2):
        st = torch.cuda.Stream()
        x = cuda(torch, normal(rng, G * W, n))
        ws = torch.empty(pkg.detint_beam_workspace(G * W, n, W), dtype=torch.uint8, device="cuda")
        a = [torch.zeros(G, W, dtype=torch.int32, device="cuda"), torch.zeros(G, W, dtype=torch.int32, device="cuda"),
             torch.full((G, W), bp.DEAD, dtype=torch.int64, device="cuda"), torch.zeros(G, W, dtype=torch.int32, device="cuda")]
        a[2][:, 0] = 0
        b = [torch.empty_like(t) for t in a]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            pkg.detint_beam_select(x, a[2], W, a[3], 17, out=b, workspace=ws, stream=st)
            pkg.detint_beam_select(x, b[2], W, b[3], 17, out=a, workspace=ws, stream=st)
        runs.append((st, g, x, a, b, ws))
    state = [(np.where(np.arange(W) == 0, 0, bp.DEAD) * np.ones((G, 1), np.int64), np.zeros((G, W), np.int32)) for _ in runs]
    for step in range(3):
        for i, (st, g, x, a, b, ws) in enumerate(runs):
            x.copy_(cuda(torch, normal(rng, G * W, n)))
        torch.cuda.synchronize()
        for st, g, *_ in runs:
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for i, (st, g, x, a, b, ws) in enumerate(runs):
            l = x.cpu().numpy()
            for got in (b, a):
                want = bp.select(l, state[i][0], W, state[i][1], 17)
                assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(got, want))
                state[i] = (want[2], want[3])


# ------------------------------------------------------------- reordering
@pytest.mark.parametrize("groups,beams,blocks", [(1, 1, 1), (1, 4, 3), (3, 5, 70), (2, 64, 130), (9, 8, 64)])
@pytest.mark.parametrize("inplace", [False, True])
def test_reorder(torch, groups, beams, blocks, inplace):
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(groups * 100 + beams)
    for trial in range(6):
        tab = rng.permutation(groups * beams * blocks).astype(np.int32).reshape(groups * beams, blocks)
        parent = rng.integers(0, beams, (groups, beams)).astype(np.int32)
        if trial == 1:
            parent[rng.random(parent.shape) < 0.4] = -1
            parent[-1, -1] = beams
        if trial == 2:
            parent[:] = np.stack([rng.permutation(beams) for _ in range(groups)])
        if trial == 3:
            parent[:] = beams - 1
        lens = rng.integers(0, blocks * 64 + 1, groups).astype(np.int32)
        if trial == 4:
            lens[:] = lens // 64 * 64
        if trial == 5:
            lens[0] = blocks * 64 + 7                    # past the table: no page that grows
        new, src, dst = bp.reorder(tab, parent, lens)
        t = cuda(torch, tab)
        out = None if inplace else torch.full_like(t, -7)
        s, d = pkg.detint_beam_reorder(t, cuda(torch, parent), cuda(torch, lens), out=out)
        assert np.array_equal((t if inplace else out).cpu().numpy(), new)
        assert np.array_equal(s.cpu().numpy(), src) and np.array_equal(d.cpu().numpy(), dst)
        # no page is copied to twice, none is both copied from and to, and growing pages stay apart
        to = dst[dst >= 0]
        assert len(set(to)) == len(to) and not set(to) & set(src[src >= 0])
        for g in range(groups):
            if lens[g] % 64 and lens[g] // 64 < blocks:
                assert len(set(new[g * beams:(g + 1) * beams, lens[g] // 64])) == beams


@pytest.mark.parametrize("n_kv,d,weighed", [(1, 64, False), (3, 128, True), (8, 64, True)])
def test_copy_pages(torch, n_kv, d, weighed):
    rng = np.random.default_rng(n_kv)
    pages = kp.Pages(20, n_kv, d, rng)
    dev = Dev(torch, pages, np.zeros((1, 4), np.int32), kp.params(n_kv, d, rng), n_kv)
    import deterministic_integer_only_gb300 as pkg
    w = rng.integers(-(1 << 62), 1 << 62, (20, n_kv, 64))
    wt = cuda(torch, w)
    src, dst = np.array([3, -1, 7, 5, 0, 7], np.int32), np.array([4, 9, -1, 6, 19, 8], np.int32)
    pkg.detint_kv4_copy(dev.cache, cuda(torch, src), cuda(torch, dst), weight=wt if weighed else None)
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            for x in (pages.k, pages.v, pages.ck, pages.cv) + ((w,) if weighed else ()):
                x[b] = x[a]
    dev.holds(pages)
    assert np.array_equal(wt.cpu().numpy(), w) and not dev.status.any()
    pkg.detint_kv4_copy(dev.cache, cuda(torch, np.array([20, 1], np.int32)), cuda(torch, np.array([2, 20], np.int32)))
    dev.holds(pages)                                     # pages past the pool: nothing moves, and it is recorded
    assert dev.status[1] == 1


# ------------------------------------------------- together: a beam search
@pytest.mark.parametrize("captured", [False, True])
def test_beam_search_over_the_paged_cache(torch, captured):
    """70 steps of beam search with a made-up model: a step appends every beam's
    token to its pages, attends, and makes logits of the attention's rows. The
    beams share their prompt's pages and reorder by tables and page copies; the
    plain run keeps a cache of its own for every beam and copies it whole."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(1)
    G, W, n_q, n_kv, d, V, prompt, steps = 2, 3, 4, 2, 64, 203, 130, 70
    R, blocks = G * W, 4
    width, end = (n_q + 2 * n_kv) * d, 202
    prm = kp.params(n_kv, d, rng)
    cos, sin = tables(d, 256)
    emb = rng.integers(-6000, 6000, (V, width)).astype(np.int32)
    head = rng.integers(-9, 10, (n_q * d, V)).astype(np.int32)
    # pages: 2 whole ones of a group's prompt shared, the others of each beam; the prompt's third page is beam 0's
    pages = kp.Pages(G * 2 + R * 2, n_kv, d, rng)
    tab = np.zeros((R, blocks), np.int32)
    for r in range(R):
        tab[r] = [r // W * 2, r // W * 2 + 1, G * 2 + 2 * r, G * 2 + 2 * r + 1]
    plain = [kp.Pages(blocks, n_kv, d, rng) for _ in range(R)]
    for r, pl in enumerate(plain):
        first = tab[r // W * W]                          # every beam starts as its group's first
        for x in ("k", "v", "ck", "cv"):
            getattr(pl, x)[:] = getattr(pages, x)[first]
    for r in range(R):
        for x in (pages.k, pages.v, pages.ck, pages.cv):
            x[tab[r, 2]] = x[tab[r // W * W, 2]]
    dev = Dev(torch, pages, tab, prm, n_q)
    rope = pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin))
    emb_t, head_t = cuda(torch, emb), cuda(torch, head.astype(np.float64))
    tok = torch.zeros(R, dtype=torch.int32, device="cuda")
    seq = torch.arange(R, dtype=torch.int32, device="cuda")
    pos = torch.full((R,), prompt, dtype=torch.int32, device="cuda")
    lens = torch.full((G,), prompt + 1, dtype=torch.int32, device="cuda")
    scores = torch.full((G, W), bp.DEAD, dtype=torch.int64, device="cuda")
    scores[:, 0] = 0
    done = torch.zeros(G, W, dtype=torch.int32, device="cuda")
    ws = torch.empty(pkg.detint_beam_workspace(R, V, W), dtype=torch.uint8, device="cuda")
    outs = [torch.empty(G, W, dtype=torch.int64 if i == 2 else torch.int32, device="cuda") for i in range(4)]
    src, dst = (torch.empty(G, W, dtype=torch.int32, device="cuda") for _ in range(2))
    logits = torch.empty(R, V, dtype=torch.int32, device="cuda")

    def step():
        q = pkg.detint_kv4_append(dev.cache, rope, emb_t[tok.long()], seq, pos)
        o = pkg.detint_kv4_decode(dev.cache, *q, seq, pos, 256)
        logits.copy_(torch.floor(o.double() @ head_t / 16).clamp(-2 ** 31 + 1, 2 ** 31 - 1))   # (sums below 2^53: exact)
        pkg.detint_beam_select(logits, scores, W, done, end, out=outs, workspace=ws)
        scores.copy_(outs[2])
        done.copy_(outs[3])
        tok.copy_(outs[1].view(-1).clamp(min=0))
        pkg.detint_beam_reorder(dev.table, outs[0], lens, src=src, dst=dst)
        pkg.detint_kv4_copy(dev.cache, src, dst)
        pos.add_(1)
        lens.add_(1)

    graph = None
    if captured:
        keep = [t.clone() for t in (tok, pos, lens, scores, done, dev.table, dev.k, dev.v, dev.ck, dev.cv)]
        st = torch.cuda.Stream()
        with torch.cuda.stream(st):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            step()
        for t, k in zip((tok, pos, lens, scores, done, dev.table, dev.k, dev.v, dev.ck, dev.cv), keep):
            t.copy_(k)
        torch.cuda.synchronize()
    p_tok, p_scores = np.zeros(R, np.int64), np.where(np.arange(W) == 0, 0, bp.DEAD) * np.ones((G, 1), np.int64)
    p_done, own = np.zeros((G, W), np.int32), np.arange(blocks, dtype=np.int32)[None]
    for s in range(steps):
        graph.replay() if graph else step()
        if captured:
            torch.cuda.synchronize()
        at, zero = np.array([prompt + s]), np.zeros(1, np.int32)
        want = np.empty((R, V), np.int64)
        for r in range(R):
            q = kp.append(plain[r], own, prm, n_q, cos, sin, False, (None, None), 0, emb[p_tok[r]][None], zero, at)
            o = kp.attention(plain[r], own, prm, n_q, *q[:3], zero, at)
            want[r] = np.clip((o.astype(np.int64) @ head)[0] >> 4, -2 ** 31 + 1, 2 ** 31 - 1)
        assert np.array_equal(logits.cpu().numpy(), want), s
        sel = bp.select(want, p_scores, W, p_done, end)
        assert all(np.array_equal(t.cpu().numpy(), w) for t, w in zip(outs, sel)), s
        kids = []
        for g in range(G):
            for b in range(W):
                p = g * W + max(int(sel[0][g, b]), 0)
                c = kp.Pages(0, n_kv, d, rng)
                c.n_blocks = blocks
                c.k, c.v, c.ck, c.cv = (getattr(plain[p], x).copy() for x in ("k", "v", "ck", "cv"))
                kids.append(c)
        plain, p_tok, p_scores, p_done = kids, np.maximum(sel[1].reshape(-1), 0), sel[2], sel[3]
    assert not dev.status.any()
