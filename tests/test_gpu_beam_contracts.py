"""What the entry points of beam search and eviction promise beyond equal bits:
lists that are whole whatever another stream does, pages whose contents follow
their beams."""
import numpy as np
import pytest

import kv4_plain as kp
from test_gpu_kv4 import Dev, cuda
from test_gpu_kv4_evict import setup

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


@pytest.mark.parametrize("max_len", [40000, 524288])
def test_evict_while_another_stream_changes_the_weights(torch, max_len):
    """Which places are kept is anyone's choice then, but the lists are whole:
    ascending places of the sequence from the first ones on, -1 behind them, no
    entry left as it was (the move reads rows by them). Under the larger bound the
    keys are read again in every pass."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(1)
    n_kv, n, keep, sinks, recent = 8, 40000, 1000, 5, 9
    pages, tab, new = setup(rng, [n], keep, n_kv, 64)
    dev = Dev(torch, pages, tab, kp.params(n_kv, 64, rng), n_kv)
    a, b = (cuda(torch, np.rint(np.exp(rng.normal(m, 4, (pages.n_blocks, n_kv, 64)))).astype(np.int64)) for m in (8, 14))
    w = a.clone()
    other, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    seq, lens, nt = cuda(torch, np.zeros(1, np.int32)), cuda(torch, np.array([n], np.int32)), cuda(torch, new)
    kept = [torch.full((1, n_kv, keep), 39990, dtype=torch.int32, device="cuda") for _ in range(60)]
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=other):
        for _ in range(20):
            w.copy_(b)
            w.copy_(a)
    for k in kept:
        with torch.cuda.stream(other):
            g.replay()
        for _ in range(2):
            pkg.detint_kv4_evict(dev.cache, w, seq, lens, max_len, keep, nt, sinks, recent, k)
    torch.cuda.synchronize()
    for k in kept:
        for row in k[0].cpu().numpy():
            m = int((row >= 0).sum())
            assert m >= sinks and (row[m:] == -1).all()
            assert (np.diff(row[:m]) > 0).all() and row[m - 1] < n and row[:sinks].tolist() == list(range(sinks))
    assert not dev.status.any()


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("parents,n", [
    ([[2, 1, 2]], 70), ([[0, 1, 2]], 70), ([[1, 1, 2]], 129), ([[2, -1, 2]], 70), ([[1, -1, 1]], 63), ([[-1, -1, -1]], 1),
    ([[3, 3, 3, 3], [0, 0, 2, 3]], 200), ([[1, 0, -1, 7], [3, 1, 1, -1]], 100), ([[0, 0]], 128), ([[0]], 5), (None, 191)])
def test_reorder_moves_what_the_beams_hold(torch, parents, n, inplace):
    """Every token's slot is marked with its beam and place; after tables and
    copies a row reads its parent's marks. A beam that names itself reads its own.
    A row without a parent reads its own whole pages and a growing page that is
    no other row's."""
    import deterministic_integer_only_gb300 as pkg
    if parents is None:
        parents = np.random.default_rng(n).integers(-1, 16, (5, 16)).tolist()
    G, W = len(parents), len(parents[0])
    n_kv, d, blocks = 2, 64, n // 64 + 2
    pool = G * W * blocks
    rng = np.random.default_rng(n + W)
    tab = rng.permutation(pool).astype(np.int32).reshape(G * W, blocks)
    pages = kp.Pages(pool, n_kv, d, rng)
    mark = np.zeros((pool, n_kv, 64), np.int64)
    for r in range(G * W):
        for h in range(n_kv):
            mark[tab[r], h] = (r * 1000 + h) * 1000 + np.arange(blocks * 64).reshape(blocks, 64)
    pages.ck[:] = mark % 251 + 1
    dev, w = Dev(torch, pages, tab, kp.params(n_kv, d, rng), n_kv), cuda(torch, mark)
    lens = torch.full((G,), n, dtype=torch.int32, device="cuda")
    out = None if inplace else torch.empty_like(dev.table)
    src, dst = pkg.detint_beam_reorder(dev.table, cuda(torch, np.array(parents, np.int32)), lens, out=out)
    pkg.detint_kv4_copy(dev.cache, src, dst, weight=w)
    new, w, ck = (dev.table if inplace else out).cpu().numpy(), w.cpu().numpy(), dev.ck.cpu().numpy()
    for g in range(G):
        for b in range(W):
            p = parents[g][b]
            if 0 <= p < W:
                size, of = n, g * W + p
            else:
                size, of = n // 64 * 64, g * W + b
            at = np.arange(size)
            for h in range(n_kv):
                want = (of * 1000 + h) * 1000 + at
                got = new[g * W + b, at // 64]
                assert np.array_equal(w[got, h, at % 64], want)
                assert np.array_equal(ck.reshape(w.shape)[got, h, at % 64], want % 251 + 1)
        if n % 64:
            assert len(set(new[g * W:(g + 1) * W, n // 64])) == W
    assert not dev.status.any()


def test_beam_search_arrays_may_touch_but_not_overlap(torch):
    """Neighbouring slices of one buffer are fine; in place is refused."""
    import beam_plain as bp
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(4)
    G, W, V = 3, 4, 500
    logits, scores = np.rint(rng.normal(0, 99999, (G * W, V))).astype(np.int32), -rng.integers(0, 1 << 20, (G, W))
    want = bp.select(logits, scores, W, None, -1)
    buf = torch.zeros(8 * G * W, dtype=torch.int32, device="cuda")
    part = [buf[i * G * W:(i + 1) * G * W] for i in range(8)]
    sc = buf[4 * G * W:6 * G * W].view(torch.int64).view(G, W)
    sc.copy_(cuda(torch, scores))
    lg, s2 = cuda(torch, logits), buf[2 * G * W:4 * G * W].view(torch.int64)
    got = pkg.detint_beam_select(lg, sc, W, out=(part[0], part[1], s2, part[6]))
    assert all(np.array_equal(a.cpu().numpy().reshape(b.shape), b) for a, b in zip(got, want))
    assert np.array_equal(sc.cpu().numpy(), scores)
    done = torch.zeros(G, W, dtype=torch.int32, device="cuda")
    tab, lens = torch.arange(G * W * 3, dtype=torch.int32, device="cuda").view(G * W, 3), torch.full((G,), 70, dtype=torch.int32, device="cuda")
    par = cuda(torch, want[0])
    for f in (lambda: pkg.detint_beam_select(lg, sc, W, out=(part[0], part[1], sc, part[6])),
              lambda: pkg.detint_beam_select(lg, sc, W, done, 3, out=(part[0], part[1], s2, done)),
              lambda: pkg.detint_beam_select(lg, sc, W, out=(part[0], part[0], s2, part[6])),
              lambda: pkg.detint_beam_reorder(tab, par, lens, src=par),
              lambda: pkg.detint_beam_reorder(tab, par, lens, src=done, dst=done)):
        with pytest.raises(pkg.DetintError):
            f()
    assert np.array_equal(sc.cpu().numpy(), scores) and np.array_equal(par.cpu().numpy(), want[0]) and not done.any()
