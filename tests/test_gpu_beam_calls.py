"""How the operators of beam search, weights and eviction may be called: first
in a capture, from host threads at once, on another stream, with more tokens
than a launch takes, on pools past 32-bit offsets, and what the binding refuses."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest

import beam_plain as bp
import kv4_plain as kp
from test_gpu_kv4 import Dev, cuda, ragged, tables
from test_gpu_kv4_evict import append_axes_plain

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


class Case:
    """Inputs of every operator on one small cache, and what they give."""

    def __init__(self, torch, seed, n_q=8, n_kv=2, d=64, n=300, T=160):
        rng = np.random.default_rng(seed)
        self.torch, self.n = torch, n
        blocks = -(-n // 64)
        self.pages = kp.Pages(3 * blocks + 4, n_kv, d, rng)
        self.tab = kp.table([n, n], blocks, 2 * blocks, rng)
        self.prm = kp.params(n_kv, d, rng, units=90.0)
        self.dev = Dev(torch, self.pages, self.tab, self.prm, n_q)
        self.new = np.arange(3 * blocks, 3 * blocks + 4, dtype=np.int32).reshape(2, 2)
        self.seq, self.pos = ragged([(0, n - T // 2, T // 2), (1, 3, T - T // 2)])
        self.q = kp.queries(T, n_q, d, rng)
        self.w = np.zeros((3 * blocks + 4, n_kv, 64), np.int64)
        bp.weigh(self.pages, self.w, self.tab, self.prm, n_q, *self.q, self.seq, self.pos)
        self.logits = np.rint(rng.normal(0, 130000, (6, 4001))).astype(np.int32)
        self.scores = -rng.integers(0, 1 << 20, (2, 3))
        self.best = bp.select(self.logits, self.scores, 3)
        self.dq = [cuda(torch, x) for x in (*self.q, self.seq, self.pos)]
        self.wt = torch.zeros(self.w.shape, dtype=torch.int64, device="cuda")
        self.lg, self.sc = cuda(torch, self.logits), cuda(torch, self.scores)
        self.nt, self.lens, self.ids = cuda(torch, self.new), cuda(torch, np.array([n, n - 7], np.int32)), cuda(torch, np.arange(2, dtype=np.int32))
        self.moved = (self.pages, self.w.copy())
        self.kept = bp.evict(self.pages, self.moved[1], self.tab, [0, 1], [n, n - 7], 100, 3, 5, self.new)
        torch.cuda.synchronize()

    def calls(self, pkg, stream=None):
        """[the four outputs of selection, weights, kept places]"""
        out = pkg.detint_beam_select(self.lg, self.sc, 3, stream=stream)
        pkg.detint_kv4_weigh_block(self.dev.cache, *self.dq, self.n, self.wt, stream=stream)
        return [*out, pkg.detint_kv4_evict(self.dev.cache, self.wt, self.ids, self.lens, self.n, 100, self.nt, 3, 5, stream=stream)]

    def check(self, got):
        for g, w in zip(got, [*self.best, self.kept]):
            assert np.array_equal(g.cpu().numpy(), w)
        assert np.array_equal(self.wt.cpu().numpy(), self.moved[1])
        self.dev.holds(self.pages)
        assert not self.dev.status.any()


FIRST_CALL = """
import sys
sys.path[:0] = [%(root)r, %(tests)r]
import numpy as np, torch
import deterministic_integer_only_gb300 as pkg
import test_gpu_beam_calls as t
c = t.Case(torch, 5)
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = c.calls(pkg)
g.replay()
torch.cuda.synchronize()
c.check(got)
"""


def test_first_calls_of_a_process_may_be_captured(torch):
    here = os.path.dirname(os.path.abspath(__file__))
    subprocess.run([sys.executable, "-c", FIRST_CALL % dict(root=os.path.dirname(here), tests=here)], check=True, timeout=300)


def test_host_threads_and_streams_at_once(torch):
    """Two host threads, each on a stream of its own, with outputs and
    workspaces made for that stream."""
    import deterministic_integer_only_gb300 as pkg
    cases = [Case(torch, 7), Case(torch, 8, n_q=20, n_kv=4, d=128, n=500, T=300)]

    def work(c):
        s = torch.cuda.Stream()
        for _ in range(10):
            with torch.cuda.stream(s):
                c.wt.zero_()
            got = c.calls(pkg, s)
        s.synchronize()
        return got

    with ThreadPoolExecutor(2) as ex:
        for c, got in zip(cases, list(ex.map(work, cases))):
            c.check(got)


def test_two_captured_selections_with_workspaces_of_their_own(torch):
    import deterministic_integer_only_gb300 as pkg
    a, b = Case(torch, 9), Case(torch, 10)
    graphs, outs = [], []
    for c in (a, b):
        st, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        ws = torch.empty(pkg.detint_beam_workspace(6, 4001, 3), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=st):
            outs.append(pkg.detint_beam_select(c.lg, c.sc, 3, workspace=ws))
        graphs.append((st, g, ws))
    for _ in range(20):
        for st, g, _ in graphs:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for c, out in zip((a, b), outs):
        assert all(np.array_equal(x.cpu().numpy(), w) for x, w in zip(out, c.best))


@pytest.mark.parametrize("block,n_q", [(False, 1), (True, 16)])
def test_weigh_more_tokens_than_a_launch_takes(torch, block, n_q):
    """65600 tokens: past a launch's 65535 tokens, and blocks of one token."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(n_q)
    T, d = 65600, 64
    pages = kp.Pages(4, 1, d, rng)
    tab, prm = np.array([[2, 0], [1, 3]], np.int32), kp.params(1, d, rng, units=90.0)
    dev = Dev(torch, pages, tab, prm, n_q)
    q8, mq, kq = kp.queries(T, n_q, d, rng)
    seq, pos = rng.integers(0, 2, T).astype(np.int32), np.full(T, -1, np.int32)
    live = np.concatenate([[0, 1, 2], rng.integers(3, T, 40), np.arange(65530, 65540), [T - 1]])
    pos[live] = rng.integers(0, 128, len(live))
    w = np.zeros((4, 1, 64), np.int64)
    bp.weigh(pages, w, tab, prm, n_q, q8, mq, kq, seq, pos)
    wt = torch.zeros(w.shape, dtype=torch.int64, device="cuda")
    f = pkg.detint_kv4_weigh_block if block else pkg.detint_kv4_weigh
    f(dev.cache, *(cuda(torch, x) for x in (q8, mq, kq, seq, pos)), 128, wt)
    assert np.array_equal(wt.cpu().numpy(), w) and not dev.status.any()


def test_pools_past_32_bit_offsets(torch):
    """More than 4 GB of keys, of values and of weights: pages at the far end are
    appended to, weighed, copied and moved at the right place."""
    import deterministic_integer_only_gb300 as pkg
    rng = np.random.default_rng(9)
    n_q, n_kv, d = 8, 8, 64
    nb = (1 << 32) // (n_kv * 64 * 8) + 70
    k, v = (torch.zeros((nb, n_kv, 64, d // 2), dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((nb, n_kv, 64), dtype=torch.uint8, device="cuda") for _ in range(2))
    wt = torch.zeros((nb, n_kv, 64), dtype=torch.int64, device="cuda")
    small = kp.Pages(7, n_kv, d, rng)
    far = np.array([nb - 1, nb - 68, 1, nb - 2, nb - 3, nb - 5, 4], np.int32)
    at = cuda(torch, far.astype(np.int64))
    pk, pv = small.packed()
    k[at], v[at], ks[at], vs[at] = cuda(torch, pk), cuda(torch, pv), cuda(torch, small.ck), cuda(torch, small.cv)
    tab = np.array([[0, 1, 2]], np.int32)
    prm = kp.params(n_kv, d, rng, units=90.0)
    cache = pkg.KV4Cache(k, v, ks, vs, cuda(torch, far[tab]), cuda(torch, prm), n_q)
    seq, pos = ragged([(0, 60, 9), (0, 130, 62)])
    cos, sin = tables(d, 200)
    qkv = np.rint(rng.normal(0, 4096, (len(pos), 24 * d))).astype(np.int32)
    rp = rng.integers(0, 200, (1, len(pos))).astype(np.int32)
    want = append_axes_plain(small, tab, prm, n_q, cos, sin, False, (None, None), 0, qkv, seq, pos, rp, np.zeros(32, np.uint8))
    q = pkg.detint_kv4_append_axes(cache, pkg.RopeNorm(cuda(torch, cos), cuda(torch, sin)), cuda(torch, qkv), cuda(torch, seq),
                                   cuda(torch, pos), cuda(torch, rp))
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(q, want))
    w = np.zeros((7, n_kv, 64), np.int64)
    for f in (pkg.detint_kv4_weigh, pkg.detint_kv4_weigh_block):
        f(cache, *q, cuda(torch, seq), cuda(torch, pos), 192, wt)
        bp.weigh(small, w, tab, prm, n_q, *want[:3], seq, pos)
    kept = pkg.detint_kv4_evict(cache, wt, cuda(torch, np.zeros(1, np.int32)), cuda(torch, np.array([192], np.int32)), 192, 100,
                                cuda(torch, far[[[3, 4]]]), 2, 3)
    assert np.array_equal(kept.cpu().numpy(), bp.evict(small, w, tab, [0], [192], 100, 2, 3, np.array([[3, 4]])))
    pkg.detint_kv4_copy(cache, cuda(torch, far[[3, 4]]), cuda(torch, far[[5, 6]]), weight=wt)
    for x in (small.k, small.v, small.ck, small.cv, w):
        x[5], x[6] = x[3], x[4]
    pk, pv = small.packed()
    for got, exp in ((k, pk), (v, pv), (ks, small.ck), (vs, small.cv), (wt, w)):
        assert np.array_equal(got[at].cpu().numpy(), exp)


def test_binding_refusals(torch):
    import deterministic_integer_only_gb300 as pkg
    c = Case(torch, 3)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    bad = [
        lambda: pkg.detint_beam_select(c.lg[:5], c.sc, 3),
        lambda: pkg.detint_beam_select(c.lg.long(), c.sc, 3),
        lambda: pkg.detint_beam_select(c.lg, c.sc.int(), 3),
        lambda: pkg.detint_beam_select(c.lg, c.sc.view(-1), 3),
        lambda: pkg.detint_beam_select(c.lg, c.sc, 3, done=i32(5), end_id=1),
        lambda: pkg.detint_beam_select(c.lg, c.sc, 3, out=(i32(6), i32(6), i32(6), i32(6))),
        lambda: pkg.detint_beam_select(c.lg, c.sc, 3, out=(i32(6), i32(5), c.sc, i32(6))),
        lambda: pkg.detint_beam_select(c.lg, c.sc, 3, workspace=torch.zeros(1 << 20, dtype=torch.uint8)),
        lambda: pkg.detint_beam_select(c.lg.t().contiguous().t(), c.sc, 3),
        lambda: pkg.detint_beam_reorder(i32(6, 4), i32(2, 4), i32(2)),
        lambda: pkg.detint_beam_reorder(i32(6, 4), i32(2, 3), i32(1)),
        lambda: pkg.detint_beam_reorder(i32(6, 4), i32(2, 3), i32(2), out=i32(6, 3)),
        lambda: pkg.detint_beam_reorder(i32(6, 4), i32(2, 3), i32(2), dst=i32(5)),
        lambda: pkg.detint_kv4_copy(c.dev.cache, i32(3), i32(2)),
        lambda: pkg.detint_kv4_copy(c.dev.cache, i32(3), i32(3), weight=c.wt[:2]),
        lambda: pkg.detint_kv4_copy(c.dev.cache, i32(3).long(), i32(3)),
        lambda: pkg.detint_kv4_weigh(c.dev.cache, *c.dq, c.n, c.wt.int()),
        lambda: pkg.detint_kv4_weigh(c.dev.cache, *c.dq, c.n, c.wt[:3]),
        lambda: pkg.detint_kv4_weigh_block(c.dev.cache, c.dq[0][:3], *c.dq[1:], c.n, c.wt),
        lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens[:1], c.n, 100, c.nt),
        lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens, c.n, 200, c.nt),
        lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens, c.n, 100, c.nt, kept=i32(10)),
        lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt.cpu(), c.ids, c.lens, c.n, 100, c.nt),
        lambda: pkg.detint_kv4_append_axes(c.dev.cache, pkg.RopeNorm(None, None, max_pos=9), i32(3, 12 * 64), i32(3), i32(3), i32(2, 2)),
        lambda: pkg.detint_kv4_append_axes(c.dev.cache, pkg.RopeNorm(None, None, max_pos=9), i32(3, 12 * 64), i32(3), i32(3), i32(3).long()),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for f in (lambda: pkg.detint_beam_select(c.lg, c.sc, 0), lambda: pkg.detint_beam_select(c.lg, c.sc, 65),
              lambda: pkg.detint_beam_select(c.lg, c.sc, (1 << 32) + 3), lambda: pkg.detint_beam_select(c.lg, c.sc, 3, end_id=4001),
              lambda: pkg.detint_beam_select(c.lg, c.sc, 3, end_id=1 << 33),
              lambda: pkg.detint_beam_select(c.lg, c.sc, 3, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda")),
              lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens, c.n, 0, c.nt),
              lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens, c.n, 100, c.nt, sinks=101),
              lambda: pkg.detint_kv4_evict(c.dev.cache, c.wt, c.ids, c.lens, (1 << 32) + 64, 100, c.nt),
              lambda: pkg.detint_kv4_weigh(c.dev.cache, *c.dq, 1 << 32, c.wt),
              lambda: pkg.detint_kv4_weigh(c.dev.cache, *c.dq, c.n, c.wt, window=-1),
              lambda: pkg.detint_kv4_append_axes(c.dev.cache, pkg.RopeNorm(None, None, max_pos=9), i32(3, 12 * 64), i32(3), i32(3), i32(5, 3))):
        with pytest.raises(pkg.DetintError):
            f()
    assert not c.wt.any() and not c.dev.status.any()
