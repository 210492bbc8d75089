"""Beam search, weights and eviction without a GPU: the plain forms against
float64 and closed forms, and the refusals of the entry points, whose argument
checks come before the first CUDA call."""
import ctypes as C

import numpy as np
import pytest

import beam_plain as bp
from test_kv4_host import P, _cache, _rope


@pytest.fixture(scope="module")
def L():
    from deterministic_integer_only_gb300 import binding, build
    build.build()
    return binding.lib()


# ------------------------------------------------------------- plain forms
@pytest.mark.parametrize("n,spread", [(1, 1.0), (2, 0.0), (1000, 0.1), (151936, 2.0), (151936, 0.0), (5000, 12.0)])
def test_lse_against_float64(n, spread):
    """The exponent's rounding is half of 2^-10 octaves, L2E's relative error 4.9e-6
    over at most 31 octaves: (2^-11 + 31 * 4.9e-6) ln 2 = 4.5e-4 relative for each
    exponential; the cubic adds 2^-13, an exponential's own rounding and those
    dropped at 31 octaves 2^-31 each of the largest; the logarithm's cut 2^-20
    octaves, its rounding 2^-17, LN2's error 7e-7 of at most 24 octaves."""
    rng = np.random.default_rng(n)
    row = np.rint(rng.normal(0, spread * 65536, n)).astype(np.int64)
    want = np.log(np.exp((row - row.max()) / 65536.0).sum()) + row.max() / 65536.0
    bound = 4.5e-4 + 2.0 ** -13 + n * 2.0 ** -30 + 2.0 ** -20 + 2.0 ** -17 + 24 * 7e-7
    assert abs(bp.lse(row) / 65536.0 - want) <= bound


def test_lse_of_one_logit_is_the_logit():
    for x in (0, 1, -(1 << 31) + 1, (1 << 31) - 1):
        assert bp.lse(np.array([x], np.int64)) == x
        assert bp.lse(np.array([x] * 4, np.int64)) == x + 90852      # ln 4 in Q16: 90852.1


def test_select_orders_ties_by_beam_then_token():
    logits = np.zeros((2, 8), np.int32)
    par, tok, score, end = bp.select(logits, np.zeros((1, 2), np.int64), 10, end_id=3)
    assert par[0].tolist() == [0] * 8 + [1] * 2 and tok[0].tolist() == [*range(8), 0, 1]
    assert (score == -136278).all() and end[0].tolist() == [0, 0, 0, 1, 0, 0, 0, 0, 0, 0]     # ln 8: 136278.2


def test_probabilities_sum_to_one():
    """Each of n probabilities is rounded by half, RS by less than one unit of at
    least 2^23: the sum is 2^24 within n / 2 + 2."""
    rng = np.random.default_rng(0)
    for n in (1, 2, 63, 1000):
        k4, ck = rng.integers(-7, 8, (n, 64)), rng.integers(1, 256, n)
        p = bp.probabilities(rng.integers(-127, 128, 64), 20000, 21, k4, ck, [0] * 6 + [20000, 22])
        assert abs(int(p.sum()) - (1 << 24)) <= n / 2 + 2


# --------------------------------------------------------------- refusals
def _select(L, **kw):
    v = dict(logits=P, stride=100, n=100, scores=P, done=None, groups=2, beams=3, end=-1, n_out=4, parent=P, token=P, score=P,
             done_out=P, ws=P, size=1 << 20)
    v.update(kw)
    return L.detint_beam_select(v["logits"], v["stride"], v["n"], v["scores"], v["done"], v["groups"], v["beams"], v["end"],
                                v["n_out"], v["parent"], v["token"], v["score"], v["done_out"], v["ws"], v["size"], None)


@pytest.mark.parametrize("code,change", [
    (1, dict(logits=None)), (1, dict(scores=None)), (1, dict(parent=None)), (1, dict(token=None)), (1, dict(score=None)),
    (1, dict(done_out=None)), (1, dict(ws=None)), (1, dict(size=100)), (1, dict(ws=P + 8)), (1, dict(groups=0)),
    (1, dict(beams=0)), (1, dict(beams=65)), (1, dict(n_out=0)), (1, dict(n_out=65)), (1, dict(groups=21846)),
    (2, dict(n=0)), (2, dict(n=(1 << 24) + 1, stride=1 << 25)), (1, dict(stride=99)), (1, dict(end=100)), (1, dict(end=-2)),
    (1, dict(done=P)), (1, dict(done=P + 2, end=3)), (1, dict(logits=P + 1)), (1, dict(scores=P + 4)), (1, dict(score=P + 4)),
    (1, dict(token=P + 2)), (1, dict(groups=-1)), (1, dict(stride=-100))])
def test_bad_select_arguments_are_refused(L, code, change):
    assert _select(L, **change) == code
    assert b"detint_beam" in L.detint_last_error()


@pytest.mark.parametrize("args", [(0, 10, 1), (1, 0, 1), (1, 10, 0), (1, 10, 65), (65536, 10, 1), (1, (1 << 24) + 1, 1)])
def test_bad_workspace_queries_are_refused(L, args):
    assert L.detint_beam_workspace(*args, C.byref(C.c_longlong())) == 1
    assert L.detint_beam_workspace(1, 10, 1, None) == 1


def test_workspace_covers_smaller_calls(L):
    def need(*a):
        v = C.c_longlong()
        assert L.detint_beam_workspace(*a, C.byref(v)) == 0
        return v.value
    assert need(12, 500, 8) >= max(need(11, 500, 8), need(12, 500, 7), need(1, 100, 1)) > 0
    assert need(12, 500, 8) >= 12 * 8 * 12


@pytest.mark.parametrize("code,change", [
    (1, dict(table=None)), (1, dict(out=None)), (1, dict(parent=None)), (1, dict(lens=None)), (1, dict(src=None)),
    (1, dict(dst=None)), (1, dict(blocks=0)), (1, dict(groups=0)), (1, dict(groups=65536)), (1, dict(beams=0)),
    (1, dict(beams=65)), (1, dict(table=P + 2)), (1, dict(lens=P + 1)), (1, dict(dst=P + 3))])
def test_bad_reorder_arguments_are_refused(L, code, change):
    v = dict(table=P, out=P, blocks=4, parent=P, lens=P, groups=2, beams=3, src=P, dst=P)
    v.update(change)
    assert L.detint_beam_reorder(v["table"], v["out"], v["blocks"], v["parent"], v["lens"], v["groups"], v["beams"], v["src"],
                                 v["dst"], None) == code


def _axes(L, c=None, r=None, **kw):
    v = dict(rp=P, axis=P, n_axes=3, qkv=P, stride=12 * 64, seq=P, pos=P, n=3, q8=P, mq=P, kq=P, kv=None, vv=None)
    v.update(kw)
    c, r = c or _cache(), r or _rope()
    return L.detint_kv4_append_axes(C.addressof(c), C.addressof(r), v["rp"], v["axis"], v["n_axes"], v["qkv"], v["stride"],
                                    v["seq"], v["pos"], v["n"], v["q8"], v["mq"], v["kq"], v["kv"], v["vv"], None)


@pytest.mark.parametrize("code,change", [
    (1, dict(rp=None)), (1, dict(axis=None)), (1, dict(n_axes=0)), (1, dict(n_axes=5)), (1, dict(n_axes=-1)), (1, dict(rp=P + 2)),
    (1, dict(qkv=None)), (1, dict(n=0)), (1, dict(stride=12 * 64 - 4)), (1, dict(q8=P + 8)), (1, dict(pos=P + 2))])
def test_bad_axes_arguments_are_refused(L, code, change):
    assert _axes(L, **change) == code
    assert b"detint_kv4_append_axes" in L.detint_last_error()


def test_axes_refuse_what_append_refuses(L):
    for code, change in ((2, dict(rot_dim=72)), (1, dict(cos=None)), (1, dict(max_pos=0)), (1, dict(q_gamma=P)), (1, dict(eps=-1))):
        assert _axes(L, r=_rope(**change)) == code
    for code, change in ((2, dict(head_dim=96)), (1, dict(k=None)), (2, dict(n_q=7))):
        assert _axes(L, _cache(**change)) == code


def _weigh(L, which, c=None, **kw):
    v = dict(q8=P, mq=P, kq=P, seq=P, pos=P, n=3, max_len=100, window=0, weight=P)
    v.update(kw)
    c = c or _cache()
    f = L.detint_kv4_weigh if which == "weigh" else L.detint_kv4_weigh_block
    return f(C.addressof(c), v["q8"], v["mq"], v["kq"], v["seq"], v["pos"], v["n"], v["max_len"], v["window"], v["weight"], None)


@pytest.mark.parametrize("which", ["weigh", "weigh_block"])
@pytest.mark.parametrize("code,change", [
    (1, dict(weight=None)), (1, dict(weight=P + 8)), (1, dict(q8=None)), (1, dict(mq=None)), (1, dict(kq=None)),
    (1, dict(seq=None)), (1, dict(pos=None)), (1, dict(n=0)), (1, dict(max_len=0)), (1, dict(max_len=(1 << 19) + 1)),
    (1, dict(window=-1)), (1, dict(q8=P + 4)), (1, dict(pos=P + 2)), (1, dict(kq=P + 1))])
def test_bad_weigh_arguments_are_refused(L, which, code, change):
    assert _weigh(L, which, **change) == code
    assert b"detint_kv4_" + which.encode() in L.detint_last_error()


def _evict(L, c=None, **kw):
    v = dict(weight=P, seq=P, lens=P, n=2, max_len=100, keep=50, sinks=4, recent=8, table=P, kept=P)
    v.update(kw)
    c = c or _cache()
    return L.detint_kv4_evict(C.addressof(c), v["weight"], v["seq"], v["lens"], v["n"], v["max_len"], v["keep"], v["sinks"],
                              v["recent"], v["table"], v["kept"], None)


@pytest.mark.parametrize("code,change", [
    (1, dict(weight=None)), (1, dict(seq=None)), (1, dict(lens=None)), (1, dict(table=None)), (1, dict(kept=None)), (1, dict(n=0)),
    (1, dict(n=65536)), (1, dict(max_len=0)), (1, dict(max_len=(1 << 19) + 1)), (1, dict(keep=0)), (1, dict(keep=(1 << 19) + 1)),
    (1, dict(sinks=-1)), (1, dict(recent=-1)), (1, dict(sinks=43)), (1, dict(recent=47)), (1, dict(sinks=(1 << 31) - 1)),
    (1, dict(weight=P + 8)), (1, dict(lens=P + 2)), (1, dict(kept=P + 1))])
def test_bad_evict_arguments_are_refused(L, code, change):
    assert _evict(L, **change) == code


def test_bad_copies_and_caches_are_refused(L):
    for change in (dict(k=None), dict(n_kv=0), dict(head_dim=96), dict(k=P + 8), dict(status=P + 2)):
        c = _cache(**change)
        code = 2 if "n_kv" in change or "head_dim" in change else 1
        assert _evict(L, c) == code and _weigh(L, "weigh", c) == code and _weigh(L, "weigh_block", c) == code
        assert L.detint_kv4_copy(C.addressof(c), P, P, 3, None, None) == code
    c = _cache()
    for a in ((None, P, 3, None), (P, None, 3, None), (P, P, 0, None), (P, P, -1, None), (P + 2, P, 3, None), (P, P, 3, P + 8)):
        assert L.detint_kv4_copy(C.addressof(c), *a, None) == 1


def test_the_binding_refuses_cpu_tensors_and_wide_integers():
    torch = pytest.importorskip("torch")
    import deterministic_integer_only_gb300 as pkg
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="cuda"):
        pkg.detint_beam_select(i32(4, 100), torch.zeros(2, 2, dtype=torch.int64), 2)
    with pytest.raises(ValueError, match="cuda"):
        pkg.detint_beam_reorder(i32(4, 8), i32(2, 2), i32(2))
    for a in (((1 << 32) + 1, 10, 1), (1, (1 << 32) + 10, 1), (1, 10, (1 << 32) + 1)):
        with pytest.raises(pkg.DetintError):
            pkg.detint_beam_workspace(*a)
