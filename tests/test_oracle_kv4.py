"""Pins of the oracle's 4-bit K/V cache (arithmetic specification, section 16):
the quantiser against exact rationals, the parameter conversion against the
real scales it stands for, the attention row against a float64 softmax with a
bound derived from its roundings, closed forms, one decoder layer recomposed
from the oracle's primitives, and the prefill / decode invariance at
tolerance 0."""
from fractions import Fraction

import numpy as np
import pytest

import float_model
import oracle
import synth


def test_quant4_is_nearest_with_the_smallest_scale_code():
    rng = np.random.default_rng(0)
    rows = [rng.integers(-a, a + 1, 64) for a in (1, 3, 7, 8, 50, 127, 700, 1785) for _ in range(20)]
    rows += [np.zeros(64, np.int64), np.full(64, 1785), np.full(64, -1785), np.eye(64, dtype=np.int64)[3] * 1779]
    x = np.array(rows)
    q, c = oracle.quant4(x)
    for r in range(len(x)):
        a = int(np.abs(x[r]).max())
        assert c[r] == max(1, -(-a // 7)) and 1 <= c[r] <= 255
        assert np.abs(q[r]).max() <= 7
        # q = nearest of x R / 2^(b+16) with R within one of 2^(b+16) / c: off
        # x / c by at most 1/2 + |x| / 2^(b+16), |x| <= 7 c < 7 2^b
        for xi, qi in zip(x[r], q[r]):
            assert abs(Fraction(int(xi), int(c[r])) - int(qi)) <= Fraction(1, 2) + Fraction(7, 1 << 16)


def test_kv4_params_stand_for_the_scales_in_fourteenths(tiny_artifact):
    art = float_model.load(tiny_artifact)
    d = art["d"]
    for ly in art["layers"]:
        for kvp in ly["kvp"]:
            p = [int(v) for v in oracle.kv4_params(kvp, d)]
            k = [int(v) for v in kvp]
            assert Fraction(p[0], 1 << p[1]) == 14 * Fraction(k[0], 1 << k[1])
            assert Fraction(p[2], 1 << p[3]) == 14 * Fraction(k[2], 1 << k[3])
            # a dyadic mantissa of at least 2^14 rounds by at most half a unit
            for got, want in ((Fraction(p[4], 1 << p[5]), Fraction(128 * k[4], 14 << k[5])),
                              (Fraction(p[6], 1 << p[7]), Fraction(k[6], 14 << k[7]))):
                assert abs(got / want - 1) <= Fraction(1, 1 << 15)
            assert p[8:] == k[8:] + k[8:]


def _row_case(rng, ctx, d, spread):
    K = rng.integers(-7, 8, (ctx, d))
    V = rng.integers(-7, 8, (ctx, d))
    ck = rng.integers(100, 256, ctx)
    cv = rng.integers(1, 256, ctx)
    q = rng.integers(-127, 128, d)
    mq, kq = int(rng.integers(1 << 14, 1 << 15)), 20
    cstm, cstk = 1 << 14, int(round(14 + np.log2(1.0 / spread)))
    mv, kv = 20000, 22
    return q, mq, kq, K, ck, V, cv, np.array([1, 0, 1, 0, mv, kv, cstm, cstk] + [0] * d, np.int32)


@pytest.mark.parametrize("ctx,d,spread", [(1, 64, 1e-3), (2, 64, 1e-3), (40, 64, 1e-3), (300, 128, 1e-3), (300, 128, 1e-5),
                                          (1000, 64, 1e-2)])
def test_attention4_row_vs_float64(ctx, d, spread):
    rng = np.random.default_rng(ctx + d)
    for _ in range(5):
        q, mq, kq, K, ck, V, cv, prm = _row_case(rng, ctx, d, spread)
        o, sigma = oracle.attention4_row(q, mq, kq, K, ck, V, cv, prm)
        u = (K @ q) * ck * (mq / 2.0 ** kq) * (prm[6] / 2.0 ** float(prm[7]))       # base-2 logits
        p = 2.0 ** (u - u.max())
        p /= p.sum()
        unit = prm[4] / 2.0 ** float(prm[5]) / 128.0                                # real value of a cached unit
        want = (p[:, None] * (V * cv[:, None])).sum(0) * unit * 4096.0
        # each E: the exponent is off by half a unit of 2^-10 (a factor within
        # 2^(1/2048)), exp2q by 2^-13, the rounding and the cap at 2^15 - 1 by one
        # unit; numerator and denominator both carry it. W adds half a unit of
        # 128 / Sigma per key, the division and the two shifts half a unit each.
        big = np.abs(V * cv[:, None]).max()
        rel = 2.0 ** (1 / 2048.0) - 1 + 2.0 ** -13
        tol = (2 * (rel + ctx / sigma) * big + 64.0 * 7 * ctx / sigma) * unit * 4096.0
        tol += np.abs(want) * 2.0 ** -22 + unit * 4096.0 * 128 * 2.0 ** -16 + 1.0
        assert (np.abs(o - want) <= tol).all(), (np.abs(o - want).max(), tol.min())


def test_attention4_row_closed_forms():
    rng = np.random.default_rng(1)
    q, mq, kq, K, ck, V, cv, prm = _row_case(rng, 6, 64, 1e-3)
    # no key: zeros; one key: its own values, whatever the score
    o, sigma = oracle.attention4_row(q, mq, kq, K, ck, V, cv, prm, first=6)
    assert not o.any() and sigma == 0
    o, sigma = oracle.attention4_row(q, mq, kq, K[:1], ck[:1], V[:1], cv[:1], prm)
    assert sigma == 32767
    W = (32767 * int(cv[0]) + 64) >> 7
    RS = (1 << (15 + 23)) // 32767
    for c in range(64):
        t = (W * int(V[0, c]) * RS + (1 << 21)) >> 22
        assert o[c] == (t * int(prm[4]) + (1 << 25)) >> 26
    # a window is the same keys alone; a zero query weighs all keys alike
    o1, _ = oracle.attention4_row(q, mq, kq, K, ck, V, cv, prm, first=4)
    o2, _ = oracle.attention4_row(q, mq, kq, K[4:], ck[4:], V[4:], cv[4:], prm)
    assert np.array_equal(o1, o2)
    _, sigma = oracle.attention4_row(np.zeros(64), 0, 0, K, ck, V, cv, prm)
    assert sigma == 6 * 32767


def test_one_layer_recomposed_from_primitives(tiny_artifact):
    """The model's 4-bit path of layer 0, token by token, from the oracle's own
    row functions in Python: parameter conversion, head mapping, cache use."""
    art = float_model.load(tiny_artifact)
    m = oracle.Model(tiny_artifact, kv_bits=4)
    prompt = synth.prompt_ids(0, 3, 9, m.vocab)
    seq = m.new_seq(16)
    nq, nkv, d, H, half = art["nq"], art["nkv"], art["d"], art["H"], art["d"] // 2
    ly = art["layers"][0]
    eps_h, eps_qk = int(round(art["eps"] * 2 ** 32)), int(round(1e-6 * 2 ** 24))
    prm = np.array([oracle.kv4_params(ly["kvp"][g], d) for g in range(nkv)])
    K, V = [[] for _ in range(nkv)], [[] for _ in range(nkv)]
    ck, cv = [[] for _ in range(nkv)], [[] for _ in range(nkv)]

    def lin(x, F, w, mw, fout):
        q8, mt, kt = x
        return oracle.requant(oracle.gemm_i8(q8, w).ravel(), int(mt[0]), int(kt[0]), mw, fout)

    sat = lambda x, b: np.clip(x, -b, b)  # noqa: E731
    for pos, tok in enumerate(prompt):
        _, _, hid = seq.feed([tok], want_hidden=True)
        h = hid[0].astype(np.int64)
        qkv = sat(lin(oracle.normquant(h, ly["attn_gamma"], eps_h), 0, ly["w_qkv"], ly["m_qkv"], 12), 2 ** 31 - 1)
        rows = qkv.reshape(nq + 2 * nkv, d)
        c, s = art["rope_cos"][pos], art["rope_sin"][pos]
        o = np.empty((nq, d), np.int64)
        for g in range(nkv):
            e = prm[g, 8:].astype(np.int64)
            y = oracle.rope(oracle.qknorm(rows[nq + g], ly["k_gamma"], eps_qk)[0], c, s).astype(np.int64)
            for x, ks, vs in ((sat(oracle.rshr((y << e) * int(prm[g, 0]), prm[g, 1]), 1785), K, ck),
                              (sat(oracle.rshr(rows[nq + nkv + g] * int(prm[g, 2]), prm[g, 3]), 1785), V, cv)):
                q4, code = oracle.quant4(x)
                ks[g].append(q4[0])
                vs[g].append(code[0])
        for hq in range(nq):
            g = hq // (nq // nkv)
            e = prm[g, 8:].astype(np.int64)
            y = oracle.rope(oracle.qknorm(rows[hq], ly["q_gamma"], eps_qk)[0], c, s).astype(np.int64) << (e.max() - e)
            q8, mq, kq = oracle.actquant(y, 14)
            o[hq], _ = oracle.attention4_row(q8[0], mq[0], kq[0], np.array(K[g]), np.array(ck[g]), np.array(V[g]),
                                             np.array(cv[g]), prm[g])
        h = sat(h + sat(lin(oracle.actquant(o.ravel(), 12), 12, ly["w_o"], ly["m_o"], 16), 2 ** 31 - 1), 2 ** 31 - 1)
        x = oracle.normquant(h, ly["ffn_gamma"], eps_h)
        gt, up = (sat(lin(x, 0, ly["w_" + n], ly["m_" + n], 12), 1 << 24) for n in ("gate", "up"))
        h = sat(h + sat(lin(oracle.actquant(oracle.swiglu(gt, up), 10), 10, ly["w_down"], ly["m_down"], 16), 2 ** 31 - 1),
                2 ** 31 - 1)
        assert np.array_equal(h, hid[1])


def test_kv4_prefill_equals_token_by_token(tiny_artifact):
    m = oracle.Model(tiny_artifact, kv_bits=4)
    prompt = synth.prompt_ids(0, 0, 33, m.vocab)
    _, want = m.new_seq(64).feed(prompt)
    for cut in (1, 16, 32):
        s = m.new_seq(64)
        s.feed(prompt[:cut])
        _, got = s.feed(prompt[cut:])
        assert np.array_equal(got, want)
    # a cache of its own: the 8-bit model gives other logits
    _, other = oracle.Model(tiny_artifact).new_seq(64).feed(prompt)
    assert not np.array_equal(other, want)
