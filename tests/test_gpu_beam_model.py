"""Beam search of whole models: tokens and scores against a plain search whose
logits are the oracle's for each hypothesis fed afresh, and the reordering of
sequences that it rests on."""
import numpy as np
import pytest

import beam_plain as bp
import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    oracle.set_threads(oracle.max_threads())
    return pkg


class Fed:
    """The oracle's logits after a list of tokens, continued where a prefix is held."""

    def __init__(self, path, kv_bits, room):
        self.m, self.room, self.rows = oracle.Model(path, kv_bits=kv_bits), room, {}

    def __call__(self, tokens):
        key = tuple(tokens)
        if key not in self.rows:
            s = self.m.new_seq(self.room)
            self.rows[key] = s.feed(np.asarray(tokens, np.int32))[1]
        return self.rows[key]


def plain_search(fed, prompt, beams, steps, end):
    """([beams][steps] tokens, [beams] scores): every hypothesis fed to the oracle afresh at every step."""
    par, tok, score, done = bp.select(fed(prompt)[None], np.zeros((1, 1), np.int64), beams, None, end)
    hyps = [[int(t)] for t in tok[0]]
    for _ in range(steps - 1):
        if end >= 0 and done.all():
            break
        rows = np.stack([fed(list(prompt) + h) for h in hyps])
        par, tok, score, done = bp.select(rows, score, beams, done if end >= 0 else None, end)
        hyps = [hyps[p] + [int(t)] for p, t in zip(par[0], tok[0])]
    fill = end if end >= 0 else 0
    return np.array([h + [fill] * (steps - len(h)) for h in hyps], np.int32), score[0]


@pytest.mark.parametrize("kv_bits", [8, 4])
@pytest.mark.parametrize("beams,lens,steps", [(1, [7], 5), (3, [60, 64, 33], 12), (4, [5], 70)])
def test_beam_search(pkg, tiny_artifact, kv_bits, beams, lens, steps):
    fed = Fed(tiny_artifact, kv_bits, 160)
    prompts = [synth.prompt_ids(3, i, n, 1024) for i, n in enumerate(lens)]
    m = pkg.Model(tiny_artifact, max_batch=len(lens) * beams, max_ctx=160, kv_bits=kv_bits)
    toks, scores = m.beam_search(prompts, beams, steps)
    for g, p in enumerate(prompts):
        want, ws = plain_search(fed, list(p), beams, steps, -1)
        assert np.array_equal(toks[g], want) and np.array_equal(scores[g], ws)
    assert (m.status() == 0).all()
    if beams == 1:                                       # one beam is the greedy decode
        m.reset_seq(0)
        greedy, _ = m.generate(prompts, steps, keep_logits=False)
        assert np.array_equal(toks[:, 0], greedy)
    m.close()


def test_beam_search_ends(pkg, tiny_artifact):
    """An end token that the search meets: finished beams keep their score and
    fill up with it; once all have, the search is over."""
    prompt = list(synth.prompt_ids(3, 9, 20, 1024))
    fed = Fed(tiny_artifact, 8, 64)
    free, _ = plain_search(fed, prompt, 4, 8, -1)
    for end in {int(free[0, 1]), int(free[2, 3]), int(free[0, 0])}:
        m = pkg.Model(tiny_artifact, max_batch=4, max_ctx=64)
        toks, scores = m.beam_search([prompt], 4, 8, end_id=end)
        want, ws = plain_search(fed, prompt, 4, 8, end)
        assert np.array_equal(toks[0], want) and np.array_equal(scores[0], ws)
        m.close()


@pytest.mark.parametrize("kv_bits", [8, 4])
def test_reorder_seqs_equals_fresh_prefills(pkg, tiny_artifact, kv_bits):
    """Sequences of different lengths, swapped, repeated and dropped: each
    continues as its parent would, and every block comes back in the end."""
    import torch
    m = pkg.Model(tiny_artifact, max_batch=5, max_ctx=192, kv_bits=kv_bits)
    dev = torch.device("cuda")
    rng = np.random.default_rng(2)
    text = [list(rng.integers(0, 1024, n)) for n in (64, 70, 1, 130, 63)]
    one = oracle.Model(tiny_artifact, kv_bits=kv_bits)

    def prefill(ids, chunks):
        lg = torch.empty((len(ids), m.vocab), dtype=torch.int32, device=dev)
        cu = np.concatenate([[0], np.cumsum([len(c) for c in chunks])])
        m.prefill(ids, torch.tensor(np.concatenate(chunks), dtype=torch.int32, device=dev), cu, lg)
        m.stream.synchronize()
        return lg.cpu().numpy()

    with torch.cuda.stream(m.stream):
        prefill(range(5), text)
        for parents in ([1, 0, 2, 3, 4], [3, 3, 3, 3, 3], [0, 1, 2, 3, 4], [4, 4, 1, 1, 0], [2, 0, 2, 0, 2]):
            m.reorder_seqs([0, 1, 2, 3, 4], parents)
            text = [list(text[p]) for p in parents]
            assert [m.seq_len(i) for i in range(5)] == [len(t) for t in text]
            tok = torch.tensor([7 * i + len(parents) for i in range(5)], dtype=torch.int32, device=dev)
            lg = torch.empty((5, m.vocab), dtype=torch.int32, device=dev)
            m.decode_step(range(5), tok, lg)
            m.stream.synchronize()
            for i, t in enumerate(text):
                t.append(int(tok[i]))
                assert np.array_equal(lg[i].cpu().numpy(), one.new_seq(192).feed(np.asarray(t, np.int32))[1]), (parents, i)
        m.reorder_seqs([3, 1], [1, 0])                   # some of them only
        text[1], text[3] = text[3], text[1]
        lg = prefill([1, 3], [[5], [6, 7]])
        for row, t in ((0, text[1] + [5]), (1, text[3] + [6, 7])):
            assert np.array_equal(lg[row], one.new_seq(192).feed(np.asarray(t, np.int32))[1])
        for i in range(5):
            m.reset_seq(i)
        prefill(range(5), [list(rng.integers(0, 1024, 192)) for _ in range(5)])      # the whole pool again
    assert (m.status() == 0).all()
    m.close()


def test_reorder_seqs_refusals(pkg, tiny_artifact):
    m = pkg.Model(tiny_artifact, max_batch=4, max_ctx=64)
    for code, ids, parents in ((9, [0, 0], [0, 1]), (9, [0, 4], [0, 1]), (9, [-1], [0]), (1, [0, 1], [0, 2]), (1, [0], [-1]),
                               (1, [0, 1, 2, 3, 0], [0] * 5), (1, [], [])):
        with pytest.raises(pkg.DetintError) as e:
            m.reorder_seqs(ids, parents)
        assert e.value.code == code
    with pytest.raises(ValueError):
        m.reorder_seqs([0, 1], [0])
    with pytest.raises(ValueError):
        m.beam_search([[1, 2]], 0, 3)
    with pytest.raises(ValueError):
        m.beam_search([[1, 2]], 2, 3, seq_ids=[0])
    with pytest.raises(pkg.DetintError):
        m.beam_search([[1, 2]], 5, 3)                    # more sequences than the model has
    m.close()
