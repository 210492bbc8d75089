"""Models with the 4-bit K/V cache on the GPU against the oracle's, bit for
bit: prefill, decode, batches, split prefill, forked prefixes, contexts that
cross pages and the decode attention's forms, graphs on and off, 16-bit
weights."""
import numpy as np
import pytest

import oracle
import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import deterministic_integer_only_gb300 as pkg
    pkg.lib()
    return torch


def oracle_run(path, prompt, steps, ctx=1024):
    s = oracle.Model(path, kv_bits=4).new_seq(ctx)
    am, lg = s.feed(prompt)
    toks, rows = [am], [lg]
    for _ in range(steps - 1):
        am, lg = s.feed([am])
        toks.append(am)
        rows.append(lg)
    return toks, rows


@pytest.mark.parametrize("graph,fused", [(True, True), (False, True), (True, False)])
def test_tiny_ragged_batch_equals_the_oracle(torch, tiny_artifact, graph, fused):
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(tiny_artifact, max_batch=4, max_ctx=256, kv_bits=4)
    m.set_graph(graph)
    m.set_fused_decode(fused)
    prompts = [synth.prompt_ids(0, i, n, m.vocab) for i, n in enumerate((1, 16, 63, 130))]
    toks, rows = m.generate(prompts, 12)
    for b, p in enumerate(prompts):
        wt, wr = oracle_run(tiny_artifact, p, 12)
        assert toks[b].tolist() == wt
        assert all(np.array_equal(rows[s][b], wr[s]) for s in range(12))
    assert not m.status().any()


def test_tiny_contexts_across_graph_sizes(torch, tiny_artifact):
    """Decode steps from 505 on: the captured graph's context bound of 512 is
    left for the next one."""
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(tiny_artifact, max_batch=1, max_ctx=1024, kv_bits=4)
    p = synth.prompt_ids(0, 5, 505, m.vocab)
    toks, rows = m.generate([p], 14)
    wt, wr = oracle_run(tiny_artifact, p, 14)
    assert toks[0].tolist() == wt
    assert all(np.array_equal(rows[s][0], wr[s]) for s in range(14))


def test_tiny_split_prefill_and_fork(torch, tiny_artifact):
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(tiny_artifact, max_batch=3, max_ctx=256, kv_bits=4)
    p = synth.prompt_ids(0, 2, 100, m.vocab)
    _, want = oracle_run(tiny_artifact, p, 2)
    dev = lambda a: torch.tensor(np.asarray(a, np.int32), device="cuda")  # noqa: E731
    lg = torch.empty((1, m.vocab), dtype=torch.int32, device="cuda")
    with torch.cuda.stream(m.stream):
        m.prefill([0], dev(p[:37]), [0, 37], lg)
        m.prefill([0], dev(p[37:70]), [0, 33], lg)
        m.fork_seq(0, 2, 70)                             # one whole page shared, six tokens copied
        tok = m.prefill([0], dev(p[70:]), [0, 30], lg)
        m.stream.synchronize()
        assert np.array_equal(lg.cpu().numpy()[0], want[0])
        tok2 = m.prefill([2], dev(p[70:]), [0, 30], lg)
        m.stream.synchronize()
        assert np.array_equal(lg.cpu().numpy()[0], want[0])
        for sid, t in ((0, tok), (2, tok2)):
            m.decode_step([sid], t, lg, t)
            m.stream.synchronize()
            assert np.array_equal(lg.cpu().numpy()[0], want[1])
    m.reset_seq(0)
    toks, rows = m.generate([p], 2, seq_ids=[0])
    assert np.array_equal(rows[1][0], want[1])


def test_tiny_wide_batch(torch, tiny_artifact):
    """Twelve sequences: the layer-by-layer decode path."""
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(tiny_artifact, max_batch=12, max_ctx=128, kv_bits=4)
    prompts = [synth.prompt_ids(0, 20 + i, 3 + 5 * i, m.vocab) for i in range(12)]
    toks, rows = m.generate(prompts, 4)
    for b in (0, 4, 11):
        wt, wr = oracle_run(tiny_artifact, prompts[b], 4)
        assert toks[b].tolist() == wt and np.array_equal(rows[3][b], wr[3])
    m1 = pkg.Model(tiny_artifact, max_batch=1, max_ctx=128, kv_bits=4)
    for b in (2, 7):
        _, solo = m1.generate([prompts[b]], 4)
        assert all(np.array_equal(solo[s][0], rows[s][b]) for s in range(4))
        m1.reset_seq(0)


def test_sixteen_bit_weights(torch):
    import deterministic_integer_only_gb300 as pkg
    path = synth.ensure_artifact("tiny", 0, wide=True)
    m = pkg.Model(path, max_batch=2, max_ctx=128, kv_bits=4)
    prompts = [synth.prompt_ids(0, i, 20 + 50 * i, m.vocab) for i in range(2)]
    toks, rows = m.generate(prompts, 4)
    for b, p in enumerate(prompts):
        wt, wr = oracle_run(path, p, 4)
        assert toks[b].tolist() == wt and np.array_equal(rows[3][b], wr[3])


def test_qwen_shape(torch, qwen_artifact):
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(qwen_artifact, max_batch=2, max_ctx=512, kv_bits=4)
    prompts = [synth.prompt_ids(0, 0, 24, m.vocab), synth.prompt_ids(0, 1, 70, m.vocab)]
    toks, rows = m.generate(prompts, 4)
    wt, wr = oracle_run(qwen_artifact, prompts[0], 4, 64)
    assert toks[0].tolist() == wt
    assert all(np.array_equal(rows[s][0], wr[s]) for s in range(4))


def test_llama_shape_long_batch_equals_one_sequence(torch, llama_artifact):
    """A batch whose decode attention takes the two-launch form gives the rows
    that single sequences (one launch) give."""
    import deterministic_integer_only_gb300 as pkg
    m = pkg.Model(llama_artifact, max_batch=20, max_ctx=2400, kv_bits=4)
    prompts = [synth.prompt_ids(0, i, 2150 + i, m.vocab) for i in range(20)]
    toks, hashes = m.generate(prompts, 3, keep_logits="hash")
    m1 = pkg.Model(llama_artifact, max_batch=1, max_ctx=2400, kv_bits=4)
    for b in (0, 17):
        t1, h1 = m1.generate([prompts[b]], 3, keep_logits="hash")
        assert t1[0].tolist() == toks[b].tolist() and h1[0] == hashes[b]
        m1.reset_seq(0)
    assert not m.status().any()


def test_load_refuses_contexts_past_the_tables(torch, tiny_artifact):
    import deterministic_integer_only_gb300 as pkg
    with pytest.raises(pkg.DetintError) as e:
        pkg.Model(tiny_artifact, max_batch=1, max_ctx=4096, kv_bits=4)
    assert e.value.code == 2
    # more pages than the device has memory for is an error code, not a crash
    with pytest.raises(pkg.DetintError) as e:
        pkg.Model(tiny_artifact, max_batch=1 << 23, max_ctx=1024, kv_bits=4)
    assert e.value.code in (2, 8)
