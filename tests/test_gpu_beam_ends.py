"""Beam search of whole models with prompts that finish at different steps."""
import numpy as np
import pytest

import synth
from test_gpu_beam_model import Fed, pkg, plain_search  # noqa: F401

pytestmark = pytest.mark.gpu


def test_a_finished_prompt_leaves_its_context_alone(pkg, tiny_artifact):  # noqa: F811
    """A prompt of 60 tokens whose one beam ends at the first step, in contexts of
    64 places, next to one of 7 tokens that goes on for 20: alone neither runs out
    of places, so together they do not."""
    long, short = (list(synth.prompt_ids(3, i, n, 1024)) for i, n in ((1, 60), (2, 7)))
    fed = Fed(tiny_artifact, 8, 96)
    end = int(plain_search(fed, long, 1, 1, -1)[0][0, 0])
    for prompts in ([long, short], [short, long], [long, short, long]):
        m = pkg.Model(tiny_artifact, max_batch=len(prompts), max_ctx=64)
        toks, scores = m.beam_search(prompts, 1, 20, end_id=end)
        for g, p in enumerate(prompts):
            want, ws = plain_search(fed, p, 1, 20, end)
            assert np.array_equal(toks[g], want) and np.array_equal(scores[g], ws)
            assert m.seq_len(g) == len(p) + ([*want[0], end].index(end) if end in want[0] else 19)
        m.close()


@pytest.mark.parametrize("kv_bits", [8, 4])
@pytest.mark.parametrize("beams,ends", [(1, [(3, 9), (2, 4), (1, 6), (5, 8)]), (2, [(5, 1), (3, 1)])])
def test_prompts_that_finish_at_different_steps(pkg, tiny_artifact, beams, ends, kv_bits):  # noqa: F811
    """Six prompts and, as end token in turn, a token that the free search of one
    of them meets: some finish, the others go on beside them."""
    fed = Fed(tiny_artifact, kv_bits, 96)
    prompts = [list(synth.prompt_ids(3, 20 + i, n, 1024)) for i, n in enumerate((60, 5, 64, 33, 1, 63))]
    met = set()
    for g, step in ends:
        end = int(plain_search(fed, prompts[g], beams, 10, -1)[0][0, step])
        m = pkg.Model(tiny_artifact, max_batch=6 * beams, max_ctx=96, kv_bits=kv_bits)
        ids = list(range(6 * beams - 1, -1, -1))
        toks, scores = m.beam_search(prompts, beams, 10, end_id=end, seq_ids=ids)
        for i, p in enumerate(prompts):
            want, ws = plain_search(fed, p, beams, 10, end)
            assert np.array_equal(toks[i], want) and np.array_equal(scores[i], ws)
            met.add(m.seq_len(ids[beams * i]) - len(p))
        assert (m.status() == 0).all()
        m.close()
    assert len(met) > 1                                  # they did not all run to the end
