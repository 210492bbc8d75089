"""Refusals of beam selection and reordering whose arrays overlap, without a GPU:
the checks come before the first CUDA call. A group's outputs are written while
other groups' inputs are read, so none may share memory."""
import pytest

from test_beam_host import L, _select  # noqa: F401

P = 1 << 24

# arrays of 2 groups of 3 rows of 100 logits, 4 continuations each, well apart
SELECT = dict(logits=P, scores=P + 0x10000, done=P + 0x20000, end=1, parent=P + 0x30000, token=P + 0x40000, score=P + 0x50000,
              done_out=P + 0x60000, ws=P + 0x1000000, size=1 << 20)


@pytest.mark.parametrize("change", [
    dict(score=SELECT["scores"]), dict(score=SELECT["scores"] + 40), dict(score=SELECT["scores"] - 56),
    dict(done_out=SELECT["done"]), dict(done_out=SELECT["done"] + 20), dict(done_out=SELECT["done"] - 28), dict(parent=SELECT["done"]),
    dict(token=SELECT["logits"] + 4 * 599), dict(token=SELECT["parent"]), dict(token=SELECT["parent"] + 28),
    dict(done_out=SELECT["score"] + 60), dict(ws=SELECT["scores"]), dict(parent=SELECT["ws"] + 64), dict(logits=SELECT["ws"] - 2396),
    dict(stride=1000, token=SELECT["logits"] + 4 * 5099)])
def test_select_refuses_outputs_that_overlap(L, change):  # noqa: F811
    assert _select(L, **{**SELECT, **change}) == 1
    assert b"overlaps" in L.detint_last_error()


# tables of 2 groups of 3 rows of 4 columns
REORDER = dict(table=P, out=P + 0x10000, parent=P + 0x20000, lens=P + 0x30000, src=P + 0x40000, dst=P + 0x50000)


@pytest.mark.parametrize("change", [
    dict(src=REORDER["parent"]), dict(dst=REORDER["parent"] + 20), dict(dst=REORDER["src"]), dict(dst=REORDER["src"] - 20),
    dict(src=REORDER["lens"]), dict(src=REORDER["table"]), dict(dst=REORDER["out"] + 92), dict(out=REORDER["table"] + 16),
    dict(out=REORDER["table"] - 92), dict(out=REORDER["parent"]), dict(out=REORDER["lens"] - 88),
    dict(out=REORDER["table"], src=REORDER["table"] + 4), dict(out=REORDER["table"], parent=REORDER["table"] + 64)])
def test_reorder_refuses_outputs_that_overlap(L, change):  # noqa: F811
    v = {**REORDER, **change}
    assert L.detint_beam_reorder(v["table"], v["out"], 4, v["parent"], v["lens"], 2, 3, v["src"], v["dst"], None) == 1
    assert b"overlaps" in L.detint_last_error()
