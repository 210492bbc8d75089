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
