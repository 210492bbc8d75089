"""Beam search and context eviction over the 4-bit paged key/value cache, as cases that can be timed and compared.

Five operators, each of whole numbers, exact:

  select   log-probabilities of int32 Q16 logits rows, added to the beams' scores, and the best continuations of a group
  reorder  the block tables of the chosen beams: whole pages are shared, a page that still grows gets one owner, and the
           pages that have to be copied for that are
  axes     append with rotary positions of their own (one or several axes) beside the places in the cache
  weigh    the attention probabilities of query tokens, added up for each cached key of each key/value head
  evict    the keys of the largest weights (first and last ones always) moved to new pages

Where `own` is false `run` computes them with elementary torch operations; where it is true it calls the library.

A page holds 64 tokens of one key/value head, two 4-bit codes (value + 8) in a byte. Keys are token-major: byte b of
32-bit word w of a token's row holds channel 8w + b in its low and 8w + 4 + b in its high nibble. Values are stored by
groups of 16 channels as [channel % 8][key / 16][channel / 8 % 2][key / 8 % 2][key % 4], the low nibble for key / 4 % 2 = 0.
A token's 4-bit values times its scale code (1..255, one byte for each token and head) are the cached integers.
"""
import math

import numpy as np
import torch

own = False

BLK = 64               # tokens in a page
XMAX = 1785            # 7 * 255: the largest cached magnitude
L64 = torch.int64
DEAD = -(1 << 63)      # the score of a beam that is not there
MASKED = -(1 << 31)    # a logit that is no candidate


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one prompt, four beams, a Qwen3-0.6B-shaped vocabulary: a step that latency decides
        dict(name="select 1 x 4", op="select", groups=1, beams=4, vocab=151936, n_out=4, pad=0, end=True, banned=0),
        # a batch of prompts on a Llama-3.2-1B-shaped vocabulary: twice the beams out, banned tokens, padded rows,
        # some beams finished, some not there yet
        dict(name="select 24 x 5", op="select", groups=24, beams=5, vocab=128256, n_out=10, pad=64, end=True, banned=999),
        # the beams of one short prompt after a step
        dict(name="reorder 1 x 4", op="reorder", groups=1, beams=4, n_q=16, n_kv=8, d=128, lo=575, hi=575, weight=False),
        # 32 prompts of about 4096 tokens with 8 beams each, kept weights moving along
        dict(name="reorder 32 x 8", op="reorder", groups=32, beams=8, n_q=16, n_kv=8, d=128, lo=3900, hi=4200, weight=True),
        # one token of a context that lost most of its keys: its place is 1024, its position 20000
        dict(name="axes 1 token", op="axes", n_q=16, n_kv=8, d=128, seqs=1, start=1024, new=1, rot=128, inter=False,
             norm=True, axes=1, weave=False, far=20000),
        # two pictures' patches and text: time, height and width in sections of the head
        dict(name="axes 2 x 4096", op="axes", n_q=16, n_kv=8, d=128, seqs=2, start=17, new=4096, rot=128, inter=False,
             norm=True, axes=3, weave=False, far=4096),
        # one generated token of a middling context
        dict(name="weigh 1 x 4000", op="weigh", n_q=16, n_kv=8, d=128, seqs=1, lo=3999, hi=3999, new=1, window=0, fork=False),
        # a full serving batch of long, ragged contexts
        dict(name="weigh 64 x 4k-16k", op="weigh", n_q=32, n_kv=8, d=128, seqs=64, lo=4000, hi=16383, new=1, window=0,
             fork=False),
        # the last tokens of long prompts, which decide what is kept of them
        dict(name="weigh 3 x 61 of 8k", op="weigh", n_q=32, n_kv=8, d=64, seqs=3, lo=8000, hi=8100, new=61, window=0,
             fork=False),
        # every token of a 4096-token prompt
        dict(name="weigh 1 x 4096", op="weigh", n_q=16, n_kv=8, d=128, seqs=1, lo=0, hi=0, new=4096, window=0, fork=False),
        # one context back to its budget
        dict(name="evict 1 x 4097", op="evict", n_q=16, n_kv=8, d=128, seqs=1, lo=4097, hi=4097, keep=1024, sinks=4, recent=64),
        # a batch of long contexts, an odd budget
        dict(name="evict 16 x 20k", op="evict", n_q=32, n_kv=8, d=128, seqs=16, lo=9000, hi=32768, keep=4099, sinks=16,
             recent=517),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["select", "reorder", "axes", "weigh", "evict"])
    if op == "select":
        vocab = _log_int(rng, 1000, 200000)
        groups = _log_int(rng, 1, 64)
        beams = _log_int(rng, 1, max(1, min(16, 24 * 5 * 128256 // (vocab * groups))))
        return dict(op=op, groups=groups, beams=beams, vocab=vocab, n_out=beams * rng.choice([1, 2]), pad=rng.choice([0, 0, 3, 64]),
                    end=rng.random() < 0.7, banned=rng.choice([0, 0, rng.randint(1, vocab - 100)]))
    n_kv = rng.choice([1, 2, 4, 8])
    n_q = n_kv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128])
    if op == "reorder":
        groups, beams = _log_int(rng, 1, 32), _log_int(rng, 2, 8)
        lo = _log_int(rng, 1, 4096)
        return dict(op=op, groups=groups, beams=beams, n_q=n_q, n_kv=n_kv, d=d, lo=lo, hi=lo + rng.randint(0, 200),
                    weight=rng.random() < 0.5)
    if op == "axes":
        seqs = _log_int(rng, 1, 64)
        per_token = (n_q + 2 * n_kv) * d                    # at most the listed 8192 tokens of 4096 values
        new = rng.choice([1, _log_int(rng, 1, max(1, min(4096, 8192 * 4096 // (per_token * seqs))))])
        return dict(op=op, n_q=n_q, n_kv=n_kv, d=d, seqs=seqs, start=_log_int(rng, 1, 50000) - 1, new=new,
                    rot=rng.choice([d, d // 2, d // 4]), inter=rng.random() < 0.5, norm=rng.random() < 0.5,
                    axes=rng.choice([1, 2, 3, 4]), weave=rng.random() < 0.5, far=_log_int(rng, 100, 60000))
    if op == "weigh":
        seqs = _log_int(rng, 1, 64)
        if rng.random() < 0.5:                              # single tokens
            hi = _log_int(rng, 1, min(131072, 64 * 10000 * 32 * 128 // (seqs * max(n_q, 8) * d)))
            return dict(op=op, n_q=n_q, n_kv=n_kv, d=d, seqs=seqs, lo=_log_int(rng, 1, hi) - 1, hi=hi - 1, new=1,
                        window=rng.choice([0, 0, _log_int(rng, 1, 4096)]), fork=rng.random() < 0.3)
        seqs = min(seqs, 8)
        lo = _log_int(rng, 1, 8192) - 1
        hi = rng.randint(lo, 8192)
        room = 4096 * 4096 * 16 // 2 // (seqs * n_q * (hi + 1))   # new * (hi + new) within the listed 1 x 4096
        return dict(op=op, n_q=n_q, n_kv=n_kv, d=d, seqs=seqs, lo=lo, hi=hi, new=_log_int(rng, 2, max(2, min(2048, room))),
                    window=rng.choice([0, 0, _log_int(rng, 1, 2048)]), fork=rng.random() < 0.3)
    seqs = _log_int(rng, 1, 16)
    hi = _log_int(rng, 2, 32768)
    keep = _log_int(rng, 1, max(1, min(4099, hi)))
    sinks = rng.choice([0, min(4, keep), rng.randint(0, keep // 2)])
    return dict(op=op, n_q=n_q, n_kv=n_kv, d=d, seqs=seqs, lo=_log_int(rng, 1, hi), hi=hi, keep=keep, sinks=sinks,
                recent=rng.choice([0, rng.randint(0, keep - sinks)]))


def _spread(n, lo, hi):
    """Lengths spread over [lo, hi], not sorted."""
    return [lo + (hi - lo) * ((i * 37 + n // 2) % n) // max(1, n - 1) for i in range(n)]


def _keys(case):
    """(query tokens, pairs of a query token and a key, cached tokens that are read) of a weigh case."""
    w, pairs, read = case["window"], 0, 0
    for a in _spread(case["seqs"], case["lo"], case["hi"]):
        t = np.arange(a + 1, a + case["new"] + 1)
        pairs += int((np.minimum(t, w) if w else t).sum())
        read += a + case["new"] - (max(0, a + 1 - w) if w else 0)
    return case["seqs"] * case["new"], pairs, read


def work(case):
    op = case["op"]
    if op == "select":
        rows = case["groups"] * case["beams"]
        return dict(bytes=rows * (4 * case["vocab"] + 12) + case["groups"] * case["n_out"] * 20, flops=rows * case["vocab"] * 16)
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    if op == "reorder":
        # tables in and out, parents, and on average half of the pages that grow, in and out
        rows = case["groups"] * case["beams"]
        pages = -(-(case["lo"] + case["hi"]) // (2 * BLK))
        return dict(bytes=rows * (8 * pages + 4) + rows // 2 * 2 * n_kv * BLK * (d + 2 + 8 * case["weight"]), flops=0)
    if op == "axes":
        t = case["seqs"] * case["new"]
        b = t * (4 * (n_q + 2 * n_kv) * d + n_q * (d + 8) + n_kv * (d + 2) + 4 * n_kv * d + 8 + 4 * case["axes"])
        return dict(bytes=b + min(t, case["far"]) * 2 * case["rot"], flops=t * (n_q + n_kv) * d * 8)
    if op == "weigh":
        t, pairs, read = _keys(case)
        return dict(bytes=read * n_kv * (d // 2 + 1 + 8) + t * n_q * (d + 8), flops=2 * pairs * n_q * d)
    lens = _spread(case["seqs"], case["lo"], case["hi"])
    kept = sum(min(x, case["keep"]) for x in lens)
    return dict(bytes=n_kv * (8 * sum(lens) + kept * (2 * (d + 2) + 8 + 4)), flops=0)


# ----------------------------------------------------------------- inputs
def _dyadic_of(x):
    """(m, k) with m / 2^k next to x and 2^14 <= m <= 2^15."""
    k = 14 - math.floor(math.log2(x))
    return int(round(x * 2.0 ** k)), k


def _params(case, g):
    """[n_kv][8 + d]: KQM KQS VQM VQS MV KV CSTM CSTK, then the key exponents of the channels."""
    d, n_kv = case["d"], case["n_kv"]
    rows = []
    for h in range(n_kv):
        unit = 1.0 / (400.0 + 10.0 * h)                              # real value of a cached unit
        sharp = 1.6 * unit * math.log2(math.e) / math.sqrt(d) / 8.0  # 8 = 2^E, E the largest exponent
        rows.append([*_dyadic_of(1.0 / (unit * 8 * 2.0 ** 14)), *_dyadic_of(1.0 / (unit * 2.0 ** 12)),
                     *_dyadic_of(unit * 128), *_dyadic_of(sharp if case["op"] == "axes" else sharp * 8)])
    p = torch.zeros(n_kv, 8 + d, dtype=torch.int32, device="cuda")
    p[:, :8] = torch.tensor(rows, dtype=torch.int32, device="cuda")
    e = torch.randint(0, 4, (n_kv, d // 2), generator=g, device="cuda", dtype=torch.int32)
    p[:, 8:] = e.repeat_interleave(2, 1) if case.get("inter") else torch.cat([e, e], 1)
    return p


def _codes(shape, g):
    lo = torch.randn(shape, generator=g, device="cuda").mul_(2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    hi = torch.randn(shape, generator=g, device="cuda").mul_(2.6).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
    return lo | (hi << 4)


def _scales(shape, g):
    return torch.randn(shape, generator=g, device="cuda").mul_(30).add_(170).round_().clamp_(1, 255).to(torch.uint8)


def _int(shape, lo, hi, g, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _prepare_select(case, g):
    rows, v = case["groups"] * case["beams"], case["vocab"]
    # Q16 logits: most near the mean, a few dozen plausible ones above
    x = torch.randn(rows, v, generator=g, device="cuda").mul_(2.2)
    hot = _int((rows, 40), 0, v, g, L64)
    x.scatter_add_(1, hot, torch.rand(rows, 40, generator=g, device="cuda").mul_(9))
    buf = torch.zeros(rows, v + case["pad"], dtype=torch.int32, device="cuda")
    logits = buf[:, :v]
    logits.copy_((x * 65536).round().clamp(-2 ** 31 + 1, 2 ** 31 - 1))
    if case["banned"]:
        at = torch.randperm(v, generator=g, device="cuda")[:case["banned"]]
        logits[:, at] = MASKED
    scores = -(torch.rand(rows, generator=g, device="cuda").mul_(12 * 65536 * 8).to(L64))
    done = torch.zeros(rows, dtype=torch.int32, device="cuda")
    if case["beams"] > 1:
        done[torch.rand(rows, generator=g, device="cuda") < (0.1 if case["end"] else 0.0)] = 1
        scores[torch.rand(rows, generator=g, device="cuda") < 0.07] = DEAD
    shape = (case["groups"], case["beams"])
    return dict(logits=logits, scores=scores.view(shape), done=done.view(shape) if case["end"] else None,
                end_id=v * 3 // 4 if case["end"] else -1)


def _prepare_reorder(case, g):
    n_kv, d, G, W = case["n_kv"], case["d"], case["groups"], case["beams"]
    lens = _spread(G, case["lo"], case["hi"])
    whole = [x // BLK for x in lens]
    blocks = max(whole) + 2
    pages = sum(whole) + 2 * G * W
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((G * W, blocks), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(whole):         # a group's beams share what came before, and have two pages each to grow into
        table[i * W:(i + 1) * W, :n] = order[at:at + n]
        at += n
        table[i * W:(i + 1) * W, n:n + 2] = order[at:at + 2 * W].view(W, 2)
        at += 2 * W
    parent = (torch.rand(G, W, generator=g, device="cuda").square_() * W).to(torch.int32)
    parent[torch.rand(G, W, generator=g, device="cuda") < 0.02] = -1
    s = dict(lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), parent=parent, table=table, new_table=torch.empty_like(table),
             src=torch.empty(G, W, dtype=torch.int32, device="cuda"), dst=torch.empty(G, W, dtype=torch.int32, device="cuda"),
             w=_int((pages, n_kv, BLK), 0, 1 << 33, g, L64) if case["weight"] else None)
    return s, pages


def _own_pages(done, new, first, g, shared=0, extra=3):
    """(table, pages): a block table whose sequences own their pages from `first` on, in random order; the first `shared`
    pages of every sequence are those of sequence 0."""
    blocks = -(-(max(done) + new) // BLK)
    last = [-(-(x + new) // BLK) for x in done]
    pages = sum(b - a for a, b in zip(first, last)) + extra
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((len(done), blocks), -1, dtype=torch.int32, device="cuda")
    at = 0
    for i in range(len(done)):
        table[i, first[i]:last[i]] = order[at:at + last[i] - first[i]]
        at += last[i] - first[i]
    for i in range(1, len(done)):
        n = min(shared, last[i], last[0])
        table[i, :n] = table[0, :n]
    return table, pages


def _rope_tables(case, max_pos):
    i = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    p = torch.arange(max_pos, dtype=torch.float64, device="cuda")[:, None]
    a = p * (1e6 ** (-2.0 * i / case["rot"]))[None]
    return (torch.cos(a) * 16384).round().to(torch.int16), (torch.sin(a) * 16384).round().to(torch.int16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=dict(case))
    op = case["op"]
    if op == "select":
        s.update(_prepare_select(case, g))
        return s
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    if op == "reorder":
        more, pages = _prepare_reorder(case, g)
        s.update(more)
    elif op == "evict":
        lens = _spread(case["seqs"], case["lo"], case["hi"])
        n, room = len(lens), -(-case["keep"] // BLK)
        s["table"], pages = _own_pages(lens, 0, [0] * n, g, extra=n * room)
        used = s["table"][s["table"] >= 0].to(L64)
        free = torch.ones(pages, dtype=torch.bool, device="cuda")
        free[used] = False
        s["new_table"] = free.nonzero().view(-1)[:n * room].to(torch.int32).view(n, room)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["seq"] = torch.arange(n, dtype=torch.int32, device="cuda")
        # a few keys take most of the attention, many take next to none; small whole weights repeat
        w = torch.randn(pages, n_kv, BLK, generator=g, device="cuda").mul_(3.0).add_(10).exp_()
        s["w"] = torch.where(torch.rand(pages, n_kv, BLK, generator=g, device="cuda") < 0.3, w.mul(1e-4).floor(), w * 1024).to(L64)
        s["kept"] = torch.empty(n, n_kv, case["keep"], dtype=torch.int32, device="cuda")
        s["max_len"] = max(lens)
    elif op == "axes":
        new = case["new"]
        done = [case["start"] + 5 * i for i in range(case["seqs"])]
        s["table"], pages = _own_pages(done, new, [x // BLK for x in done], g)
        t = len(done) * new
        s["seq"] = torch.arange(len(done), dtype=torch.int32, device="cuda").repeat_interleave(new)
        s["pos"] = torch.cat([torch.arange(x, x + new, dtype=torch.int32, device="cuda") for x in done])
        # positions of a grid's rows and columns, or of a context whose places do not count its tokens any more
        base = torch.arange(t, dtype=torch.int32, device="cuda")
        steps = [1] + [_int((1,), 2, 97, g) for _ in range(3)]
        far = case["far"]
        rp = [(far - 1 - base % far) if a == 0 else (base // steps[a] + 13 * a) % far for a in range(case["axes"])]
        s["rope_pos"] = torch.stack(rp).to(torch.int32).contiguous()
        i = torch.arange(case["rot"] // 2, device="cuda")
        s["axis"] = (i % case["axes"] if case["weave"] else i * case["axes"] // (case["rot"] // 2)).to(torch.uint8)
        x = torch.randn(t, n_q + 2 * n_kv, d, generator=g, device="cuda")     # Q12 projections, some channels hot
        x *= torch.where(torch.rand(n_q + 2 * n_kv, d, generator=g, device="cuda") < 0.02, 6.0, 1.0)
        s["qkv"] = (x * 4096).round().to(torch.int32).reshape(t, -1)
        s["cos"], s["sin"] = _rope_tables(case, far)
        s["qg"], s["kg"] = _int((2, d), 2048, 8192, g, torch.int16).unbind(0)
        s["eps"] = 17
        s["kv"] = torch.empty(2, t, n_kv, d, dtype=torch.int16, device="cuda")
        s["q8"] = torch.empty(t, n_q, d, dtype=torch.int8, device="cuda")
        s["mq"] = torch.empty(t, n_q, dtype=torch.int32, device="cuda")
        s["kq"] = torch.empty(t, n_q, dtype=torch.int32, device="cuda")
    else:
        done, new = _spread(case["seqs"], case["lo"], case["hi"]), case["new"]
        s["table"], pages = _own_pages(done, new, [0] * len(done), g, shared=min(done) // BLK // 2 if case["fork"] else 0)
        start = torch.tensor(done, dtype=torch.int32, device="cuda")
        s["seq"] = torch.arange(len(done), dtype=torch.int32, device="cuda").repeat_interleave(new)
        s["pos"] = (start[:, None] + torch.arange(new, dtype=torch.int32, device="cuda")[None]).reshape(-1).contiguous()
        t = len(done) * new
        s["q8"] = torch.randn(t, n_q, d, generator=g, device="cuda").mul_(40).round_().clamp_(-127, 127).to(torch.int8)
        s["mq"], s["kq"] = _int((t, n_q), 1 << 14, 1 << 15, g), _int((t, n_q), 19, 22, g)
        s["w"] = torch.empty(pages, n_kv, BLK, dtype=L64, device="cuda")
        s["max_len"] = max(done) + new
    s.update(n_q=n_q, n_kv=n_kv, d=d, params=_params(case, g), k=_codes((pages, n_kv, BLK, d // 2), g),
             v=_codes((pages, n_kv, BLK, d // 2), g), ks=_scales((pages, n_kv, BLK), g), vs=_scales((pages, n_kv, BLK), g))
    return s


# ------------------------------------------------------------- plain form
def _rshr(x, s):
    """x / 2^s to the nearest integer, ties up."""
    if not isinstance(s, torch.Tensor):
        return x if s == 0 else (x + (1 << (s - 1))) >> s
    return (x + ((torch.ones_like(s) << s) >> 1)) >> s


def _bits(x):
    """Binary digits of x >= 0 (below 2^53)."""
    return torch.frexp(x.to(torch.float64))[1].to(L64)


def _octave(f):
    """2^(f / 1024) in Q15 for 0 <= f < 1024."""
    return 32768 + _rshr(f * (22787 + _rshr(f * (7419 + _rshr(2562 * f, 10)), 10)), 10)


def _exp2q(delta):
    """2^(delta / 1024) in Q15 for delta <= 0."""
    ip, p = delta >> 10, _octave(delta & 1023)
    return torch.where(ip <= -24, torch.zeros_like(p), _rshr(p, (-ip).clamp(max=23)))


def _select_plain(s):
    case = s["case"]
    G, W, v, n = case["groups"], case["beams"], case["vocab"], case["n_out"]
    l = s["logits"].to(L64)
    live = l > MASKED
    top = l.masked_fill(~live, -(1 << 40)).amax(1, keepdim=True)
    delta = _rshr((l - top).clamp_(min=-(1 << 22)) * 47274, 21)
    ip = delta >> 10
    e = _rshr(_octave(delta & 1023) << 15, (-ip).clamp(max=40))
    e.masked_fill_(~live | (ip <= -31), 0)
    total = e.sum(1).clamp(min=1)
    # log2 by repeated squaring of the mantissa in [1, 2), which its leading 32 bits hold
    b = _bits(total)
    y = torch.where(b <= 32, total << (32 - b).clamp(min=0), total >> (b - 32).clamp(min=0))
    lg = b - 31
    for _ in range(20):
        # a square of 32 bits does not fit 64 with a sign: by halves, its upper 33 bits
        hi, lo = y >> 16, y & 65535
        z = ((hi * hi) << 1) + ((2 * hi * lo + (lo * lo >> 16)) >> 15)           # y y / 2^31
        bit = z >> 32
        y = z >> bit
        lg = 2 * lg + bit
    lse = top.squeeze(1) + _rshr(lg * 726817, 24)
    score = s["scores"].reshape(-1)
    there = score >= -(1 << 62)
    cand = (score - lse)[:, None] + l
    live &= there[:, None]
    if s["done"] is not None:
        d = s["done"].reshape(-1) != 0
        live &= ~d[:, None]
        cand[:, s["end_id"]] = torch.where(d, score, cand[:, s["end_id"]])
        live[:, s["end_id"]] |= d & there
    cand, live = cand.view(G, W * v), live.view(G, W * v)
    best = cand.masked_fill(~live, -(1 << 61)).amax(1, keepdim=True)
    # equal ones: the lower beam, then the lower token
    key = ((cand - best).clamp_(min=-(1 << 40)) << 22) + (1 << 22) - 1 - torch.arange(W * v, device=cand.device)
    key.masked_fill_(~live, -(1 << 63))
    at = torch.topk(key, n, dim=1)
    have = at.values > -(1 << 63)
    at = at.indices
    tok = at % v
    out = torch.where(have, cand.gather(1, at), torch.full_like(at, DEAD))
    row = torch.div(at, v, rounding_mode="floor")
    end = have & (tok == s["end_id"])
    if s["done"] is not None:
        end |= have & (s["done"].gather(1, row) != 0)
    none = torch.full_like(tok, -1)
    return [torch.where(have, row, none).to(torch.int32), torch.where(have, tok, none).to(torch.int32), out, end.to(torch.int32)]


def _reorder_plain(s):
    G, W = s["parent"].shape
    old = s["table"].view(G, W, -1)
    blocks = old.shape[2]
    i = torch.arange(W, device="cuda")
    p = s["parent"].to(L64)
    ok = (p >= 0) & (p < W)
    p = torch.where(ok, p, i)
    full = (s["lens"] // BLK).to(L64)
    past = torch.arange(blocks, device="cuda")[None] < full[:, None]
    new = torch.where(past[:, None], old.gather(1, p[..., None].expand(-1, -1, blocks)), old)
    same = (p[:, :, None] == p[:, None, :]) & ok[:, :, None] & ok[:, None, :]
    first = ok & ~same.tril(-1).any(2)                      # takes its parent's growing page over
    claimed = ((p[:, :, None] == i) & ok[:, :, None]).any(1)
    at = full.clamp(max=blocks - 1)[:, None, None].expand(-1, W, 1)
    tail = old.gather(2, at).squeeze(2)
    spare = tail.gather(1, torch.sort(claimed.to(torch.int32), dim=1, stable=True).indices)
    mine = torch.where(first, tail.gather(1, p), spare.gather(1, ((~first).cumsum(1) - 1).clamp(min=0)))
    grows = ((s["lens"] % BLK != 0) & (full < blocks))[:, None]
    new.scatter_(2, at, torch.where(grows, mine, new.gather(2, at).squeeze(2))[..., None])
    s["new_table"].copy_(new.view_as(s["new_table"]))
    moved = grows & ok & ~first
    none = torch.full_like(mine, -1)
    s["src"].copy_(torch.where(moved, tail.gather(1, p), none))
    s["dst"].copy_(torch.where(moved, mine, none))
    src, dst = s["src"][moved].to(L64), s["dst"][moved].to(L64)
    for x in ("k", "v", "ks", "vs", "w"):
        if s[x] is not None:
            s[x][dst] = s[x][src]
    return [s["new_table"], s["src"], s["dst"], s["k"], s["v"], s["ks"], s["vs"], s["w"]]


def _norm(x, gamma, eps):
    """Integer RMS norm of the last axis (a power of two wide), Q14 out."""
    d = x.shape[-1]
    a = x.abs().amax(-1, keepdim=True)
    sig = _bits(a) - 24
    m = torch.where(sig >= 0, x.abs() >> sig.clamp(min=0), x.abs() << (-sig).clamp(min=0)) * x.sign()
    e = torch.where(sig >= 0, torch.full_like(sig, eps) >> (2 * sig).clamp(0, 62),
                    torch.full_like(sig, eps) << (-2 * sig).clamp(0, 48))
    ms = ((m * m).sum(-1, keepdim=True) >> (d.bit_length() - 1)) + e
    r = ms.to(torch.float64).sqrt().to(L64)
    r = r - (r * r > ms).to(L64)
    r = (r + ((r + 1) * (r + 1) <= ms).to(L64)).clamp(min=1)
    b = _bits(r)
    y = _rshr(m * gamma.to(L64) * torch.div(torch.ones_like(r) << (b + 23), r, rounding_mode="floor"), b + 21)
    return torch.where(a == 0, torch.zeros_like(y), y)


def _rotate(y, c, s, rot, inter):
    """The first rot channels in pairs (2i, 2i + 1) or (i, i + rot / 2); the others pass."""
    if inter:
        x0, x1 = y[..., 0:rot:2], y[..., 1:rot:2]
    else:
        x0, x1 = y[..., :rot // 2], y[..., rot // 2:rot]
    z0, z1 = _rshr(x0 * c - x1 * s, 14), _rshr(x1 * c + x0 * s, 14)
    z = torch.stack([z0, z1], -1).flatten(-2) if inter else torch.cat([z0, z1], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _quant4(x):
    """4-bit values and the scale code of each row of |x| <= 1785."""
    c = ((x.abs().amax(-1, keepdim=True) + 6) // 7).clamp(min=1)
    b = _bits(c)
    return _rshr(x * torch.div(torch.ones_like(c) << (b + 16), c, rounding_mode="floor"), b + 16), c


def _put_values(vpages, page, off, w):
    """Codes w [t][n_kv][d / 16][8][2] of t tokens into their places of the value pages."""
    vp = vpages.view(vpages.shape[0], vpages.shape[1], -1, 8, 4, 2, 2, 4)
    high = (off >> 2 & 1).bool()
    lo, hi = (~high).nonzero().squeeze(1), high.nonzero().squeeze(1)
    at_lo = (page[lo], slice(None), slice(None), slice(None), off[lo] >> 4, slice(None), off[lo] >> 3 & 1, off[lo] & 3)
    at_hi = (page[hi], slice(None), slice(None), slice(None), off[hi] >> 4, slice(None), off[hi] >> 3 & 1, off[hi] & 3)
    vp[at_lo] = (vp[at_lo] & 0xF0) | w[lo]
    vp[at_hi] = (vp[at_hi] & 0x0F) | (w[hi] << 4)


def _axes_plain(s):
    n_q, n_kv, d, case = s["n_q"], s["n_kv"], s["d"], s["case"]
    x = s["qkv"].view(-1, n_q + 2 * n_kv, d).to(L64)
    q, k, v = x[:, :n_q], x[:, n_q:n_q + n_kv], x[:, n_q + n_kv:]
    q, k = (_norm(q, s["qg"], s["eps"]), _norm(k, s["kg"], s["eps"])) if case["norm"] else (q * 4, k * 4)
    at = s["pos"].to(L64)
    pair = torch.arange(case["rot"] // 2, device="cuda")
    row = s["rope_pos"].to(L64)[s["axis"].to(L64)].t()                       # [tokens][pairs]
    c, sn = s["cos"][row, pair].to(L64)[:, None], s["sin"][row, pair].to(L64)[:, None]
    q, k = _rotate(q, c, sn, case["rot"], case["inter"]), _rotate(k, c, sn, case["rot"], case["inter"])
    p = s["params"].to(L64)
    e = p[:, 8:]
    q = q << (e.amax(1, keepdim=True) - e).repeat_interleave(n_q // n_kv, 0)
    a = q.abs().amax(-1, keepdim=True)
    b = _bits(a)
    zero = a == 0
    a1 = a.clamp(min=1)
    q8 = _rshr(q * torch.div(127 << (b + 16), a1, rounding_mode="floor"), b + 16)
    kk = 21 - b
    kk = kk + ((a1 << (kk + 20)) < (127 << 34)).to(L64)
    m = torch.div(((2 * a1) << (kk + 20)) + (127 << 20), 254 << 20, rounding_mode="floor")
    s["q8"].copy_(torch.where(zero, torch.zeros_like(q8), q8))
    s["mq"].copy_(torch.where(zero, torch.zeros_like(m), m).squeeze(-1))
    s["kq"].copy_(torch.where(zero, torch.zeros_like(kk), kk + 14).squeeze(-1))
    xk = _rshr((k << e) * p[:, 0:1], p[:, 1:2].expand(n_kv, d)).clamp(-XMAX, XMAX)
    xv = _rshr(v * p[:, 2:3], p[:, 3:4].expand(n_kv, d)).clamp(-XMAX, XMAX)
    k4, ck = _quant4(xk)
    v4, cv = _quant4(xv)
    page, off = s["table"].to(L64)[s["seq"].to(L64), at // BLK], at % BLK
    t = at.numel()
    w = (k4 + 8).to(torch.uint8).view(t, n_kv, d // 8, 2, 4)
    s["k"][page, :, off] = (w[..., 0, :] | (w[..., 1, :] << 4)).reshape(t, n_kv, d // 2)
    s["ks"][page, :, off] = ck.squeeze(-1).to(torch.uint8)
    s["vs"][page, :, off] = cv.squeeze(-1).to(torch.uint8)
    _put_values(s["v"], page, off, (v4 + 8).to(torch.uint8).view(t, n_kv, d // 16, 2, 8).transpose(3, 4))
    s["kv"][0].copy_(k4 * ck)
    s["kv"][1].copy_(v4 * cv)
    return [s["q8"], s["mq"], s["kq"], s["kv"], s["k"], s["v"], s["ks"], s["vs"]]


def _weigh_plain(s):
    n_q, n_kv, d, new = s["n_q"], s["n_kv"], s["d"], s["case"]["new"]
    n, grp = s["table"].shape[0], s["n_q"] // s["n_kv"]
    page = s["table"].clamp(min=0).to(L64)
    lk = page.shape[1] * BLK
    kb = s["k"][page].view(n, -1, n_kv, BLK, d // 8, 4)                     # [n][blocks][heads][64][words][bytes]
    k4 = torch.stack([kb & 15, kb >> 4], -2).to(torch.float32).view(n, -1, n_kv, BLK, d) - 8
    k4 = k4.permute(0, 2, 4, 1, 3).reshape(n * n_kv, d, lk)
    ck = s["ks"][page].transpose(1, 2).reshape(n, n_kv, 1, 1, lk).to(L64)
    q = s["q8"].view(n, new, n_kv, grp, d).permute(0, 2, 1, 3, 4).reshape(n * n_kv, new * grp, d).to(torch.float32)
    # |S| <= 127 * 7 * d < 2^24: exact in 32 bits
    t = torch.bmm(q, k4).view(n, n_kv, new, grp, lk).to(L64) * ck
    del k4
    pos = s["pos"].view(n, 1, new, 1, 1).to(L64)
    j = torch.arange(lk, device="cuda")
    keep = j <= pos
    if s["case"]["window"]:
        keep = keep & (j > pos - s["case"]["window"])
    t.masked_fill_(~keep, -(1 << 40))
    t -= t.amax(-1, keepdim=True)
    t.clamp_(min=-(1 << 28))                      # past every kept one: |t| < 2^27
    p = s["params"].to(L64).view(1, n_kv, 1, 1, 8 + d)
    mq = s["mq"].view(n, new, n_kv, grp, 1).transpose(1, 2).to(L64)
    sh = (s["kq"].view(n, new, n_kv, grp, 1).transpose(1, 2) + p[..., 7:8] - 10).clamp(0, 62)
    e = _exp2q(_rshr(t * (mq * p[..., 6:7]), sh)).clamp_(max=32767)
    e.masked_fill_(~keep, 0)
    del t, keep
    total = e.sum(-1, keepdim=True)
    b = _bits(total)
    r = torch.div(torch.ones_like(b) << (b + 23), total, rounding_mode="floor")
    w = _rshr(e * r, b - 1).sum((2, 3)).view(n, n_kv, -1, BLK).transpose(1, 2).reshape(-1, n_kv, BLK)
    s["w"].zero_()
    s["w"].index_add_(0, page.reshape(-1), w)
    return s["w"]


def _evict_plain(s):
    case, n_kv, d = s["case"], s["n_kv"], s["d"]
    n, keep = s["lens"].numel(), case["keep"]
    src = s["table"][s["seq"].to(L64)].clamp(min=0).to(L64)
    lk = src.shape[1] * BLK
    lens = s["lens"].to(L64).view(n, 1, 1)
    j = torch.arange(lk, device="cuda")
    w = s["w"][src].transpose(1, 2).reshape(n, n_kv, lk)
    always = (j < case["sinks"]) | (j >= lens - case["recent"])
    w = torch.where(always, torch.full_like(w, (1 << 62)), w)
    w.masked_fill_((j >= lens).expand_as(w), -(1 << 62))
    m = min(keep, lk)
    at = torch.sort(w, dim=-1, descending=True, stable=True).indices[..., :m]        # equal weights: the lower place
    there = torch.arange(m, device="cuda") < lens
    at = torch.where(there, at, torch.full_like(at, lk)).sort(-1).values             # ascending, the missing ones last
    s["kept"].fill_(-1)
    s["kept"][..., :m] = torch.where(there, at, torch.full_like(at, -1))
    i, g, slot = there.expand(n, n_kv, m).nonzero(as_tuple=True)
    j = at[i, g, slot]
    old, to = src[i, j // BLK], s["new_table"].to(L64)[i, slot // BLK]
    j, slot = j % BLK, slot % BLK
    s["k"][to, g, slot] = s["k"][old, g, j]
    s["ks"][to, g, slot] = s["ks"][old, g, j]
    s["vs"][to, g, slot] = s["vs"][old, g, j]
    s["w"][to, g, slot] = s["w"][old, g, j]
    vp = s["v"].view(-1, 1, d // 16, 8, 4, 2, 2, 4)
    old, to = old * n_kv + g, to * n_kv + g
    zero = torch.zeros_like(g)
    codes = vp[old, zero, :, :, j >> 4, :, j >> 3 & 1, j & 3]
    codes = torch.where((j >> 2 & 1).bool().view(-1, 1, 1, 1), codes >> 4, codes & 15)
    _put_values(s["v"].view(-1, 1, BLK, d // 2), to, slot, codes.unsqueeze(1))
    return [s["kept"], s["k"], s["v"], s["ks"], s["vs"], s["w"]]


_PLAIN = dict(select=_select_plain, reorder=_reorder_plain, axes=_axes_plain, weigh=_weigh_plain, evict=_evict_plain)


# --------------------------------------------------------------- one pass
def _handles(s):
    """The library's views of the cache and the tables and its workspaces, kept with the state as a program keeps them."""
    if "handles" not in s:
        import deterministic_integer_only_gb300 as detint
        case = s["case"]
        if case["op"] == "select":
            need = detint.detint_beam_workspace(case["groups"] * case["beams"], case["vocab"], case["n_out"])
            s["handles"] = (detint, None, torch.empty(need, dtype=torch.uint8, device="cuda"))
            return s["handles"]
        cache = detint.KV4Cache(s["k"], s["v"], s["ks"], s["vs"], s["table"], s["params"], s["n_q"])
        rope = None
        if case["op"] == "axes":
            rope = detint.RopeNorm(s["cos"], s["sin"], interleaved=case["inter"], eps=s["eps"] if case["norm"] else 0,
                                   q_gamma=s["qg"] if case["norm"] else None, k_gamma=s["kg"] if case["norm"] else None)
        s["handles"] = (detint, cache, rope)
    return s["handles"]


def run(state):
    s, case = state, state["case"]
    if not own:
        return _PLAIN[case["op"]](s)
    detint, cache, more = _handles(s)
    if case["op"] == "select":
        return list(detint.detint_beam_select(s["logits"], s["scores"], case["n_out"], done=s["done"], end_id=s["end_id"],
                                              workspace=more))
    if case["op"] == "reorder":
        detint.detint_beam_reorder(s["table"], s["parent"], s["lens"], out=s["new_table"], src=s["src"], dst=s["dst"])
        detint.detint_kv4_copy(cache, s["src"], s["dst"], weight=s["w"])
        return [s["new_table"], s["src"], s["dst"], s["k"], s["v"], s["ks"], s["vs"], s["w"]]
    if case["op"] == "axes":
        detint.detint_kv4_append_axes(cache, more, s["qkv"], s["seq"], s["pos"], s["rope_pos"], s["axis"], q8=s["q8"], mq=s["mq"],
                                      kq=s["kq"], k_val=s["kv"][0], v_val=s["kv"][1])
        return [s["q8"], s["mq"], s["kq"], s["kv"], s["k"], s["v"], s["ks"], s["vs"]]
    if case["op"] == "weigh":
        s["w"].zero_()
        weigh = detint.detint_kv4_weigh if case["new"] == 1 else detint.detint_kv4_weigh_block
        return weigh(cache, s["q8"], s["mq"], s["kq"], s["seq"], s["pos"], s["max_len"], s["w"], window=case["window"])
    detint.detint_kv4_evict(cache, s["w"], s["seq"], s["lens"], s["max_len"], case["keep"], s["new_table"], sinks=case["sinks"],
                            recent=case["recent"], kept=s["kept"])
    return [s["kept"], s["k"], s["v"], s["ks"], s["vs"], s["w"]]


# ------------------------------------------------- the definition, in 64 bits
def _near(x, s):
    """x / 2^s rounded to the nearest, ties up (numpy int64 or Python integers)."""
    return x if s == 0 else (x + (1 << (s - 1))) >> s


def _octave_of(f):
    inner = 7419 + _near(2562 * f, 10)
    return _near(32768 + _near(f * (22787 + _near(f * inner, 10)), 10), 0)


def _exact_row_exp(delta):
    out = np.zeros_like(delta)
    for octave in range(24):
        m = delta >> 10 == -octave
        out[m] = _near(_octave_of(delta[m] & 1023), octave)
    return np.minimum(out, 32767)


def _exact_select(s):
    case = s["case"]
    logits, scores = s["logits"].cpu().numpy().astype(np.int64), s["scores"].cpu().numpy()
    done = s["done"].cpu().numpy() if s["done"] is not None else np.zeros_like(scores, np.int32)
    W, n, end = case["beams"], case["n_out"], s["end_id"]
    out = [np.full((case["groups"], n), x, t) for x, t in ((-1, np.int32), (-1, np.int32), (DEAD, np.int64), (0, np.int32))]
    for g in range(case["groups"]):
        found = []
        for b in range(W):
            score, row = int(scores[g, b]), logits[g * W + b]
            if score < -(1 << 62):
                continue
            if done[g, b]:
                found.append((-score, b, end, 1))
                continue
            ids = np.flatnonzero(row != MASKED)
            if not len(ids):
                continue
            x, m = row[ids], int(row[ids].max())
            delta = _near((x - m) * 47274, 21)
            total = 0
            for octave in range(31):
                total += int(_near(_octave_of(delta[delta >> 10 == -octave] & 1023) * 32768, octave).sum())
            # log2(total / 2^30) to 20 bits below the point, cut: the square of the mantissa tells the next bit
            bits = total.bit_length()
            y = total << (32 - bits) if bits <= 32 else total >> (bits - 32)
            lg = bits - 31
            for _ in range(20):
                z = y * y
                lg, y = (2 * lg + 1, z >> 32) if z >> 63 else (2 * lg, z >> 31)
            lse = m + _near(lg * 726817, 24)
            for at in np.lexsort((ids, -x))[:n]:
                found.append((-(score - lse + int(x[at])), b, int(ids[at]), int(ids[at] == end)))
        for i, (score, b, tok, e) in enumerate(sorted(found)[:n]):
            out[0][g, i], out[1][g, i], out[2][g, i], out[3][g, i] = b, tok, -score, e
    return out


def _exact_reorder(s):
    c = {x: s[x].cpu().numpy() for x in ("parent", "lens", "table", "k", "v", "ks", "vs")}
    w = s["w"].cpu().numpy() if s["w"] is not None else None
    G, W = c["parent"].shape
    new = c["table"].copy()
    src, dst = np.full((G, W), -1, np.int32), np.full((G, W), -1, np.int32)
    for g in range(G):
        old, full, grows = c["table"][g * W:(g + 1) * W], c["lens"][g] // BLK, c["lens"][g] % BLK
        taken = set()
        spare = [old[q][full] for q in range(W) if q not in set(c["parent"][g].tolist())] if grows else []
        for b in range(W):
            p = int(c["parent"][g, b])
            if 0 <= p < W:
                new[g * W + b, :full] = old[p, :full]
            if not grows:
                continue
            if 0 <= p < W and p not in taken:
                taken.add(p)
                new[g * W + b, full] = old[p][full]
                continue
            page = spare.pop(0)
            new[g * W + b, full] = page
            if 0 <= p < W:
                src[g, b], dst[g, b] = old[p][full], page
    pools = [c["k"], c["v"], c["ks"], c["vs"]] + ([w] if w is not None else [])
    for a, b in zip(src.reshape(-1), dst.reshape(-1)):
        if a >= 0:
            for x in pools:
                x[b] = x[a]
    return [new, src, dst, c["k"], c["v"], c["ks"], c["vs"], w]


def _k_place(ch):
    """(byte of a token's row, high nibble) of a key channel."""
    return ch // 8 * 4 + ch % 4, ch // 4 % 2


def _v_place(ch, j):
    """(byte of a page, high nibble) of a value channel of place j."""
    return ch // 16 * 512 + ch % 8 * 64 + j // 16 * 16 + ch // 8 % 2 * 8 + j // 8 % 2 * 4 + j % 4, j // 4 % 2


def _exact_axes(s):
    n_q, n_kv, d, case = s["n_q"], s["n_kv"], s["d"], s["case"]
    rot, inter = case["rot"], case["inter"]
    c = {x: s[x].cpu().numpy() for x in ("qkv", "pos", "seq", "table", "params", "cos", "sin", "qg", "kg", "k", "v", "ks", "vs",
                                         "rope_pos", "axis")}
    k, v, ks, vs, p = c["k"], c["v"].reshape(c["v"].shape[0], n_kv, -1), c["ks"], c["vs"], c["params"]
    t = len(c["pos"])
    q8, mq, kq = np.zeros((t, n_q, d), np.int8), np.zeros((t, n_q), np.int32), np.zeros((t, n_q), np.int32)
    kv = np.zeros((2, t, n_kv, d), np.int16)

    def head(x, gamma, token):
        x = [int(z) for z in x]
        if not case["norm"]:
            y = [4 * z for z in x]
        else:
            sig = max(map(abs, x)).bit_length() - 24
            m = [(abs(z) >> sig if sig >= 0 else abs(z) << -sig) * (1 if z >= 0 else -1) for z in x]
            eps = s["eps"] >> 2 * sig if sig >= 0 else s["eps"] << -2 * sig
            r = math.isqrt((sum(z * z for z in m) >> (d.bit_length() - 1)) + eps)
            b = r.bit_length()
            y = [_near(z * int(u) * ((1 << (b + 23)) // r), b + 21) for z, u in zip(m, gamma)] if any(x) else x
        for i in range(rot // 2):
            a, z = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
            at = c["rope_pos"][c["axis"][i], token]
            co, si = int(c["cos"][at, i]), int(c["sin"][at, i])
            y[a], y[z] = _near(y[a] * co - y[z] * si, 14), _near(y[z] * co + y[a] * si, 14)
        return y

    def four(x):
        code = max(1, -(-max(map(abs, x)) // 7))
        b = code.bit_length()
        return [_near(z * ((1 << (b + 16)) // code), b + 16) for z in x], code

    for i in range(t):
        at = int(c["pos"][i])
        page, off = c["table"][c["seq"][i], at // BLK], at % BLK
        row = c["qkv"][i].reshape(-1, d)
        for h in range(n_q):
            e = [int(z) for z in p[h // (n_q // n_kv), 8:]]
            y = [z << (max(e) - u) for z, u in zip(head(row[h], c["qg"], i), e)]
            a = max(map(abs, y))
            if a:
                b = a.bit_length()
                q8[i, h] = [_near(z * ((127 << (b + 16)) // a), b + 16) for z in y]
                kk = next(z for z in range(40, -40, -1) if (a << (z + 40)) < (127 << 55))
                mq[i, h], kq[i, h] = ((2 * a << (kk + 40)) + (127 << 40)) // (254 << 40), kk + 14
        for g in range(n_kv):
            e = [int(z) for z in p[g, 8:]]
            y = [z << u for z, u in zip(head(row[n_q + g], c["kg"], i), e)]
            xs = [[max(-XMAX, min(XMAX, _near(z * int(p[g, 0]), int(p[g, 1])))) for z in y],
                  [max(-XMAX, min(XMAX, _near(int(z) * int(p[g, 2]), int(p[g, 3])))) for z in row[n_q + n_kv + g]]]
            for which, x in enumerate(xs):
                x4, code = four(x)
                kv[which, i, g] = [z * code for z in x4]
                (vs if which else ks)[page, g, off] = code
                to = v[page, g] if which else k[page, g, off]
                for ch, z in enumerate(x4):
                    a, hi = _v_place(ch, off) if which else _k_place(ch)
                    to[a] = (to[a] & (0x0F if hi else 0xF0)) | (z + 8) << 4 * hi
    return [q8, mq, kq, kv, k, v.reshape(k.shape), ks, vs]


def _exact_weigh(s):
    n_q, n_kv, d, window = s["n_q"], s["n_kv"], s["d"], s["case"]["window"]
    k = s["k"].cpu().numpy()
    k4 = np.empty(k.shape[:3] + (d,), np.int8)
    for ch in range(d):
        byte, hi = _k_place(ch)
        k4[..., ch] = (k[..., byte] >> 4 if hi else k[..., byte] & 15).astype(np.int8) - 8
    ks, table, p, q8, mq, kq = (s[x].cpu().numpy().astype(np.int64) for x in ("ks", "table", "params", "q8", "mq", "kq"))
    seq, pos = s["seq"].cpu().numpy(), s["pos"].cpu().numpy()
    w = np.zeros(ks.shape, np.int64)
    for i in range(len(pos)):
        j = np.arange(max(0, pos[i] + 1 - window) if window else 0, pos[i] + 1)
        page, off = table[seq[i], j // BLK], j % BLK
        for g in range(n_kv):
            # (products of at most 127 * 7 * 128: exact)
            dots = (k4[page, g, off].astype(np.float32) @ q8[i, g * n_q // n_kv:(g + 1) * n_q // n_kv].T.astype(np.float32)).astype(np.int64)
            for x in range(n_q // n_kv):
                h = g * (n_q // n_kv) + x
                t = dots[:, x] * ks[page, g, off]
                sh = min(62, max(0, int(kq[i, h] + p[g, 7] - 10)))
                e = _exact_row_exp(np.maximum(_near((t - t.max()) * int(mq[i, h] * p[g, 6]), sh), -30 * 1024))
                total = int(e.sum())
                b = total.bit_length()
                w[page, g, off] += _near(e * ((1 << (b + 23)) // total), b - 1)
    return w


def _exact_evict(s):
    case, n_kv, d = s["case"], s["n_kv"], s["d"]
    c = {x: s[x].cpu().numpy() for x in ("k", "v", "ks", "vs", "w", "table", "new_table", "lens", "seq")}
    v = c["v"].reshape(c["v"].shape[0], n_kv, -1)
    ch = np.arange(d)
    kept = np.full((len(c["lens"]), n_kv, case["keep"]), -1, np.int32)
    for i, n in enumerate(c["lens"]):
        n = int(n)
        row, to = c["table"][c["seq"][i]], c["new_table"][i]
        j = np.arange(n)
        for g in range(n_kv):
            w = c["w"][row[j // BLK], g, j % BLK]
            if n <= case["keep"]:
                at = j
            else:
                last = n - case["recent"]
                mid = j[case["sinks"]:last]
                best = mid[np.lexsort((mid, -w[case["sinks"]:last]))][:case["keep"] - case["sinks"] - case["recent"]]
                at = np.sort(np.concatenate([j[:case["sinks"]], best, j[last:]]))
            kept[i, g, :len(at)] = at
            a, b = row[at // BLK], to[np.arange(len(at)) // BLK]
            x, y = at % BLK, np.arange(len(at)) % BLK
            for pool in (c["k"], c["ks"], c["vs"], c["w"]):
                pool[b, g, y] = pool[a, g, x]
            for z in range(len(at)):
                byte, hi = _v_place(ch, int(x[z]))
                code = v[a[z], g][byte] >> 4 if hi else v[a[z], g][byte] & 15
                byte, hi = _v_place(ch, int(y[z]))
                v[b[z], g, byte] = (v[b[z], g, byte] & (0x0F if hi else 0xF0)) | code << 4 * hi
    return [kept, c["k"], v.reshape(c["v"].shape), c["ks"], c["vs"], c["w"]]


def exact(case, seed):
    op = case["op"]
    if op == "axes" and case["seqs"] * case["new"] * (case["n_q"] + 2 * case["n_kv"]) * case["d"] > 1_000_000:
        return None
    if op == "weigh":
        t, pairs, read = _keys(case)
        if pairs * case["n_q"] > 12_000_000 or t * case["n_q"] > 20_000 or read * case["n_kv"] > 3_000_000:
            return None
    if op == "evict" and case["seqs"] * min(case["keep"], case["hi"]) * case["n_kv"] > 600_000:
        return None
    return {"select": _exact_select, "reorder": _exact_reorder, "axes": _exact_axes, "weigh": _exact_weigh,
            "evict": _exact_evict}[op](prepare(case, seed))
