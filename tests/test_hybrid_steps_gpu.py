"""The example stack (examples/hybrid_decoder.py) step by step: what its attention layer
writes and reads in each step against a plain fp64 form, single tokens by themselves, and
the states that a prompt taken in uneven steps and single tokens leaves."""
import numpy as np
import pytest
import torch

import kv4_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from test_hybrid_example_gpu import _example

pytestmark = pytest.mark.gpu

TAKES = [[64, 1, 100], [3, 0, 30], [1, 1, 1], [1, 1, 1], [4, 0, 6], [1, 1, 1], [1, 1, 1], [1, 1, 1]]
LENS = [sum(t) for t in zip(*TAKES)]


def prompts(ex):
    gen = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(n, 512, device="cuda", generator=gen).bfloat16() for n in LENS]


def steps(model, xs, after=lambda take: None):
    done, got = [0] * len(LENS), [[] for _ in LENS]
    for take in TAKES:
        y = model.step(torch.cat([x[d:d + t] for x, d, t in zip(xs, done, take)]), take)
        after(take)
        for i, part in enumerate(y.split(take)):
            got[i].append(part)
        done = [d + t for d, t in zip(done, take)]
    assert done == LENS
    return [torch.cat(g) for g in got]


def f64(t):
    return t.double().cpu().numpy()


def test_attention_of_each_step(monkeypatch):
    """The keys and values of every step lie at their slots as they were rounded, whatever was written
    after them, and each token's output is the attention over its own sequence's."""
    ex = _example()
    append, attention = kda.kda_kv4_append, kda.kda_kv4_attention
    written, calls = [], []

    def record_append(k, v, slots, cache):
        written.append((k.clone(), v.clone(), slots.clone()))
        append(k, v, slots, cache)

    def record_attention(q, cache, table, lens, **kw):
        o = attention(q, cache, table, lens, **kw)
        calls.append((q.clone(), o.clone(), lens.tolist()))
        return o

    monkeypatch.setattr(kda, "kda_kv4_append", record_append)
    monkeypatch.setattr(kda, "kda_kv4_attention", record_attention)
    model = ex.HybridDecoder(3, 160, page_size=16)
    seqs = [[np.zeros((0, 2, 128)), np.zeros((0, 2, 128))] for _ in LENS]

    def after(take):
        k, v = (ref.value(*ref.stored(f64(x))) for x in written[-1][:2])
        q, o, lens = calls[-1]
        q, o, a = f64(q), f64(o), 0
        for i, n in enumerate(take):
            seqs[i] = [np.concatenate([old, new[a:a + n]]) for old, new in zip(seqs[i], (k, v))]
            assert lens[i] == len(seqs[i][0])
            if n:
                kk, vv = seqs[i]
                want, _ = ref.attention(q[a:a + n], kk, vv, 128 ** -0.5)
                to, _ = ref.attention_bound(q[a:a + n], kk, vv, 128 ** -0.5, n, 1)
                assert (np.abs(o[a:a + n] - want) <= to + 2.0 ** -8 * np.abs(want)).all(), (take, i)
            a += n

    steps(model, prompts(ex), after)
    assert len(written) == len(calls) == len(TAKES)
    cache = model.layers[3]["cache"]
    for k, v, slots in written:
        for got, x in zip(kda.kda_kv4_gather(cache, slots), (k, v)):
            assert np.array_equal(f64(got), ref.value(*ref.stored(f64(x))))
    slots = torch.cat([w[2] for w in written])
    assert slots.min() >= 0 and slots.unique().numel() == sum(LENS)
    assert kda.kda_device_error() == (0, 0)


def test_each_token_and_the_states_after_one_step_and_after_many():
    ex = _example()
    xs = prompts(ex)
    whole, parts = ex.HybridDecoder(3, 160, page_size=16), ex.HybridDecoder(3, 160, page_size=16)
    want = whole.step(torch.cat(xs), LENS).split(LENS)
    got = steps(parts, xs)
    # A layer's outputs agree to 2e-2 of their rms between the two runs (chunked against single tokens); four layers add
    # theirs, and a token by itself may be off by twice what all are on average.
    for i, (a, b) in enumerate(zip(got, want)):
        rel = (a.float() - b.float()).norm(dim=-1) / b.float().norm(dim=-1)
        assert (rel <= 2 * 4 * 2e-2).all(), (i, rel.max())
    # A state is within 1e-2 of the exact one of its inputs in either run; layer n's inputs are off by what n layers
    # before it added, and twice that counts: keys, values, gates and strengths all come from them.
    for n in range(3):
        for i in range(len(LENS)):
            a, b = (m.layers[n]["state"][i] for m in (parts, whole))
            rel = float((a - b).norm() / b.norm())
            assert rel <= 2 * 1e-2 + n * 2 * 2e-2, (n, i, rel)
    assert kda.kda_device_error() == (0, 0)
