"""Attention over the 4-bit cache at the ends of its range, on the GPU: very long
sequences, whose tables name a few pages again and again, against the closed form."""
import numpy as np
import pytest
import torch

import kv4_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda
from test_kv4_attention_gpu import Setup, kernel, run_check  # noqa: F401  (a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def no_error():
    assert kda.kda_device_error() == (0, 0)


def one_token_far_away(L, ps, at, D=64, dt=BF):
    """One query over L tokens that all have the key 0 and the value 1, but for the one at
    position ``at``, whose score is 72 (by 6 * 1.5 * 64 / 8) and whose value is -3.  Its page and
    the last one are pages of their own; what lies behind L in the last one is not finite.
    exp(72) = 1.8e31 leaves the others, exp(0) each, below 2^-70 of the sum."""
    cache = kda.kda_kv4_cache(3, 1, ps, D)
    k, v = torch.zeros((3 * ps, 1, D), dtype=BF, device=DEV), torch.ones((3 * ps, 1, D), dtype=BF, device=DEV)
    last = (L - 1) // ps
    k[2 * ps + (L - 1) % ps + 1:] = float("nan")
    v[2 * ps + (L - 1) % ps + 1:] = float("inf")
    page = 2 if at // ps == last else 1
    k[page * ps + at % ps], v[page * ps + at % ps] = 6.0, -3.0
    kda.kda_kv4_append(k, v, torch.arange(3 * ps, dtype=torch.int32, device=DEV), cache)
    table = torch.zeros((1, last + 1), dtype=torch.int32, device=DEV)
    table[0, at // ps] = 1
    table[0, last] = 2
    q = torch.full((1, 1, D), 1.5, dtype=dt, device=DEV)
    o, lse = kda.kda_kv4_attention(q, cache, table, i32([L]), sm_scale=0.125, return_lse=True)
    assert (o == -3.0).all(), o
    # a score is off by 2^-20 of its products' sum at most: fp32 factors and sums; the logarithm rounds four times more
    assert abs(float(lse) - 72.0) <= 72 * (2.0 ** -20 + 2.0 ** -22)
    no_error()


@pytest.mark.parametrize("ps", [16, 48])
def test_pages_beyond_two_to_the_24(ps):
    """More table entries than 24 bits count, and the token that matters behind them."""
    one_token_far_away(((1 << 24) + 9) * ps + 3, ps, ((1 << 24) + 5) * ps + 7)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 2, [3000] * 40), (16, 8, [701, 0, 4000, 65] * 7), (4, 4, [20000])])
def test_cut_segments_are_joined_alike_every_time(dt, Hq, Hkv, lens):
    """Most workers' parts end inside a segment here, so that its pieces go through the workspace: which workers
    have them depends on the lengths alone.  Between the calls others leave their own sums in shared memory."""
    ps, D = 32, 128
    gen = torch.Generator(device=DEV).manual_seed(len(lens))
    T = max(lens)
    cache = kda.kda_kv4_cache(-(-T // ps), Hkv, ps, D)
    k, v = (torch.randn(T, Hkv, D, device=DEV, generator=gen).to(BF) for _ in range(2))
    kda.kda_kv4_append(k, v, torch.arange(T, dtype=torch.int32, device=DEV), cache)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device=DEV).repeat(len(lens), 1)
    q = torch.randn(len(lens), Hq, D, device=DEV, generator=gen).to(dt)
    dl, other = i32(lens), i32([17 + 31 * i for i in range(len(lens))])
    want = kda.kda_kv4_attention(q, cache, table, dl, return_lse=True)
    for _ in range(20):
        kda.kda_kv4_attention(q, cache, table, other)
        got = kda.kda_kv4_attention(q, cache, table, dl, return_lse=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # the same rows in calls of their own, cut at other places, agree to the output's rounding
    for n in range(0, len(lens), 9):
        o, lse = kda.kda_kv4_attention(q[n:n + 1], cache, table[n:n + 1], dl[n:n + 1], return_lse=True)
        if lens[n] == 0:
            assert not o.any() and torch.isneginf(lse).all()
            continue
        # Two evaluations: each score off by ds = 2^-20 sum |q k| sm_scale (below 16 for these q, k), each weight by 2 ds and
        # its rounding (fp16, or two parts, and e^x), the output by half a step, on values of at most 6; the logarithm by ds
        # and fp32 roundings.
        ds = 2.0 ** -16
        step = 2 * ds + (2.0 ** -8 + 2.0 ** -11 if dt is BF else 2.0 ** -19)
        assert ((o - want[0][n:n + 1]).float().abs() <= 2 * step * 6).all()
        assert ((lse - want[1][n:n + 1]).abs() <= 2 * (ds + 2.0 ** -21 * lse.abs())).all()
    no_error()


@pytest.mark.parametrize("at", [0, (1 << 31) - 2])
def test_the_longest_sequence(at):
    """2^31 - 1 tokens, the one that matters the first or the last of them."""
    one_token_far_away((1 << 31) - 1, 4096, at)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_keys_far_above_and_queries_far_below_one(dt, D, kernel):
    """Finite scores (of a few tens) whose sums pass 2^128 when a row of q is scaled to 2^14."""
    s = Setup(dt, D, 8, 1, 16, [300, 40], [1, 2], spread=2.0 ** -98, kscale=2.0 ** 112)
    s.check(*s.run(sm_scale=2.0 ** -15), scale=2.0 ** -15)


@pytest.mark.parametrize("dt", [BF, F32])
def test_scale_of_zero_with_the_largest_keys(dt, kernel):
    """sm_scale = 0: every token the same weight, whatever its key."""
    s = Setup(dt, 128, 8, 2, 16, [300, 40], [1, 2], kscale=2.0 ** 122)
    s.check(*s.run(sm_scale=0.0), scale=0.0)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("spread", [1.0, 64.0])
def test_not_finite_values_of_tokens_whose_weight_is_far_below_the_largest(dt, spread, kernel):
    """A query sees them wherever they lie, also where fp32 has no weight as small (spread 64: most weights here)."""
    def edit(k, v, rng):
        for tok, head, ch in [(5, 0, 40), (63, 1, 3), (200, 0, 100), (395, 1, 70), (397, 0, 5)]:
            v[tok, head, ch] = np.inf if tok % 2 else np.nan
    run_check(dt, 128, 8, 2, 16, [400, 30], [6, 1], edit=edit, spread=spread)
    run_check(dt, 64, 4, 4, 32, [400], [3], edit=lambda k, v, rng: edit(k, np.concatenate([v, v], -1), rng), spread=spread)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("exps,grow", [((0, -15, -30, -45), 0), ((-60, 10, -20, 40), 0), ((-90, -40, 0, -65), 30), ((0, -30, 0, -30), -9)])
def test_channel_groups_of_far_apart_sizes(dt, exps, grow, kernel):
    """Each group of 32 channels has the precision of its own values, however large another group's are (grow: by
    2^grow every 60 tokens)."""
    def edit(k, v, rng):
        v *= np.ldexp(1.0, np.array(exps).repeat(32))
        v *= np.ldexp(1.0, grow * (np.arange(v.shape[0]) // 60))[:, None, None]
    s = Setup(dt, 128, 8, 2, 16, [300, 45], [3, 1], edit=edit)
    o, lse = s.run()
    s.check(o, lse)
    q, got, step = s.q.double().cpu().numpy(), o.double().cpu().numpy(), torch.finfo(dt).eps / 2
    a = b = 0
    for L, n in zip(s.lens, s.qn):
        k, v, x = s.k[a:a + L], s.v[a:a + L], q[b:b + n]
        want, _ = ref.attention(x, k, v, s.scale)
        for j in range(4):
            if np.isnan(want[..., 32 * j:32 * j + 32]).all():   # values that grew beyond the type; check() has seen them
                continue
            own = np.zeros_like(v)   # the bound counts the largest value of the group alone
            own[..., 32 * j:32 * j + 32] = v[..., 32 * j:32 * j + 32]
            unit = 2.0 ** np.floor(np.log2(np.abs(own).max()))
            to, _ = ref.attention_bound(x, k, own / unit, s.scale, n, 1 if dt is BF else 2)
            c = slice(32 * j, 32 * j + 32)
            tol = to[..., c] * unit + step * np.abs(want[..., c]) + 2.0 ** -133
            assert (np.abs(got[b:b + n][..., c] - want[..., c]) <= tol).all(), j
        a, b = a + L, b + n


@pytest.mark.parametrize("dt,Hq,Hkv,ps,lens,qn", [(BF, 8, 1, 64, [131072], [1]), (F32, 2, 1, 16, [60000], [1]),
                                                  (BF, 4, 2, 32, [30001, 17], [5, 2]), (F32, 3, 1, 64, [20000], [7])])
def test_long_sequences(dt, Hq, Hkv, ps, lens, qn):
    run_check(dt, 128, Hq, Hkv, ps, lens, qn, spread=2.0)


def test_long_sequences_of_chunks(kernel):
    run_check(BF, 128, 2, 1, 16, [20011], [35], spread=2.0)
    run_check(BF, 64, 1, 1, 64, [30000, 200], [33, 129])
