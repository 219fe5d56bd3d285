"""Attention over the 4-bit cache at the ends of its range, on the GPU: very long
sequences, whose tables name a few pages again and again, against the closed form."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunk_gb300 as kda

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
