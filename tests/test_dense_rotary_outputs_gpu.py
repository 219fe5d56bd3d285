"""Rotary positions into parts of one buffer: outputs between one another's tokens or heads, and between those of the inputs."""
import pytest
import torch

import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


def _inputs(T, Hq, Hk, D, dt):
    g = torch.Generator().manual_seed(T + D)
    q, k = (torch.randn(T, h, D, generator=g).to(dt).cuda() for h in (Hq, Hk))
    return q, k, torch.arange(T, dtype=torch.int32, device="cuda") * 991 - 1, kda.kda_rotary_freqs(D // 2)[0]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D,extra", [(64, 0), (20, 3)])
@pytest.mark.parametrize("T", [1, 2, 37, 3000])
def test_outputs_of_one_buffer(T, D, extra, dt):
    Hq, Hk = 6, 2
    q, k, pos, freqs = _inputs(T, Hq, Hk, D, dt)
    yq, yk = kda.kda_rotary(q, k, pos, freqs)
    rows = torch.full((T, (Hq + 2 * Hk) * D + extra), -5.0, device="cuda", dtype=dt)     # tokens of queries, keys and values
    oq, ok = rows[:, :Hq * D].unflatten(1, (Hq, D)), rows[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D))
    a, b = kda.kda_rotary(q, k, pos, freqs, q_out=oq, k_out=ok)
    assert a is oq and b is ok and torch.equal(oq, yq) and torch.equal(ok, yk) and (rows[:, (Hq + Hk) * D:] == -5).all()
    heads = torch.full((T, 2 * Hk, 3, D), -5.0, device="cuda", dtype=dt)                  # keys' heads beside as many queries'
    oq, ok = heads[:, :Hk, 0], heads[:, Hk:, 2]
    kda.kda_rotary(q[:, :Hk], k, pos, freqs, q_out=oq, k_out=ok)
    assert torch.equal(oq, yq[:, :Hk]) and torch.equal(ok, yk) and (heads[:, :, 1] == -5).all() and (heads[:, Hk:, 0] == -5).all()


@pytest.mark.parametrize("T", [1, 2, 37])
def test_outputs_beside_inputs(T):
    """The keys' input where it lies, between the tokens or heads of the queries' output; and an output beside its own input."""
    H, D = 4, 64
    q, k, pos, freqs = _inputs(T, H, H, D, torch.bfloat16)
    yq, yk = kda.kda_rotary(q, k, pos, freqs)
    for cut in (lambda b: (b[:, 0], b[:, 1]), lambda b: (b.view(T, H, 2, D)[:, :, 0], b.view(T, H, 2, D)[:, :, 1])):
        both = torch.zeros(T, 2, H, D, device="cuda", dtype=torch.bfloat16)
        one, two = cut(both)
        two.copy_(k)
        kda.kda_rotary(q, two, pos, freqs, q_out=one, k_out=two)             # keys in place
        assert torch.equal(one, yq) and torch.equal(two, yk)
        two.copy_(k)
        _, b = kda.kda_rotary(q, two, pos, freqs, q_out=one)                 # keys read there
        assert torch.equal(one, yq) and torch.equal(b, yk) and torch.equal(two, k)
        one.copy_(q)
        kda.kda_rotary(one, None, pos, freqs, q_out=two)                     # from one half to the other
        assert torch.equal(two, yq) and torch.equal(one, q)


@pytest.mark.parametrize("T", [1, 5])
def test_outputs_over_one_another(T):
    H, D = 4, 64
    q, k, pos, freqs = _inputs(T, H, H, D, torch.bfloat16)
    b = torch.zeros(T, 3 * H, D, device="cuda", dtype=torch.bfloat16)
    flat = torch.zeros(T * 3 * H * D, device="cuda", dtype=torch.bfloat16)
    half = flat[D // 2:D // 2 + T * 2 * H * D].view(T, 2 * H, D)
    for oq, ok in ((b[:, :H], b[:, :H]), (b[:, :H], b[:, H - 1:2 * H - 1]), (b[:, 0:2 * H:2], b[:, H:2 * H]), (b[:, :H], b[:, 1:2 * H + 1:2]),
                   (flat[:T * 2 * H * D].view(T, 2 * H, D)[:, 0::2], half[:, 0::2])):
        with pytest.raises(kda.KdaError):
            kda.kda_rotary(q, k, pos, freqs, q_out=oq, k_out=ok)
    b[:, :H] = q
    for out in (b[:, 1:H + 1], b[:, H - 1:2 * H - 1], b[:, 0:2 * H:2]):
        with pytest.raises(kda.KdaError):
            kda.kda_rotary(b[:, :H], None, pos, freqs, q_out=out)
