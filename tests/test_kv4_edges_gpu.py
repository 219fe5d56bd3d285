"""The cache's bookkeeping and values at the edges of what fits, on the GPU."""
import numpy as np
import pytest
import torch

import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("room", [0, 1, 14, 15, 64, 99])
def test_page_map_without_room_leaves_no_stale_entries(room):
    """A page whose first token has no place in slot_map gets the entry -1, whatever the table held there
    before: the lengths count its tokens, and attention must not read another request's page."""
    ps, cached, new = 16, [3, 0, 40], [40, 49, 11]
    free = list(range(50, 70))
    table = np.full((3, 6), 777)
    table[0, 0], table[2, :3] = 20, [21, 22, 23]
    t = i32(table)
    cu, lens, slots, pos, nxt = kda.kda_page_map(i32(cached), i32(new), t, i32(free), i32([1]), ps, room)
    want, at, x0 = table.copy(), 1, 0
    for i, (c, n) in enumerate(zip(cached, new)):
        for j in range(-(-c // ps), -(-(c + n) // ps)):
            want[i, j] = free[at] if x0 + j * ps - c < room else -1
            at += 1
        x0 += n
    assert t.tolist() == want.tolist()
    assert cu.tolist() == [0, 40, 89, 100] and lens.tolist() == [43, 49, 51] and nxt.tolist() == [at]
    assert kda.kda_device_error()[0] == 1


def test_page_map_without_room_many_requests():
    """More requests than threads of a block, rows that are too short among them; what is behind a row is untouched."""
    rng = np.random.default_rng(0)
    N, ps, mp = 1500, 16, 4
    cached, new = rng.integers(0, 40, N), rng.integers(0, 60, N)
    room = int(new.sum()) // 2
    t = torch.full((N + 1, mp), 777, dtype=torch.int32, device=DEV)
    have, full = -(-cached // ps), -(-(cached + new) // ps)
    total = int((full - have).sum())
    kda.kda_page_map(i32(cached), i32(new), t[:N], i32(np.arange(1000, 1000 + total)), i32([0]), ps, room)
    want, at, x0 = np.full((N + 1, mp), 777), 1000, 0
    for i in range(N):
        for j in range(have[i], full[i]):
            if j < mp:
                want[i, j] = at if x0 + j * ps - cached[i] < room else -1
            at += 1
        x0 += new[i]
    assert np.array_equal(t.cpu().numpy(), want)
    assert kda.kda_device_error()[0] == 1


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_the_largest_values_read_back_as_infinite(dt):
    """From 3.5 * 2^126 on a value rounds to 4 * 2^126 = 2^128, which neither type holds; below, to finite ones."""
    x = torch.zeros((4, 1, 64), dtype=torch.float32, device=DEV)
    x[0, 0, 3], x[1, 0, 3], x[2, 0, 3], x[3, 0, 3] = 3.5 * 2.0 ** 126, -torch.finfo(torch.bfloat16).max, 3.484375 * 2.0 ** 126, 2.0 ** 127
    x = x.to(dt)
    cache = kda.kda_kv4_cache(1, 1, 16, 64)
    slots = i32(range(4))
    kda.kda_kv4_append(x, x, slots, cache)
    for got in kda.kda_kv4_gather(cache, slots, dt):
        got = got[:, 0, 3].double().tolist()
        assert got == [float("inf"), -float("inf"), 3.0 * 2.0 ** 126, 2.0 ** 127]
    assert kda.kda_device_error() == (0, 0)
