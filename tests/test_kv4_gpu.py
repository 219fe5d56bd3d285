"""Page maps, and the 4-bit cache's write and read-back, on the GPU against plain
forms in fp64.  Both are exact: integers, and a rounding whose result is defined
for every input."""
import numpy as np
import pytest
import torch

import kv4_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def no_error():
    assert kda.kda_device_error() == (0, 0)


# ------------------------------------------------------------------ page map
def run_map(cached, new, ps, free, start, max_pages, room, fill=-1):
    rng = np.random.default_rng(len(cached) + ps)
    table = np.full((len(cached), max_pages), fill, np.int64)
    have = [min(-(-max(c, 0) // ps), max_pages) for c in cached]
    ids = rng.permutation(10000 + sum(have))
    at = 0
    for i, n in enumerate(have):
        table[i, :n] = ids[at:at + n]
        at += n
    t = i32(table)
    cu, lens, slots, pos, nxt = kda.kda_page_map(i32(cached), i32(new), t, i32(free), i32([start]), ps, room)
    got = [x.cpu().numpy() for x in (t, cu, lens, slots, pos, nxt)]
    want = ref.page_map(cached, new, table, free, start, ps, room)
    for name, a, b in zip(("table", "cu", "lens", "slots", "pos"), got, want):
        assert np.array_equal(a, b), name
    assert got[5].tolist() == [want[5]]


@pytest.mark.parametrize("N,ps,most_cached,most_new", [(1, 16, 0, 1), (1, 64, 63, 1), (1, 64, 64, 1), (2, 16, 5, 700),
                                                       (7, 32, 100, 90), (255, 64, 4000, 1), (513, 128, 300, 9),
                                                       (1025, 16, 40, 40), (28672, 16, 20, 3)])
def test_page_map(N, ps, most_cached, most_new):
    rng = np.random.default_rng(N * ps)
    cached = rng.integers(0, most_cached + 1, N).tolist()
    new = rng.integers(0, most_new + 1, N).tolist()
    total = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(cached, new))
    free = rng.permutation(total + 5).tolist()
    most = max(-(-(c + n) // ps) for c, n in zip(cached, new))
    run_map(cached, new, ps, free, 3, most + 1, sum(new) + N % 7)
    no_error()


def test_page_map_nothing_new_and_no_request():
    run_map([0, 5, 16], [0, 0, 0], 16, [1, 2], 0, 2, 0)
    run_map([0, 5, 16], [0, 0, 0], 16, [1, 2], 0, 2, 3)
    cu, lens, slots, pos, nxt = kda.kda_page_map(i32([]), i32([]), torch.zeros((0, 4), dtype=torch.int32, device=DEV),
                                                 i32([1]), i32([1]), 16, 5)
    assert cu.tolist() == [0] and lens.numel() == 0 and slots.tolist() == [-1] * 5 and pos.tolist() == [-1] * 5
    assert nxt.tolist() == [1]
    no_error()


def test_page_map_same_inputs_same_outputs():
    """The entries that a call wrote do not change what the same call writes again."""
    cached, new = [10, 0, 33], [40, 17, 1]
    t = i32([[7, -1, -1, -1], [-1] * 4, [8, 9, 10, -1]])
    a = [x.clone() for x in kda.kda_page_map(i32(cached), i32(new), t, i32(range(20, 40)), i32([2]), 16, 58)]
    t1 = t.clone()
    b = kda.kda_page_map(i32(cached), i32(new), t, i32(range(20, 40)), i32([2]), 16, 58)
    assert torch.equal(t, t1) and all(torch.equal(x, y) for x, y in zip(a, b))
    no_error()


@pytest.mark.parametrize("cached,new,free,start,max_pages,room", [
    ([0, 0, 0], [40, 40, 40], 5, 0, 4, 120),        # 9 pages wanted, 5 free
    ([0, 30], [100, 5], 20, 0, 3, 105),             # the row is too short
    ([0, 0], [50, 50], 20, 0, 8, 64),               # more new tokens than room
    ([-3, 4], [5, -2], 20, 0, 4, 10),               # negative lengths count as 0
    ([0], [20], 4, 4, 4, 20),                       # nothing free
])
def test_page_map_reports_what_does_not_fit(cached, new, free, start, max_pages, room):
    run_map(cached, new, 16, list(range(50, 50 + free)), start, max_pages, room)
    assert kda.kda_device_error()[0] == 1
    no_error()


def test_page_map_partly_filled_page_without_entry():
    t = i32([[-1, -1]])
    _, _, slots, pos, _ = kda.kda_page_map(i32([5]), i32([13]), t, i32([3, 4]), i32([0]), 16, 13)
    assert slots.tolist() == [-1] * 11 + [48, 49] and pos.tolist() == list(range(5, 18)) and t.tolist() == [[-1, 3]]
    assert kda.kda_device_error()[0] == 1


# ------------------------------------------------------------ write and read
def make(T, H, D, dt, seed, wild=False):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H, D)) * np.exp(rng.standard_normal((H, D)))
    if wild:   # every exponent, ties, zeros and groups that are not finite
        x = rng.integers(-24, 25, (T, H, D)) / 4.0
        x *= np.ldexp(1.0, rng.integers(-140, 125, (T, H, D // 32))).repeat(32, -1)
        x[rng.random(x.shape) < 0.1] = 0.0
        x[rng.random(x.shape) < 0.002] = np.inf
        x[rng.random(x.shape) < 0.002] = np.nan
        x[0] = 0.0
    return torch.tensor(x).to(dt).to(DEV)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H,ps,wild", [(1, 1, 16, False), (5, 3, 16, True), (33, 2, 64, True), (200, 5, 48, True),
                                         (129, 8, 4096, False)])
def test_append_and_gather(D, dt, T, H, ps, wild):
    pages = -(-T // ps) + 2
    rng = np.random.default_rng(T + D)
    slots = rng.permutation(pages * ps)[:T]
    if T > 4:
        slots[T // 2] = -1
    k, v = make(T, H, D, dt, 1, wild), make(T, H, D, dt, 2, wild)
    cache = kda.kda_kv4_cache(pages, H, ps, D)
    kda.kda_kv4_append(k, v, i32(slots), cache)
    want = np.zeros((pages, H, ps // 16, 17 * D), np.uint8)
    codes = [ref.stored(f64(x)) for x in (k, v)]
    zero = np.zeros((16, D), np.uint8)
    for u in {(s // ps, s % ps // 16) for s in slots if s >= 0}:
        for h in range(H):
            kc, vc = zero.copy(), zero.copy()
            kb, vb = np.zeros((16, D // 32), np.uint8), np.zeros((16, D // 32), np.uint8)
            for i, s in enumerate(slots):
                if s >= 0 and (s // ps, s % ps // 16) == u:
                    r = s % 16
                    kc[r], kb[r], vc[r], vb[r] = codes[0][0][i, h], codes[0][1][i, h], codes[1][0][i, h], codes[1][1][i, h]
            want[u[0], h, u[1]] = ref.unit_bytes(kc, kb, vc, vb)
    assert np.array_equal(cache.cpu().numpy(), want)
    gk, gv = kda.kda_kv4_gather(cache, i32(slots), dt)
    for got, (c, b) in zip((gk, gv), codes):
        val = ref.value(c, b)
        val[slots < 0] = 0.0
        # the values are exact in either type down to its smallest subnormal
        assert np.array_equal(f64(got), f64(torch.tensor(val).to(dt)), equal_nan=True)
    no_error()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_append_of_strided_parts(dt):
    """Keys and values cut out of a fused projection, and heads that are not next to each other."""
    T, H, D, ps = 70, 4, 128, 32
    x = make(T, 3 * H, D, dt, 5)
    slots = i32(np.random.default_rng(0).permutation(128)[:T])
    for k, v in [(x[:, H:2 * H], x[:, 2 * H:]), (x[:, 0::3], x[:, 1::3]), (x[0].expand(T, -1, -1)[:, :H], x[:, :1].expand(-1, H, -1))]:
        a, b = kda.kda_kv4_cache(4, H, ps, D), kda.kda_kv4_cache(4, H, ps, D)
        kda.kda_kv4_append(k, v, slots, a)
        kda.kda_kv4_append(k.contiguous(), v.contiguous(), slots, b)
        assert torch.equal(a, b)
    odd = torch.zeros(T * H * D + 8, dtype=dt, device=DEV)[1:1 + T * H * D].view(T, H, D)
    with pytest.raises(kda.KdaError):
        kda.kda_kv4_append(odd, x[:, :H], slots, a)   # not on a 16-byte boundary
    no_error()


def test_slots_beyond_the_cache_are_reported():
    T, H, D = 6, 2, 64
    k = make(T, H, D, torch.bfloat16, 1)
    cache = kda.kda_kv4_cache(2, H, 16, D)
    kda.kda_kv4_append(k, k, i32([0, 32, 5, 2 ** 31 - 1, -7, 31]), cache)
    assert kda.kda_device_error()[0] == 1
    gk, _ = kda.kda_kv4_gather(cache, i32([0, 5, 31, 1]), torch.bfloat16)
    no_error()
    c, b = ref.stored(f64(k))
    want = ref.value(c, b)[[0, 2, 5, 0]]
    want[3] = 0
    assert np.array_equal(f64(gk), want)
    gk, gv = kda.kda_kv4_gather(cache, i32([32, 0]), torch.float32)
    assert kda.kda_device_error()[0] == 1 and not gk[0].any() and not gv[0].any() and gk[1].any()


def test_far_cache_offsets():
    """Pages whose bytes lie beyond 2^32."""
    H, D, ps = 8, 128, 4096
    pages = 1100                                    # 4.9 GB
    cache = torch.empty((pages, H, ps // 16, 17 * D), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 32
    k = make(3, H, D, torch.bfloat16, 3)
    slots = i32([pages * ps - 1, 5, (pages - 1) * ps])
    kda.kda_kv4_append(k, -k, slots, cache)
    gk, gv = kda.kda_kv4_gather(cache, slots, torch.bfloat16)
    c, b = ref.stored(f64(k))
    assert np.array_equal(f64(gk), ref.value(c, b)) and np.array_equal(f64(gv), -ref.value(c, b))
    no_error()


def test_other_stream():
    """Work on a stream that is not the current one is ordered on that stream."""
    T, H, D = 512, 8, 128
    k = make(T, H, D, torch.bfloat16, 1)
    cache = kda.kda_kv4_cache(32, H, 16, D)
    slots = i32(np.arange(T))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    kda.kda_kv4_append(k, k, slots, cache, stream=s)
    a, _ = kda.kda_kv4_gather(cache, slots, stream=s)
    b, _ = kda.kda_kv4_gather(cache, slots, stream=s.cuda_stream)
    s.synchronize()
    c, sb = ref.stored(f64(k))
    assert np.array_equal(f64(a), ref.value(c, sb)) and torch.equal(a, b)
    no_error()
