"""Attention over the 4-bit cache on the GPU against a plain fp64 form on the values
that the cache holds."""
import numpy as np
import pytest
import torch

import kv4_testutil as ref
import linear_attention_recurrence_chunk_gb300 as kda

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def no_error():
    assert kda.kda_device_error() == (0, 0)


def f64(t):
    return t.double().cpu().numpy()


class Setup:
    """A cache whose unused bytes are random (scale bytes of 255 among them), sequences
    of the given lengths on pages in random order, and queries."""

    def __init__(self, dt, D, Hq, Hkv, ps, lens, qn, seed=0, spread=1.0, kscale=1.0, vscale=1.0, edit=None):
        rng = np.random.default_rng(seed)
        self.dt, self.D, self.Hq, self.Hkv, self.lens, self.qn = dt, D, Hq, Hkv, list(lens), list(qn)
        pages = [-(-n // ps) for n in lens]
        total = sum(pages) + 3
        ids = rng.permutation(total)
        table = np.full((len(lens), max(max(pages), 1) + 1), -1, np.int64)
        at = 0
        for i, n in enumerate(pages):
            table[i, :n] = ids[at:at + n]
            at += n
        self.cache = torch.from_numpy(rng.integers(0, 256, (total, Hkv, ps // 16, 17 * D)).astype(np.uint8)).to(DEV)
        k = rng.standard_normal((sum(lens), Hkv, D)) * kscale
        v = rng.standard_normal((sum(lens), Hkv, D)) * vscale
        if edit is not None:
            edit(k, v, rng)
        tk, tv = torch.tensor(k).to(BF).to(DEV), torch.tensor(v).to(BF).to(DEV)
        slots = [table[i, p // ps] * ps + p % ps for i, n in enumerate(lens) for p in range(n)]
        if slots:
            kda.kda_kv4_append(tk, tv, i32(slots), self.cache)
        self.k, self.v = (ref.value(*ref.stored(f64(x))) for x in (tk, tv))
        self.table, self.dlens = i32(table), i32(lens)
        self.cu = i32([0] + list(np.cumsum(qn)))
        self.q = torch.tensor(rng.standard_normal((sum(qn), Hq, D)) * spread).to(dt).to(DEV)
        self.scale = D ** -0.5

    def run(self, **kw):
        a = dict(cu_seqlens=self.cu, max_q_len=max(self.qn), sm_scale=self.scale, return_lse=True)
        a.update(kw)
        return kda.kda_kv4_attention(a.pop("q", self.q), self.cache, self.table, self.dlens, **a)

    def check(self, o, lse, scale=None):
        scale = self.scale if scale is None else scale
        parts = 1 if self.dt is BF else 2
        step = torch.finfo(self.dt).eps / 2
        q, o, lse = f64(self.q), f64(o), f64(lse)
        a = b = 0
        worst = 0.0
        for L, n in zip(self.lens, self.qn):
            k, v, x = self.k[a:a + L], self.v[a:a + L], q[b:b + n]
            want, wl = ref.attention(x, k, v, scale)
            to, tl = ref.attention_bound(x, k, v, scale, n, parts)
            got, gl = o[b:b + n], lse[b:b + n]
            assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(gl), np.isnan(wl))
            none = np.isneginf(wl)
            assert np.array_equal(none, np.isneginf(gl))
            fine = ~np.isnan(want)
            tol = to + step * np.abs(want) + 1e-300
            err = np.where(fine, np.abs(np.where(fine, got - want, 0)) / np.where(fine, tol, 1), 0)
            worst = max(worst, err.max(initial=0))
            ok = ~none & ~np.isnan(wl)
            assert (np.abs(gl[ok] - wl[ok]) <= tl[ok]).all()
            a, b = a + L, b + n
        assert worst <= 1.0, worst
        no_error()


def run_check(*a, **kw):
    s = Setup(*a, **kw)
    s.check(*s.run())
    return s


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (6, 2), (8, 1), (12, 1), (32, 2), (40, 2)])
def test_decode(D, dt, Hq, Hkv):
    """One token per sequence: one row block, several, rows that do not fill one."""
    run_check(dt, D, Hq, Hkv, 16, [1, 15, 16, 17, 0, 63, 64, 65, 200, 129], [1] * 10)


@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 128, 4096])
def test_page_sizes(ps, kernel):
    """Pages that end inside a tile, and tiles inside a page."""
    run_check(BF, 128, 8, 2, ps, [1, 47, 333, 100], [1] * 4)
    run_check(F32, 64, 4, 2, ps, [5, 161], [1] * 2)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("D,Hq,Hkv,qn", [(128, 8, 8, [1, 2, 3]), (128, 8, 2, [5, 1, 4]), (64, 12, 2, [3, 3, 8]),
                                         (128, 32, 8, [9, 2, 33]), (64, 5, 1, [70, 1, 17])])
def test_several_query_tokens(dt, D, Hq, Hkv, qn, kernel):
    """The causal edge inside a tile and over tiles; more tokens than are cached leave rows empty."""
    run_check(dt, D, Hq, Hkv, 32, [70, 2, 150], qn)
    run_check(dt, D, Hq, Hkv, 32, qn, qn)          # a prompt from its beginning


@pytest.fixture(params=["0", "1"], ids=["line", "tiled"])
def kernel(request, monkeypatch):
    """Both kernels of bf16 calls, whichever the sizes would choose."""
    monkeypatch.setenv("KDA_KV4_TILED", request.param)
    return request.param


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,ps,lens,qn", [
    (4, 1, 64, [300], [130]),                       # rows of one and a part of a block, tiles before and on the edge
    (8, 2, 16, [128, 257, 40], [128, 129, 40]),     # from the beginning of a prompt; tile-sized lengths
    (3, 1, 48, [500, 90, 0, 7], [100, 86, 3, 20]),  # uneven row blocks, more query tokens than cached ones
    (32, 2, 32, [201], [64]),                       # a token's heads fill a fraction of a block
    (6, 6, 128, [260, 1000], [259, 1])])
def test_query_chunks(D, Hq, Hkv, ps, lens, qn, kernel):
    s = run_check(BF, D, Hq, Hkv, ps, lens, qn, spread=2.0)
    a, b = s.run(), s.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_query_chunk_with_scales_that_grow_and_not_finite_tokens(kernel):
    def grow(k, v, rng):
        v *= np.ldexp(1.0, (np.arange(v.shape[0]) // 60))[:, None, None]
        k *= np.ldexp(1.0, rng.integers(-3, 4, (k.shape[0], k.shape[1], 4)).repeat(32, -1))
        k *= (1 + np.arange(k.shape[0]) / 100)[:, None, None]
    run_check(BF, 128, 8, 2, 16, [400], [100], edit=grow)

    def holes(k, v, rng):
        k[350, 0, 3] = np.inf
        v[330, 1, 100] = np.nan
        v[20, 1, 5] = np.inf
    s = run_check(BF, 128, 8, 2, 16, [400], [100], edit=holes)
    assert torch.isnan(s.run()[0]).any() and not torch.isnan(s.run()[0]).all()


def test_chunks_that_choose_the_tiled_kernel():
    """Sizes on both sides of the rule, without a forced kernel, agree with the reference."""
    run_check(BF, 64, 32, 8, 32, [300] * 4, [80] * 4)       # 8 heads x 4 sequences x 10 blocks of 32 rows: 320
    run_check(BF, 64, 32, 8, 32, [300] * 4, [40] * 4)       # 160


def test_sequences_without_query_tokens(kernel):
    run_check(BF, 128, 8, 2, 16, [100, 50, 0, 20, 300], [1, 0, 0, 2, 0])
    run_check(BF, 128, 8, 2, 16, [100, 50, 0, 20, 300], [0, 0, 0, 0, 1])


@pytest.mark.parametrize("Hq,Hkv,lens", [(8, 1, [5000]), (16, 2, [3001, 7]), (32, 1, [2049]), (8, 8, [1500] * 3),
                                         (24, 8, [777, 1, 2500, 64] * 5)])
@pytest.mark.parametrize("dt", [BF, F32])
def test_long_segments_split_over_workers(Hq, Hkv, lens, dt):
    s = run_check(dt, 128, Hq, Hkv, 64, lens, [1] * len(lens), spread=3.0)
    a, b = s.run(), s.run()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])   # the join's order is fixed


def test_many_short_sequences():
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 40, 700).tolist()
    run_check(BF, 64, 4, 2, 16, lens, [1] * 700)


def test_no_cu_seqlens():
    s = Setup(BF, 128, 16, 4, 32, [33, 1, 90], [1, 1, 1])
    a, la = s.run()
    b = kda.kda_kv4_attention(s.q, s.cache, s.table, s.dlens)
    assert torch.equal(a, b)


def test_scale_arguments():
    s = Setup(BF, 64, 8, 2, 16, [100, 3], [1, 2])
    for scale in (-0.3, 0.0, 1e-30, 2.0):
        s.check(*s.run(sm_scale=scale), scale=scale)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("spread,kscale,vscale", [(1.0, 2.0 ** 20, 2.0 ** -60), (2.0 ** -20, 2.0 ** 20, 2.0 ** 40),
                                                  (2.0 ** 60, 2.0 ** -60, 1.0), (0.0, 1.0, 2.0 ** -20)])
def test_magnitudes(dt, spread, kscale, vscale, kernel):
    """Keys, values and queries far from 1, up to scores that pick one token."""
    run_check(dt, 128, 8, 1, 16, [300, 40], [1, 2], spread=spread, kscale=kscale, vscale=vscale)


def test_value_scales_that_grow_and_differ(kernel):
    """The weights' reference follows the largest value scale; small ones keep their precision."""
    def edit(k, v, rng):
        v *= np.ldexp(1.0, rng.integers(-9, 10, (v.shape[0], v.shape[1], 4)).repeat(32, -1))
        v *= np.ldexp(1.0, (np.arange(v.shape[0]) // 40))[:, None, None]
    run_check(BF, 128, 8, 2, 16, [400], [1], edit=edit)
    run_check(F32, 128, 8, 2, 16, [400], [1], edit=edit)


@pytest.mark.parametrize("dt", [BF, F32])
def test_not_finite_tokens_reach_only_the_rows_that_see_them(dt, kernel):
    def edit(k, v, rng):
        k[60, 0, 3] = np.inf       # seen by the last two query tokens only
        v[59, 1, 100] = np.nan     # its group of channels, for the last three
    s = Setup(dt, 128, 8, 2, 16, [62], [6], edit=edit)
    o, lse = s.run()
    s.check(o, lse)
    nan = torch.isnan(o)
    assert not nan[:3].any()
    assert nan[3:, 4:, 96:].all() and not nan[:, 4:, :96].any() and not nan[:4, :4].any() and nan[4:, :4].all()


def test_not_finite_queries(kernel):
    s = Setup(BF, 128, 8, 2, 16, [62, 9], [1, 1])
    want = s.run()[0]
    q = s.q.clone()
    q[0, 3, 5] = float("nan")
    o, lse = s.run(q=q)
    assert torch.isnan(o[0, 3]).all() and torch.isnan(lse[0, 3])
    o[0, 3] = want[0, 3]
    assert torch.equal(o, want)
    no_error()


@pytest.mark.parametrize("dt", [BF, F32])
def test_strided_queries(dt, kernel):
    s = Setup(dt, 64, 6, 2, 16, [40, 99], [2, 3])
    want = s.run()
    wide = torch.zeros((5, 3, 6, 64), dtype=dt, device=DEV)
    wide[:, 1] = s.q
    a = s.run(q=wide[:, 1])
    by_head = s.q.transpose(0, 1).contiguous().transpose(0, 1)
    b = s.run(q=by_head)
    for x in (a, b):
        assert torch.equal(x[0], want[0]) and torch.equal(x[1], want[1])


def test_other_stream_and_given_buffers():
    s = Setup(BF, 128, 8, 2, 16, [400, 9], [1, 1])
    want, lse = s.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    n = kda.kda_kv4_attention_workspace_size(2, 2, 8, 2, 128, 1, BF)
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want)
    torch.cuda.synchronize()
    a = s.run(stream=st)
    b = s.run(stream=st.cuda_stream, workspace=ws, o=out)
    st.synchronize()
    assert torch.equal(a[0], want) and torch.equal(out, want) and torch.equal(b[1], lse)
    with pytest.raises(kda.KdaError):
        s.run(workspace=ws[:-256])
    no_error()


def test_captured_into_a_graph():
    """A decode step (map, write, attention) replayed as the lengths on the device grow."""
    D, Hq, Hkv, ps, N = 128, 8, 2, 16, 3
    rng = np.random.default_rng(1)
    cache = kda.kda_kv4_cache(40, Hkv, ps, D)
    table = torch.full((N, 8), -1, dtype=torch.int32, device=DEV)
    free = i32(rng.permutation(40))
    start, lens, one = i32([0]), i32([0, 0, 0]), i32([1, 1, 1])
    k, v = torch.empty((N, Hkv, D), dtype=BF, device=DEV), torch.empty((N, Hkv, D), dtype=BF, device=DEV)
    q = torch.empty((N, Hq, D), dtype=BF, device=DEV)

    def step():
        cu, total, slots, pos, nxt = kda.kda_page_map(lens, one, table, free, start, ps, N)
        kda.kda_kv4_append(k, v, slots, cache)
        o = kda.kda_kv4_attention(q, cache, table, total)
        lens.copy_(total)
        start.copy_(nxt)
        return o

    def fill(i):
        g = torch.Generator(device=DEV).manual_seed(i)
        for x in (k, v, q):
            x.copy_(torch.randn(x.shape, device=DEV, generator=g))

    fill(0)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    lens.zero_(), start.zero_(), table.fill_(-1), cache.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    ks, vs = [], []
    for i in range(37):
        fill(i)
        ks.append(ref.value(*ref.stored(f64(k))))
        vs.append(ref.value(*ref.stored(f64(v))))
        graph.replay()
    for n in range(N):
        kk, vv = np.stack([x[n] for x in ks]), np.stack([x[n] for x in vs])
        want, _ = ref.attention(f64(q)[n:n + 1], kk, vv, D ** -0.5)
        to, _ = ref.attention_bound(f64(q)[n:n + 1], kk, vv, D ** -0.5, 1, 1)
        assert (np.abs(f64(o)[n:n + 1] - want) <= to + 2.0 ** -8 * np.abs(want)).all()
    assert lens.tolist() == [37] * 3 and start.tolist() == [9]
    no_error()


def test_far_pages(kernel):
    """A sequence whose pages lie beyond 2^32 bytes."""
    D, Hq, Hkv, ps = 128, 8, 8, 64
    pages = 1 << 16                                  # 4.6 GB
    cache = torch.zeros((pages, Hkv, ps // 16, 17 * D), dtype=torch.uint8, device=DEV)
    assert cache.numel() > 1 << 32
    k = torch.randn(100, Hkv, D, device=DEV).to(BF)
    slots = torch.cat([torch.arange(64) + (pages - 1) * ps, torch.arange(36) + (pages - 3) * ps]).int().to(DEV)
    kda.kda_kv4_append(k, -k, slots, cache)
    q = torch.randn(1, Hq, D, device=DEV).to(BF)
    o = kda.kda_kv4_attention(q, cache, i32([[pages - 1, pages - 3]]), i32([100]))
    kv = ref.value(*ref.stored(f64(k)))
    want, _ = ref.attention(f64(q), kv, -kv, D ** -0.5)
    to, _ = ref.attention_bound(f64(q), kv, -kv, D ** -0.5, 1, 1)
    assert (np.abs(f64(o) - want) <= to + 2.0 ** -8 * np.abs(want)).all()
    no_error()


@pytest.mark.parametrize("what", ["page", "page_high", "len", "len_negative", "cu_start", "cu_down", "cu_beyond", "many"])
def test_bad_device_arguments_are_reported(what, kernel):
    """The other sequences' results are those of a good call."""
    s = Setup(BF, 128, 8, 2, 16, [50, 70, 33], [1, 2, 1])
    want = s.run()[0].clone()
    keep = [0, 3]                                    # the first and the last sequence's tokens
    if what == "page":
        s.table[1, 2] = -5
    elif what == "page_high":
        s.table[1, 0] = s.cache.shape[0]
    elif what == "len":
        s.dlens[1] = 1 << 30
    elif what == "len_negative":
        s.dlens[1] = -2
    elif what == "cu_start":
        s.cu[0] = 1
        keep = [3]
    elif what == "cu_down":
        s.cu[2] = 0
        keep = [0]
    elif what == "cu_beyond":
        s.cu[3] = 9
        keep = [0, 1, 2]
    elif what == "many":
        s.cu[1:] = i32([1, 3, 4])
        o = s.run(max_q_len=1)[0]
        assert kda.kda_device_error()[0] == 1 and torch.equal(o[[0, 3]], want[[0, 3]])
        return
    o = s.run()[0]
    assert kda.kda_device_error()[0] == 1
    assert torch.equal(o[keep], want[keep])
    no_error()
