"""Cases of the paged 4-bit key/value cache beside the recurrence kernels.

Four operators of a hybrid decoder's full-attention layers (the layers between
the recurrent ones):

* ``page_map``: block tables and slot maps on the GPU from request lengths;
* ``append`` (with ``gather``): new keys and values into the 4-bit cache, and
  the values that it then holds, read back;
* ``attention``: softmax attention of ragged query tokens over the cache.

The cache is uint8 ``[pages, kv heads, page_size / 16, 17 D]``; the unit of 16
tokens of a head holds, in this order,

* keys, 16 rows of D / 2 bytes: the 32-bit word at place ``t * (D / 32) + j`` has
  the eight channels ``32 j + 8 t ..`` (low nibble first);
* values, two blocks of 8 tokens: ``[8 g][8 tokens][D / 32 j]`` pairs of bytes with
  the four channels ``32 j + 4 g ..``;
* the keys' and the values' scales, 16 rows of D / 32 bytes each.

A value is an E2M1 code (sign, 0 0.5 1 1.5 2 3 4 6) times 2^(byte - 127), one
byte for 32 channels: the smallest power of two, from 2^-126 on, for which none
of them is above 6; codes are rounded to nearest, ties to the even code.

``run`` takes the framework's calls where ``own`` is true and elementary torch
operations in fp32 otherwise.
"""
import math
import random

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's bookkeeping of a full batch
        {"name": "map_decode_256", "op": "page_map", "N": 256, "page": 64, "cached": 8192, "new": 1, "spread": False},
        # a prefill batch of uneven prompts, some with a cached prefix
        {"name": "map_prefill_61", "op": "page_map", "N": 61, "page": 16, "cached": 1000, "new": 4096, "spread": True},
        # very many short requests with a few tokens each (an offline batch)
        {"name": "map_many_4096", "op": "page_map", "N": 4096, "page": 32, "cached": 2048, "new": 160, "spread": True},
        # the new token of each of 256 sequences
        {"name": "append_decode_256", "op": "append", "T": 256, "Hkv": 8, "D": 128, "page": 64, "dt": "bf16", "fused": True},
        # an odd number of fp32 tokens with small heads
        {"name": "append_odd_f32", "op": "append", "T": 1003, "Hkv": 3, "D": 64, "page": 16, "dt": "f32", "fused": False},
        # the prefill of a long prompt, keys and values cut out of the fused projection
        {"name": "append_prefill_64k", "op": "append", "T": 65536, "Hkv": 8, "D": 128, "page": 64, "dt": "bf16", "fused": True},
        # a few short conversations with small fp32 heads (a test rig)
        {"name": "attn_small_f32", "op": "attention", "N": 7, "L": 301, "q": 1, "Hq": 6, "Hkv": 2, "D": 64, "page": 16, "dt": "f32", "spread": True},
        # one user with a long document: a single token over 128K cached ones
        {"name": "attn_decode_1x128k", "op": "attention", "N": 1, "L": 131072, "q": 1, "Hq": 32, "Hkv": 4, "D": 128, "page": 64, "dt": "bf16", "spread": False},
        # a decode batch of uneven lengths
        {"name": "attn_decode_48x32k", "op": "attention", "N": 48, "L": 32000, "q": 1, "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "dt": "bf16", "spread": True},
        # a wide batch of short sequences, twelve query heads on a key head
        {"name": "attn_decode_256x2k", "op": "attention", "N": 256, "L": 2048, "q": 1, "Hq": 96, "Hkv": 8, "D": 128, "page": 32, "dt": "bf16", "spread": True},
        # draft tokens verified in one pass
        {"name": "attn_verify_32x8k", "op": "attention", "N": 32, "L": 8191, "q": 5, "Hq": 32, "Hkv": 8, "D": 128, "page": 16, "dt": "bf16", "spread": True},
        # a chunk of the prompt over what is cached already, itself included
        {"name": "attn_extend_3x2k", "op": "attention", "N": 3, "L": 9000, "q": 2048, "Hq": 32, "Hkv": 8, "D": 128, "page": 64, "dt": "bf16", "spread": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["page_map", "append", "append", "attention", "attention", "attention"])
    page = rng.choice([16, 32, 64, 128])
    if op == "page_map":
        N = _log(rng, 1, 4096)
        return {"op": op, "N": N, "page": page, "cached": _log(rng, 1, 8192), "new": _log(rng, 1, max(1, min(4096, 300000 // N))),
                "spread": rng.random() < 0.7}
    Hkv, D, dt = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128]), rng.choice(["bf16", "bf16", "f32"])
    if op == "append":
        return {"op": op, "T": _log(rng, 1, 65536 if dt == "bf16" else 16384), "Hkv": Hkv, "D": D, "page": page, "dt": dt, "fused": rng.random() < 0.6}
    group = rng.choice([1, 2, 4, 6, 8, 12, 16])
    kind = rng.choice(["decode", "decode", "verify", "extend"])
    L = _log(rng, 1, 32000)
    if kind == "decode":
        q, N = 1, _log(rng, 1, max(1, min(256, 1536000 // L)))
    elif kind == "verify":
        q, N = rng.randint(2, 8), _log(rng, 1, max(1, min(64, 260000 // L)))
    else:
        q = _log(rng, 9, 2048)
        L, group, dt = max(q, min(L, 9000)), min(group, 32 // Hkv), "bf16"
        N = rng.randint(1, max(1, min(8, 17000000 // (L * q))))
    return {"op": op, "N": N, "L": L, "q": q, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "page": page, "dt": dt, "spread": rng.random() < 0.7}


# ------------------------------------------------------- lengths, the same every time for a case
def _lens(n, most, spread, rng, least=1):
    if not spread:
        return [most] * n
    got = [max(least, min(most, int(round(math.exp(rng.uniform(math.log(max(1, most // 16)), math.log(most))))))) for _ in range(n)]
    got[rng.randrange(n)] = most
    return got


def _case_lens(case):
    """Every length of a case, as lists (the same for every seed, so that the passes cost the same)."""
    rng = random.Random("%s %s" % (sorted((k, v) for k, v in case.items() if k != "name"), 1))
    if case["op"] == "page_map":
        new = _lens(case["N"], case["new"], case["spread"], rng)
        if case["spread"]:  # some requests wait this step, some are new
            new = [0 if rng.random() < 0.1 else x for x in new[:-1]] + new[-1:]
        cached = [rng.randint(0, case["cached"]) if rng.random() < 0.9 else 0 for _ in range(case["N"])]
        return cached, new
    q = [case["q"]] * case["N"]
    if case["spread"] and case["q"] > 1:
        q = [rng.randint(1, case["q"]) for _ in q]
        q[0] = case["q"]
    lens = [max(a, b) for a, b in zip(_lens(case["N"], case["L"], case["spread"], rng), q)]
    if case["spread"] and case["N"] > 4 and case["q"] == 1:
        lens[lens.index(min(lens))] = 0  # a padded place of the batch: nothing cached, a row that sees no token
    return lens, q


# ----------------------------------------------------------------- inputs
def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _random_units(n, D, gen):
    """n units of 16 tokens of a head: codes and scales of normally distributed keys and values."""
    dev = "cuda"
    codes = (torch.randn(1 << 16, 2, device=dev, generator=gen) * 2.0)
    code = torch.bucketize(codes.abs(), torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=dev)) + 8 * (codes < 0)
    table = (code[:, 0] + 16 * code[:, 1]).to(torch.uint8)
    data = table[torch.randint(0, 1 << 16, (n, 16 * D), device=dev, generator=gen)]
    scale = torch.tensor([125, 126, 126, 126, 126, 126, 127], dtype=torch.uint8, device=dev)
    scale = scale[torch.randint(0, 7, (n, D), device=dev, generator=gen)]
    return torch.cat([data, scale], 1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case, "op": case["op"], "page": case["page"]}
    if case["op"] == "page_map":
        cached, new = _case_lens(case)
        ps = case["page"]
        have = [-(-c // ps) for c in cached]
        full = [-(-(c + n) // ps) for c, n in zip(cached, new)]
        order = torch.randperm(sum(full) + 100, device="cuda", generator=gen).to(torch.int32)
        table = np.full((case["N"], max(max(full), 1)), -1, np.int64)
        at = np.arange(table.shape[1])[None, :] < np.asarray(have)[:, None]
        table[at] = np.arange(sum(have))
        t = torch.from_numpy(table).cuda()
        s["block_table"] = torch.where(t >= 0, order[t.clamp(min=0)], -1).to(torch.int32)
        s["free_pages"] = order.roll(7 - sum(have)).contiguous()  # the pages that are free, from place 7 on
        s["free_start"] = _i32([7])
        s["cached"], s["new"], s["tokens"] = _i32(cached), _i32(new), sum(new)
        return s
    D, H, ps = case["D"], case["Hkv"], case["page"]
    dt = _DT[case["dt"]]
    if case["op"] == "append":
        T = case["T"]
        pages = -(-T // ps) + 3
        s["cache"] = torch.zeros((pages, H, ps // 16, 17 * D), dtype=torch.uint8, device="cuda")
        if T <= pages * ps // 4 or T < 2048:  # tokens of many sequences, each somewhere in its page
            slots = torch.randperm(pages * ps, device="cuda", generator=gen)[:T]
            if T > 16:
                slots[T // 3] = -1  # a padded place of the batch
        else:  # a prompt: page after page
            order = torch.randperm(pages, device="cuda", generator=gen)
            i = torch.arange(T, device="cuda")
            slots = order[i // ps] * ps + i % ps
        s["slots"] = slots.to(torch.int32)
        width = (8 + 2) * H * D if case["fused"] else 2 * H * D  # the projection's row: queries, keys, values
        x = torch.randn((T, width), device="cuda", generator=gen)
        x *= torch.exp(torch.randn((width,), device="cuda", generator=gen) * 0.7)  # channels of uneven size
        x = x.to(dt)
        k, v = x[:, width - 2 * H * D:width - H * D], x[:, width - H * D:]
        s["k"], s["v"] = k.view(T, H, D), v.view(T, H, D)
        if not case["fused"]:
            s["k"], s["v"] = s["k"].contiguous(), s["v"].contiguous()
        return s
    lens, qn = _case_lens(case)
    npages = [-(-n // ps) for n in lens]
    units = _random_units(4096, D, gen)
    pages = sum(npages) + 2
    s["cache"] = units[torch.randint(0, 4096, (pages * H * (ps // 16),), device="cuda", generator=gen)].view(pages, H, ps // 16, 17 * D)
    table = np.full((case["N"], max(npages)), -1, np.int64)
    table[np.arange(table.shape[1])[None, :] < np.asarray(npages)[:, None]] = np.arange(sum(npages))
    t = torch.from_numpy(table).cuda()
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    s["block_table"] = torch.where(t >= 0, order[t.clamp(min=0)], -1).to(torch.int32)
    s["lens"] = _i32(lens)
    s["cu"] = _i32([0] + list(np.cumsum(qn)))
    s["max_q"] = max(qn)
    s["q"] = (torch.randn((sum(qn), case["Hq"], D), device="cuda", generator=gen) * 2.0).to(dt)
    s["scale"] = 1.0 / math.sqrt(D)
    return s


# ----------------------------------------------------------- plain forms
def _map_plain(s):
    ps, cached, new, old, free = s["page"], s["cached"].long(), s["new"].long(), s["block_table"], s["free_pages"]
    start, total = s["free_start"].long(), s["tokens"]
    have, full = (cached + ps - 1) // ps, (cached + new + ps - 1) // ps
    need = full - have
    first = start + torch.cumsum(need, 0) - need
    j = torch.arange(old.shape[1], device=old.device)[None, :]
    fresh = (j >= have[:, None]) & (j < full[:, None])
    at = first[:, None] + j - have[:, None]
    table = torch.where(fresh, torch.where(at < free.numel(), free[at.clamp(0, free.numel() - 1)], -1), old)
    ends = torch.cumsum(new, 0)
    i = torch.arange(total, device=old.device)
    seq = torch.searchsorted(ends, i, right=True)
    pos = cached[seq] + i - (ends - new)[seq]
    page = table[seq, pos // ps].long()
    slots = torch.where(page >= 0, page * ps + pos % ps, -1)
    cu = torch.cat([torch.zeros_like(ends[:1]), ends])
    next_ = torch.clamp(start + need.sum(), max=free.numel())
    return [x.to(torch.int32) for x in (table, cu, cached + new, slots, pos, next_)]


def _codes(x):
    """fp32 [..., D] -> (E2M1 codes [..., D], scale bytes [..., D / 32])."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 2 - (m <= 0.75).int(), -126).clamp(min=-126)
    y = torch.ldexp(b.abs(), -e[..., None])
    c = (y > 0.25).int() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)
    return (c + 8 * torch.signbit(b)).flatten(-2), e + 127


def _places(slots, H, D, ps):
    """Byte offsets in the cache of each token's and head's key and value bytes (in the order of the channels) and scales."""
    unit = (slots // ps)[:, None] * (H * (ps // 16)) + torch.arange(H, device=slots.device) * (ps // 16) + (slots % ps // 16)[:, None]
    base, r = unit[..., None] * (17 * D), (slots % 16)[:, None, None]
    n = torch.arange(D // 2, device=slots.device)
    j, t, b = n // 16, n // 4 % 4, n % 4
    key = base + r * (D // 2) + (t * (D // 32) + j) * 4 + b
    g, b = n // 2 % 8, n % 2
    val = base + 8 * D + (r // 8) * (4 * D) + (g * 8 + r % 8) * (D // 16) + j * 2 + b
    k = torch.arange(D // 32, device=slots.device)
    ks = base + 16 * D + r * (D // 32) + k
    return key, val, ks, ks + D // 2


def _values(data, scale):
    """Bytes [..., D / 2] and scale bytes [..., D / 32] -> fp32 [..., D]."""
    lut = torch.tensor(_LEVELS + tuple(-x for x in _LEVELS), device=data.device)
    both = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], -1)
    x = both.index_select(0, data.reshape(-1).int()).view(*data.shape[:-1], -1, 32)
    return (x * (scale.int() << 23).view(torch.float32)[..., None]).flatten(-2)


def _append_plain(s):
    cache, D, H, ps = s["cache"], s["case"]["D"], s["case"]["Hkv"], s["page"]
    slots = s["slots"].long()
    kept = slots >= 0
    spare = cache.shape[0] * ps  # a padded token writes to a page of its own behind the pool
    flat = torch.cat([cache.view(-1), cache.new_zeros(cache[0].numel())])
    places = _places(torch.where(kept, slots, spare), H, D, ps)
    got = []
    for x, data, scale in ((s["k"], places[0], places[2]), (s["v"], places[1], places[3])):
        c, e = _codes(x.float())
        flat[data] = (c[..., 0::2] + 16 * c[..., 1::2]).to(torch.uint8)
        flat[scale] = e.to(torch.uint8)
        got.append(torch.where(kept[:, None, None], _values(flat[data], flat[scale]), 0.0).to(x.dtype))
    cache.view(-1).copy_(flat[:cache.numel()])
    return got


def _unpack(u, D):
    """Units [..., 17 D] -> keys and values, fp32 [..., 16, D]."""
    lead, n = u.shape[:-1], D // 32
    k = u[..., :8 * D].reshape(*lead, 16, 4, n, 4).transpose(-3, -2).reshape(*lead, 16, D // 2)
    v = u[..., 8 * D:16 * D].reshape(*lead, 2, 8, 8, n, 2)
    d = len(lead)
    v = v.permute(*range(d), d, d + 2, d + 3, d + 1, d + 4).reshape(*lead, 16, D // 2)
    ks, vs = u[..., 16 * D:16 * D + D // 2].reshape(*lead, 16, n), u[..., 16 * D + D // 2:].reshape(*lead, 16, n)
    return _values(k, ks), _values(v, vs)


def _attention_plain(s):
    q, cu, lens, D, H = s["q"], s["cu"].long(), s["lens"].long(), s["case"]["D"], s["case"]["Hkv"]
    T, Hq = q.shape[:2]
    G, mq, N = Hq // H, s["max_q"], lens.numel()
    k, v = _unpack(s["cache"][s["block_table"].clamp(min=0).long()].transpose(1, 2).flatten(2, 3), D)  # [N, H, units, 16, D]
    k, v = k.flatten(2, 3), v.flatten(2, 3)
    i = torch.arange(mq, device=q.device)
    qn = cu[1:] - cu[:-1]
    x = q[(cu[:-1, None] + i).clamp(max=T - 1)].float()  # [N, mq, Hq, D]
    x = x.view(N, mq, H, G, D).permute(0, 2, 1, 3, 4).reshape(N, H, mq * G, D)
    z = torch.matmul(x, k.transpose(-1, -2)).mul_(s["scale"]).view(N, H, mq, G, -1)
    last = (lens - qn)[:, None] + i  # the last token that a query sees
    seen = torch.arange(z.shape[-1], device=q.device) <= last[..., None]
    z.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    z.sub_(top).exp_()
    tot = z.sum(-1, keepdim=True)
    o = torch.matmul(z.view(N, H, mq * G, -1), v).view(N, H, mq, G, D) / torch.where(tot > 0, tot, 1.0)
    lse = (torch.log(tot) + top)[..., 0]
    tok = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:], tok, right=True)
    off = tok - cu[seq]
    o = o.permute(0, 2, 1, 3, 4).reshape(N, mq, Hq, D)[seq, off]
    return o.to(q.dtype), lse.permute(0, 2, 1, 3).reshape(N, mq, Hq)[seq, off]


def run(s):
    if own:
        import linear_attention_recurrence_chunk_gb300 as kda
        if s["op"] == "page_map":
            cu, lens, slots, pos, next_ = kda.kda_page_map(s["cached"], s["new"], s["block_table"], s["free_pages"], s["free_start"],
                                                           s["page"], s["tokens"])
            return [s["block_table"], cu, lens, slots, pos, next_]
        if s["op"] == "append":
            kda.kda_kv4_append(s["k"], s["v"], s["slots"], s["cache"])
            return kda.kda_kv4_gather(s["cache"], s["slots"], s["k"].dtype)
        return kda.kda_kv4_attention(s["q"], s["cache"], s["block_table"], s["lens"], cu_seqlens=s["cu"], max_q_len=s["max_q"],
                                     sm_scale=s["scale"], return_lse=True)
    return {"page_map": _map_plain, "append": _append_plain, "attention": _attention_plain}[s["op"]](s)


# -------------------------------------------------------------- work and truth
def work(case):
    a, b = _case_lens(case) if case["op"] != "append" else (None, None)
    if case["op"] == "page_map":
        ps, T = case["page"], sum(b)
        fresh = sum(-(-(c + n) // ps) - -(-c // ps) for c, n in zip(a, b))
        old = sum(-(-c // ps) for c in a)  # entries that the slots of a shared page may need: one per request at most
        return {"bytes": 4 * (4 * case["N"] + 1 + 2 * T + 2 * fresh + min(old, case["N"]) + 2), "flops": 0}
    D, H = case["D"], case["Hkv"]
    eb = 2 if case["dt"] == "bf16" else 4
    token = H * (D + D // 16)  # the cache's bytes of a token
    if case["op"] == "append":  # read, write to the cache, read it back, write the values
        return {"bytes": case["T"] * (4 * H * D * eb + 2 * token + 8), "flops": 0}
    Hq, T = case["Hq"], sum(b)
    seen = sum(n * (2 * L - n + 1) // 2 for L, n in zip(a, b))
    return {"bytes": 2 * T * Hq * D * eb + 4 * T * Hq + sum(a) * token + 4 * (sum(-(-L // case["page"]) for L in a) + 2 * case["N"]),
            "flops": 4 * D * Hq * seen}


def _truth_map(s):
    cached, new, ps = s["cached"].tolist(), s["new"].tolist(), s["page"]
    table, free, at = s["block_table"].cpu().numpy().copy(), s["free_pages"].tolist(), int(s["free_start"])
    cu, slots, pos = [0], [], []
    for i, (c, n) in enumerate(zip(cached, new)):
        for j in range(-(-c // ps), -(-(c + n) // ps)):
            table[i, j] = free[at]
            at += 1
        p = np.arange(c, c + n)
        slots.append(table[i, p // ps].astype(np.int64) * ps + p % ps)
        pos.append(p)
        cu.append(cu[-1] + n)
    got = (table, cu, [c + n for c, n in zip(cached, new)], np.concatenate(slots), np.concatenate(pos), [at])
    return [torch.from_numpy(np.asarray(x, dtype=np.int32)) for x in got]


def _truth_round(x):
    """What the cache holds of x: the nearest level, between equals the one of even place, in fp64."""
    b = x.double().unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(amax > 0, amax, 1.0))) - 3  # 6 * 2^e is below amax; then the first that is not
    for _ in range(3):
        e = torch.where(amax > 6.0 * torch.exp2(e), e + 1, e)
    unit = torch.where(amax > 0, torch.exp2(e), 0.0).clamp(min=2.0 ** -126)
    y = b.abs() / unit
    low = torch.zeros_like(y)
    for p, level in enumerate(_LEVELS[1:], 1):
        mid = (level + _LEVELS[p - 1]) / 2
        low = torch.where(y >= mid if p % 2 == 0 else y > mid, level, low)
    return (torch.sign(b) * low * unit).flatten(-2)


def _truth_unit(u, D):
    """Units [n, 17 D] of one head -> keys and values, fp64 [16 n, D], by the layout's words."""
    u = u.long()
    level = torch.tensor(_LEVELS, dtype=torch.float64, device=u.device)
    d = torch.arange(D, device=u.device)
    r = torch.arange(16, device=u.device)[:, None]

    def read(byte, scale):
        code = u[:, byte] >> (4 * (d % 2)) & 15
        x = level[code % 8] * (1.0 - 2.0 * (code // 8))
        return (x * torch.exp2(u[:, scale].double() - 127)).reshape(-1, D)

    word = d % 32 // 8 * (D // 32) + d // 32
    key = read(r * (D // 2) + 4 * word + d % 8 // 2, 16 * D + r * (D // 32) + d // 32)
    place = 8 * D + r // 8 * (4 * D) + (d % 32 // 4 * 8 + r % 8) * (D // 16) + 2 * (d // 32) + d % 4 // 2
    return key, read(place, 16 * D + D // 2 + r * (D // 32) + d // 32)


def _truth_attention(s):
    D, H, ps = s["case"]["D"], s["case"]["Hkv"], s["page"]
    q, lens, cu, table = s["q"], s["lens"].tolist(), s["cu"].tolist(), s["block_table"].long()
    G = q.shape[1] // H
    o = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    for n, L in enumerate(lens):
        lo, hi = cu[n], cu[n + 1]
        pages = table[n, :-(-L // ps)]
        for h in range(H):
            k, v = _truth_unit(s["cache"][pages, h].reshape(-1, 17 * D), D)
            x = q[lo:hi, h * G:(h + 1) * G].double()
            z = torch.einsum("qgd,ld->qgl", x, k[:L]) * s["scale"]
            late = torch.arange(L, device=q.device)[None, :] > (L - (hi - lo) + torch.arange(hi - lo, device=q.device))[:, None]
            z = z.masked_fill(late[:, None], -math.inf)
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            o[lo:hi, h * G:(h + 1) * G] = torch.einsum("qgl,ld->qgd", torch.softmax(z, -1), v[:L])
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "page_map":
        return _truth_map(s)
    if case["op"] == "append":
        kept = (s["slots"] >= 0)[:, None, None]
        return [torch.where(kept, _truth_round(x), 0.0) for x in (s["k"], s["v"])]
    return _truth_attention(s)
