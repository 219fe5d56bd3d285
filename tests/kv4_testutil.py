"""Plain numpy forms of the 4-bit key/value cache in fp64: the stored value of a
number, the byte layout of a cache unit, page and slot maps request by request,
and softmax attention row by row.  They share no code with the library."""
from __future__ import annotations

import numpy as np

LEVELS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def stored(x: np.ndarray):
    """(codes 0..15, scale bytes) of x [..., D]: groups of 32 channels, the scale
    2^e with the least e >= -126 that leaves no |x| above 6 * 2^e, codes to nearest,
    ties to the even code; groups that are not finite: byte 255, codes 0."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, 32)
    with np.errstate(invalid="ignore"):
        amax = np.abs(g).max(-1)
    fine = np.isfinite(amax)
    a = np.where(fine, amax, 0.0)
    e = np.full(a.shape, -126, np.int64)
    pos = a > 0
    e[pos] = np.ceil(np.log2(a[pos] / 6.0)).astype(np.int64)
    e = np.where(pos & (a > 6.0 * np.ldexp(1.0, e)), e + 1, e)            # log2 may round across a boundary
    e = np.where(pos & (a <= 6.0 * np.ldexp(1.0, e - 1)), e - 1, e)
    e = np.maximum(e, -126)
    y = np.abs(np.where(fine[..., None], g, 0.0)) / np.ldexp(1.0, e)[..., None]
    d = np.abs(y[..., None] - LEVELS)
    best = d.min(-1, keepdims=True)
    near = d == best                                                        # one level, or two at a tie
    code = np.where(near & (np.arange(8) % 2 == 0), np.arange(8), -1).max(-1)
    code = np.where(code >= 0, code, near.argmax(-1))
    code = code + 8 * (np.signbit(g) & fine[..., None])
    byte = np.where(fine, e + 127, 255)
    return code.reshape(x.shape).astype(np.uint8), byte.astype(np.uint8)


def value(code: np.ndarray, byte: np.ndarray) -> np.ndarray:
    """fp64 values of codes [..., D] under scale bytes [..., D / 32]."""
    c = code.astype(np.int64).reshape(*code.shape[:-1], -1, 32)
    b = byte.astype(np.int64)
    s = np.where(b == 255, np.nan, np.ldexp(1.0, b - 127))
    return (np.where(c >= 8, -1.0, 1.0) * LEVELS[c % 8] * s[..., None]).reshape(code.shape)


def unit_bytes(kc, kb, vc, vb) -> np.ndarray:
    """One cache unit [17 D] from codes [16, D] and scale bytes [16, D / 32], byte by byte."""
    D = kc.shape[1]
    n = D // 32
    u = np.zeros(17 * D, np.uint8)
    for r in range(16):
        for d in range(D):
            j, w = d // 32, d % 32
            at = r * (D // 2) + 4 * ((w // 8) * n + j) + (w % 8) // 2
            u[at] |= kc[r, d] << (4 * (d % 2))
            at = 8 * D + (r // 8) * 4 * D + ((w // 4) * 8 + r % 8) * 2 * n + 2 * j + (w % 4) // 2
            u[at] |= vc[r, d] << (4 * (d % 2))
        u[16 * D + r * n: 16 * D + (r + 1) * n] = kb[r]
        u[16 * D + 16 * n + r * n: 16 * D + 16 * n + (r + 1) * n] = vb[r]
    return u


def page_map(cached, new, table, free, start, ps, room):
    """Request by request: (table, cu, lens, slots, positions, next)."""
    table = np.array(table, np.int64)
    cu, slots, pos = [0], [], []
    at = start
    for i, (c, n) in enumerate(zip(cached, new)):
        c, n = max(c, 0), max(n, 0)
        have = -(-c // ps)
        for j in range(have, -(-(c + n) // ps)):
            page = free[at] if at < len(free) else -1
            at += 1
            if j < table.shape[1] and j * ps - c + cu[-1] < room:   # its first token is mapped
                table[i, j] = page
        for p in range(c, c + n):
            page = table[i, p // ps] if p // ps < table.shape[1] else -1
            slots.append(page * ps + p % ps if page >= 0 else -1)
            pos.append(p)
        cu.append(cu[-1] + n)
    fill = max(0, room - len(slots))
    return (table, np.array(cu), np.array([max(c, 0) + max(n, 0) for c, n in zip(cached, new)]),
            np.array((slots + [-1] * fill)[:room]), np.array((pos + [-1] * fill)[:room]), min(at, max(start, len(free))))


def attention(q, k, v, scale, n_new=None):
    """One sequence: q [n, Hq, D] over k, v [L, Hkv, D], all fp64; the i-th query sees
    tokens up to L - n + i.  (o [n, Hq, D], lse [n, Hq])."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    o = np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    for i in range(n):
        m = L - n + i + 1
        if m <= 0:
            continue
        for h in range(Hq):
            z = (k[:m, h // (Hq // Hkv)] @ q[i, h]) * scale
            top = z.max()
            p = np.exp(z - top)
            with np.errstate(invalid="ignore"):
                o[i, h] = p @ v[:m, h // (Hq // Hkv)] / p.sum()
            lse[i, h] = np.log(p.sum()) + top
    return o, lse


def attention_bound(q, k, v, scale, n_new, parts):
    """How far an fp32 evaluation may be from attention(): arrays (o [n, Hq, D] without
    the rounding of the output itself, lse [n, Hq]).

    A score is off by at most ds = 2^-20 sum_d |q_d k_d| |scale|: two fp16 parts of q or an
    exact q (2^-22), the products' sums and the three factors in fp32.  A weight is off by
    2 ds (its own score, and the sum's), its rounding to fp16 (2^-11, or 2^-21 in two
    parts), and e^x (2^-21); the tokens' sums in fp32 add 2^-23 per 16 tokens.  A weight
    times its value scale, relative to the row's largest weight and the largest scale
    2^E, is held in fp16 below 2^16: where that is subnormal, half a step is 2^-40 2^E,
    on each token's code of 6 at most.  2^E is below max|v| / 3, and counts as 2^-27 at
    least."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    to, tl = np.zeros((n, Hq, D)), np.zeros((n, Hq))
    for i in range(n):
        m = L - n + i + 1
        if m <= 0:
            continue
        for h in range(Hq):
            kk, vv = k[:m, h // (Hq // Hkv)], v[:m, h // (Hq // Hkv)]
            z = (kk @ q[i, h]) * scale
            w = np.exp(z - z.max())
            ds = 2.0 ** -20 * (np.abs(kk) @ np.abs(q[i, h])).max() * abs(scale)
            run = (m / 16 + 1) * 2.0 ** -23
            small = 6 * m * 2.0 ** -40 * max(np.abs(vv[np.isfinite(vv)]).max(initial=0) / 3, 2.0 ** -27)
            to[i, h] = small / w.sum() + (2 * ds + (2.0 ** -11 if parts == 1 else 2.0 ** -21) + 2.0 ** -21 + 2 * run) * (w @ np.abs(vv)) / w.sum()
            tl[i, h] = ds + 2.0 ** -21 + run + 2.0 ** -22 * abs(np.log(w.sum()) + z.max())
    return to, tl
