"""Plain numpy forms of the dense calls in fp64: 8-bit storage by comparing with
every level, norms and rotations row by row.  They share no code with the library."""
from __future__ import annotations

import ctypes
import os

import numpy as np


def _levels():
    """(codes 0 .. 126, their E4M3 values): sign 0, exponents of bias 7, subnormal first."""
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return c, np.where(e > 0, (8 + m) * np.ldexp(1.0, e - 10), m * 2.0 ** -9)


CODES, LEVELS = _levels()


def _grouped(x, rows):
    T, C = x.shape
    p = np.zeros((T + -T % rows, C + -C % 128))
    p[:T, :C] = x
    return p.reshape(-1, rows, p.shape[1] // 128, 128)


def scale_bytes(x, rows):
    """The byte of each block of rows x 128: the least 2^(b - 127), b >= 1, with max|x| <= 448 * 2^(b - 127)."""
    with np.errstate(invalid="ignore"):
        amax = np.abs(_grouped(np.asarray(x, np.float64), rows)).max((1, 3))
    fine = np.isfinite(amax)
    b = np.ones(amax.shape, np.int64)
    for _ in range(256):
        b = np.where(fine & (amax > 448.0 * np.ldexp(1.0, b - 127)), b + 1, b)
    return np.where(fine, b, 255).astype(np.uint8)


def per_element(scales, rows, T, C):
    return np.repeat(np.repeat(scales, rows, 0)[:T], 128, 1)[:, :C].astype(np.int64)


def stored(x, rows):
    """(codes [T, C], scale bytes): codes to the nearest level, a tie to the even code."""
    x = np.asarray(x, np.float64)
    T, C = x.shape
    scales = scale_bytes(x, rows)
    b = per_element(scales, rows, T, C)
    y = np.abs(np.where(b == 255, 0.0, x)) / np.ldexp(1.0, b - 127)
    hi = np.clip(np.searchsorted(LEVELS, y), 0, 126)
    lo = np.clip(hi - 1, 0, 126)
    dh, dl = np.abs(LEVELS[hi] - y), np.abs(y - LEVELS[lo])
    code = np.where(dh < dl, hi, np.where(dl < dh, lo, np.where(hi % 2 == 0, hi, lo)))
    return (code + 128 * (np.signbit(x) & (b != 255))).astype(np.uint8), scales


def value(codes, scales, rows):
    """fp64 values of codes [T, C] under scale bytes."""
    c = codes.astype(np.int64)
    b = per_element(scales, rows, *codes.shape)
    v = np.where(c & 127 == 127, np.nan, LEVELS[np.minimum(c & 127, 126)])
    return np.where(b == 255, np.nan, np.where(c >= 128, -v, v) * np.ldexp(1.0, b - 127))


def norm(x, r, w, eps):
    """(s, y) of s = x + r, y = s / sqrt(mean s^2 + eps) * w, fp64."""
    s = x if r is None else x + r
    with np.errstate(all="ignore"):
        y = s / np.sqrt((s * s).mean(-1, keepdims=True) + eps)
    return s, y if w is None else y * w


TWO_PI = 2 * np.arctan2(np.longdouble(0), np.longdouble(-1))   # of the extended type


def rotate(x, pos, freqs, amplitude, interleaved, inverse):
    """x [T, H, D] fp64 turned by pos * freqs, the angle reduced in extended precision."""
    T, H, D = x.shape
    half = len(freqs)
    y = np.array(x, np.float64)
    for t in range(T):
        if pos[t] < 0:
            continue
        ang = np.remainder(np.longdouble(int(pos[t])) * freqs.astype(np.longdouble), TWO_PI).astype(np.float64)
        c, s = amplitude * np.cos(ang), amplitude * np.sin(ang) * (-1 if inverse else 1)
        i = 2 * np.arange(half) if interleaved else np.arange(half)
        j = i + 1 if interleaved else i + half
        a, b = x[t][:, i], x[t][:, j]
        y[t][:, i], y[t][:, j] = a * c - b * s, a * s + b * c
    return y


def half_step(t):
    """Half a step of bf16 or fp32 values, relative."""
    return 2.0 ** -8 if t == "bf16" else 2.0 ** -24


# ------------------------------------------------------------------ cuts of the 8-bit product
def cut_library():
    """The library, with the two entries that no header has: the cut of a product, and a product by a given cut."""
    from linear_attention_recurrence_chunk_gb300 import dense
    lib = dense._lib()
    vp, i32, i64, c = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
    lib.kda_fp8_matmul_choice.argtypes = [i64, i64, i64, c, i32, ctypes.POINTER(i32)]
    lib.kda_fp8_matmul_cut.argtypes = [vp, i64, vp, vp, i64, vp, i64, i64, i64, c, vp, i64, i32, i32, i32, vp]
    return lib


def choice(M, N, K, dt, sms=152):
    """(rows, split, deep) of a product with output type dt (0: fp32, 1: bf16); rows 0: pairs of CTAs."""
    cut = (ctypes.c_int32 * 3)()
    status = cut_library().kda_fp8_matmul_choice(M, N, K, dt, sms, cut)
    assert status == 0, status
    return tuple(cut)


def force_cut(monkeypatch, cut_of):
    """kda_fp8_matmul by the cut that cut_of(M, N, K, dt) gives (None: the library's own choice)."""
    lib = cut_library()
    plain = lib.kda_fp8_matmul

    def call(*args):
        cut = cut_of(*args[6:10])
        return plain(*args) if cut is None else lib.kda_fp8_matmul_cut(*args[:-1], *cut, args[-1])

    monkeypatch.setattr(lib, "kda_fp8_matmul", call)


def cuts_by_environment(monkeypatch):
    def cut_of(M, N, K, dt):
        pair = os.environ.get("KDA_FP8_PAIR")
        if pair is None or min(M, N, K) < 1 or K % 16:
            return None
        if pair != "0":
            return 0, 1, 1
        import torch
        cut = choice(M, N, K, dt, torch.cuda.get_device_properties(0).multi_processor_count)
        return cut if cut[0] else (256, 1, 1)

    force_cut(monkeypatch, cut_of)
