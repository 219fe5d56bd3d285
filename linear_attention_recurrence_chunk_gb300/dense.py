"""What a hybrid decoder's layers need around the recurrence and the cached attention.

Thin ctypes binding of ``include/kda_dense.h``, with the C names (the 8-bit format, the
rounding and the errors are stated there):

* ``kda_add_rmsnorm(x, residual, weight, eps)`` -> ``(y, h)`` and
  ``kda_add_rmsnorm_fp8(...)`` -> ``(codes, scales, h)``: the residual's addition and a
  root-mean-square norm, in the input's type or in 8 bits;
* ``kda_fp8_quant(x, block_rows)`` -> ``(codes, scales)``: a matrix in 8 bits, and
  ``kda_fp8_values(codes, scales, block_rows, dtype)``: the values read back;
* ``kda_fp8_matmul(a, a_scales, w, w_scales, dtype)`` -> ``a w^T``: the product of 8-bit
  activations and weights;
* ``kda_rotary(q, k, positions, freqs, ...)`` -> ``(q, k)``: rotary positions, and
  ``kda_rotary_freqs(...)``: the frequencies that it takes.

8-bit matrices are ``torch.float8_e4m3fn`` codes and ``uint8`` scale bytes (2^(byte - 127)).
Tensors are CUDA tensors of one device; a ``stream`` (default: the current one) is a
``torch.cuda.Stream`` or a raw handle, and what a function allocates itself belongs to
that stream.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from .kv4 import _current_raw_stream, _run

__all__ = ["kda_add_rmsnorm", "kda_add_rmsnorm_fp8", "kda_fp8_quant", "kda_fp8_values", "kda_fp8_matmul", "kda_rotary",
           "kda_rotary_freqs"]

_E4M3, _U8 = torch.float8_e4m3fn, torch.uint8
_DT = {torch.float32: 0, torch.bfloat16: 1}
_empty = torch.empty
# The bare query: a call of these functions is mostly host time, and the tensors are CUDA tensors already.
_current_device = getattr(torch._C, "_cuda_getDevice", None)

_fns = None


def _lib():
    global _fns
    if _fns is None:
        from . import load_library
        lib = load_library()
        vp, i32, i64, f32, c = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_int
        for f, args in ((lib.kda_fp8_quant, [vp, i64, i64, i64, i32, c, vp, vp, vp]),
                        (lib.kda_fp8_values, [vp, vp, i64, i64, i32, c, vp, vp]),
                        (lib.kda_add_rmsnorm, [vp, i64, vp, i64, vp, f32, i64, i64, c, vp, vp, vp, vp, vp]),
                        (lib.kda_fp8_matmul, [vp, i64, vp, vp, i64, vp, i64, i64, i64, c, vp, i64, vp]),
                        (lib.kda_rotary, [vp, i64, i64, i32, vp, i64, i64, i32, vp, i64, i32, i32, vp, f32, i32, c, vp, i64,
                                          i64, vp, i64, i64, vp])):
            f.argtypes = args
            f.restype = c
        _fns = lib
    return _fns


def _fail(status: int, where: str):
    from . import KdaError
    raise KdaError(status, where)


def _device(name: str, t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    return dev


def _dtype(dt: torch.dtype) -> int:
    code = _DT.get(dt)
    if code is None:
        raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")
    return code


def _matrix(name: str, t: torch.Tensor, dev: int) -> Tuple[int, int, int]:
    """(rows, columns, row stride) of [rows, columns] with contiguous columns."""
    if t.dim() != 2 or t.get_device() != dev:
        raise ValueError(f"{name}: a matrix on cuda:{dev} expected, got {tuple(t.shape)} on {t.device}")
    T, C = t.shape
    s, c = t.stride()
    if c != 1 and C > 1:
        raise ValueError(f"{name}: contiguous columns expected")
    return T, C, s if T > 1 else C   # a stride over one row has no meaning


def _stored(name: str, codes: torch.Tensor, scales: torch.Tensor, block_rows: int, dev: int) -> Tuple[int, int, int, int]:
    """(rows, columns, row stride, pointer of the scales) of a matrix in 8 bits."""
    if scales.dtype is not _U8:
        raise TypeError(f"scales of {name}: uint8 expected, got {scales.dtype}")
    if codes.dim() != 2 or codes.get_device() != dev or scales.get_device() != dev or not scales.is_contiguous():
        raise ValueError(f"{name}: a matrix of codes and contiguous scales on cuda:{dev} expected, got {tuple(codes.shape)} on {codes.device}, "
                         f"{tuple(scales.shape)} on {scales.device}")
    T, C = codes.shape
    s, c = codes.stride()
    if c != 1 and C > 1:
        raise ValueError(f"{name}: contiguous columns expected")
    if scales.shape != (T if block_rows == 1 else (T + 127) // 128, (C + 127) // 128):
        raise ValueError(f"{name}: a scale for each {block_rows} x 128 values of {tuple(codes.shape)} expected, got {tuple(scales.shape)}")
    return T, C, s if T > 1 else C, scales.data_ptr()


def _block_rows(n: int):
    if n != 1 and n != 128:
        raise ValueError(f"block_rows: 1 or 128 expected, got {n}")


def kda_fp8_quant(x: torch.Tensor, block_rows: int = 1, stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """x ``[T, C]`` (any row stride) in 8 bits: codes ``[T, C]`` and a scale byte for each
    block of ``block_rows`` (1: activations, 128: weights) x 128 values."""
    dev = _device("x", x)
    if stream is not None or dev != _current_device():
        return _run(dev, stream, lambda _: kda_fp8_quant(x, block_rows))
    T, C, xs = _matrix("x", x, dev)
    dt = _dtype(x.dtype)
    _block_rows(block_rows)
    codes = _empty((T, C), dtype=_E4M3, device=x.device)
    scales = _empty((T if block_rows == 1 else (T + 127) // 128, (C + 127) // 128), dtype=_U8, device=x.device)
    st = (_fns or _lib()).kda_fp8_quant(x.data_ptr(), xs, T, C, block_rows, dt, codes.data_ptr(), scales.data_ptr(), _current_raw_stream(dev))
    if st:
        _fail(st, "kda_fp8_quant")
    return codes, scales


def kda_fp8_values(codes: torch.Tensor, scales: torch.Tensor, block_rows: int = 1, dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> torch.Tensor:
    """The values ``[T, C]`` of ``dtype`` that codes ``[T, C]`` (contiguous) and their scale
    bytes stand for."""
    if codes.dtype is not _E4M3:
        raise TypeError(f"codes: {_E4M3} expected, got {codes.dtype}")
    dev = _device("codes", codes)
    if stream is not None or dev != _current_device():
        return _run(dev, stream, lambda _: kda_fp8_values(codes, scales, block_rows, dtype))
    _block_rows(block_rows)
    T, C, _, sp = _stored("codes", codes, scales, block_rows, dev)
    if not codes.is_contiguous():
        raise ValueError("codes: a contiguous matrix is expected")
    dt = _dtype(dtype)
    y = _empty((T, C), dtype=dtype, device=codes.device)
    st = (_fns or _lib()).kda_fp8_values(codes.data_ptr(), sp, T, C, block_rows, dt, y.data_ptr(), _current_raw_stream(dev))
    if st:
        _fail(st, "kda_fp8_values")
    return y


def _norm(x, residual, weight, eps, h, fp8, stream):
    dev = _device("x", x)
    if stream is not None or dev != _current_device():
        return _run(dev, stream, lambda _: _norm(x, residual, weight, eps, h, fp8, None))
    T, C, xs = _matrix("x", x, dev)
    dtype = x.dtype
    dt, rp, rs, wp, hp, device = _dtype(dtype), None, 0, None, None, x.device
    if residual is not None:
        if residual.dtype is not dtype or residual.shape != x.shape or residual.get_device() != dev:
            raise ValueError(f"residual: {dtype} {tuple(x.shape)} on cuda:{dev} expected, got {residual.dtype} {tuple(residual.shape)} on {residual.device}")
        rs, c = residual.stride()
        if c != 1 and C > 1:
            raise ValueError("residual: contiguous columns expected")
        rp = residual.data_ptr()
    if weight is not None:
        if weight.dtype is not torch.float32:
            raise TypeError(f"weight: torch.float32 expected, got {weight.dtype}")
        if weight.shape != (C,) or weight.get_device() != dev or not weight.is_contiguous():
            raise ValueError(f"weight: a contiguous [{C}] tensor on cuda:{dev} expected, got {tuple(weight.shape)} on {weight.device}")
        wp = weight.data_ptr()
    if h is not None:
        if residual is None or h.dtype is not dtype or h.shape != x.shape or not h.is_contiguous() or h.get_device() != dev:
            raise ValueError("residual_out: a contiguous tensor of the residual's type, shape and device is expected")
        hp = h.data_ptr()
    elif residual is not None:
        h = _empty((T, C), dtype=dtype, device=device)
        hp = h.data_ptr()
    if fp8:
        y, scales = _empty((T, C), dtype=_E4M3, device=device), _empty((T, (C + 127) // 128), dtype=_U8, device=device)
        st = (_fns or _lib()).kda_add_rmsnorm(x.data_ptr(), xs, rp, rs, wp, eps, T, C, dt, hp, None, y.data_ptr(), scales.data_ptr(),
                                    _current_raw_stream(dev))
    else:
        y, scales = _empty((T, C), dtype=dtype, device=device), None
        st = (_fns or _lib()).kda_add_rmsnorm(x.data_ptr(), xs, rp, rs, wp, eps, T, C, dt, hp, y.data_ptr(), None, None, _current_raw_stream(dev))
    if st:
        _fail(st, "kda_add_rmsnorm")
    return (y, scales, h) if fp8 else (y, h)


def kda_add_rmsnorm(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                    eps: float = 1e-6, residual_out: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``(y, h)``: h = x + residual (None without a residual) and y the root-mean-square norm
    of each row of the sum, times weight.  x, residual ``[T, C]`` of one type (any row
    stride), weight fp32 ``[C]``; ``residual_out`` may be the residual itself."""
    return _norm(x, residual, weight, eps, residual_out, False, stream)


def kda_add_rmsnorm_fp8(x: torch.Tensor, residual: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                        eps: float = 1e-6, residual_out: Optional[torch.Tensor] = None,
                        stream=None) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """``(codes, scales, h)``: ``kda_add_rmsnorm`` with y in 8 bits, as ``kda_fp8_matmul`` takes it."""
    return _norm(x, residual, weight, eps, residual_out, True, stream)


def kda_fp8_matmul(a: torch.Tensor, a_scales: torch.Tensor, w: torch.Tensor, w_scales: torch.Tensor,
                   dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``a w^T``, ``[M, N]`` of ``dtype``: a ``[M, K]`` with scales ``[M, ceil(K / 128)]`` and w ``[N, K]``
    with scales ``[ceil(N / 128), ceil(K / 128)]``.  K and the row strides are multiples of 16;
    ``out`` (whose type counts then) may have any row stride."""
    if a.dtype is not _E4M3 or w.dtype is not _E4M3:
        raise TypeError(f"a and w: {_E4M3} expected, got {a.dtype} and {w.dtype}")
    dev = _device("a", a)
    if stream is not None or dev != _current_device():
        return _run(dev, stream, lambda _: kda_fp8_matmul(a, a_scales, w, w_scales, dtype, out))
    M, K, lda, sa = _stored("a", a, a_scales, 1, dev)
    N, KW, ldw, sw = _stored("w", w, w_scales, 128, dev)
    if KW != K:
        raise ValueError(f"w: [N, {K}] expected, got {tuple(w.shape)}")
    if out is None:
        dt, ldo = _dtype(dtype), N
        out = _empty((M, N), dtype=dtype, device=a.device)
    else:
        if out.shape != (M, N):
            raise ValueError(f"out: [{M}, {N}] expected, got {tuple(out.shape)}")
        dt, ldo = _dtype(out.dtype), _matrix("out", out, dev)[2]
    st = (_fns or _lib()).kda_fp8_matmul(a.data_ptr(), lda, sa, w.data_ptr(), ldw, sw, M, N, K, dt, out.data_ptr(), ldo, _current_raw_stream(dev))
    if st:
        _fail(st, "kda_fp8_matmul")
    return out


def kda_rotary_freqs(rot: int, base: float = 10000.0, scaling: Optional[str] = None, factor: float = 1.0,
                     original_len: int = 0, fast: float = 32.0, slow: float = 1.0,
                     device="cuda") -> Tuple[torch.Tensor, float]:
    """``(freqs, amplitude)`` for ``kda_rotary``: fp64 ``[rot / 2]`` radians per position, base^(-2 i / rot),
    and for contexts ``factor`` times longer than the ``original_len`` that a model was trained on

    * ``"linear"``: every frequency divided by factor;
    * ``"base"``: the base times factor^(rot / (rot - 2)), which divides the slowest by factor and
      keeps the fastest;
    * ``"ramp"``: pairs that make ``fast`` turns or more over original_len keep their frequency, those
      of ``slow`` turns or fewer have it divided by factor, and those between go from one to the
      other by their index; the amplitude is 0.1 ln(factor) + 1."""
    if rot < 0 or rot % 2 or not base > 1.0 or not factor >= 1.0:
        raise ValueError("rot even, base > 1 and factor >= 1 are expected")
    if scaling not in (None, "linear", "base", "ramp"):
        raise ValueError(f"scaling: None, 'linear', 'base' or 'ramp' expected, got {scaling!r}")
    amplitude = 1.0
    if scaling == "base" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    elif scaling == "ramp":
        if original_len <= 0 or not fast > slow > 0:
            raise ValueError("ramp: original_len > 0 and fast > slow > 0 are expected")
        lo, hi = (rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (fast, slow))
        keep = [1.0 - min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
        f = [x * k + x / factor * (1.0 - k) for x, k in zip(f, keep)]
        amplitude = 0.1 * math.log(factor) + 1.0
    return torch.tensor(f, dtype=torch.float64, device=device), amplitude


def _heads(name: str, t: torch.Tensor, T: int, dim: int, dev: int, dtype) -> Tuple[int, int]:
    """Token and head strides of [tokens, heads, dim] with contiguous channels."""
    if t.dtype is not dtype or t.dim() != 3 or t.get_device() != dev or t.shape[0] != T or t.shape[2] != dim:
        raise ValueError(f"{name}: {dtype} [{T}, heads, {dim}] on cuda:{dev} expected, got {t.dtype} {tuple(t.shape)} on {t.device}")
    ts, hs, cs = t.stride()
    if cs != 1 and dim > 1:
        raise ValueError(f"{name}: contiguous channels are expected")
    return ts, hs


def _vector(name: str, t: torch.Tensor, n: int, dtype, dev: int) -> int:
    if t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} expected, got {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous() or t.shape != (n,):
        raise ValueError(f"{name}: a contiguous [{n}] tensor on cuda:{dev} expected, got {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def kda_rotary(q: torch.Tensor, k: Optional[torch.Tensor], positions: torch.Tensor, freqs: torch.Tensor, amplitude: float = 1.0,
               interleaved: bool = False, inverse: bool = False, q_out: Optional[torch.Tensor] = None,
               k_out: Optional[torch.Tensor] = None, stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Rotary positions of q ``[T, q heads, D]`` and k ``[T, k heads, D]`` (or None), any token and head
    strides: the first 2 len(freqs) channels of each head turned by positions ``[T]`` (int32) times
    freqs (fp64), in pairs (i, i + len(freqs)), or (2 i, 2 i + 1) when interleaved.  Tokens with a
    negative position stay as they are.  Returns ``(q_out, k_out)``, new tensors unless given;
    an output may be its input (in place), and inputs and outputs may be parts of one tensor."""
    dev = _device("q", q)
    if stream is not None or dev != _current_device():
        return _run(dev, stream, lambda _: kda_rotary(q, k, positions, freqs, amplitude, interleaved, inverse, q_out, k_out))
    dtype = q.dtype
    dt = _dtype(dtype)
    if q.dim() != 3:
        raise ValueError(f"q: [tokens, heads, channels] expected, got {tuple(q.shape)}")
    T, Hq, D = q.shape
    qt, qh, qc = q.stride()
    if qc != 1 and D > 1:
        raise ValueError("q: contiguous channels are expected")
    n = freqs.numel()
    pp, fp = _vector("positions", positions, T, torch.int32, dev), _vector("freqs", freqs, n, torch.float64, dev)
    if q_out is None:
        q_out = _empty((T, Hq, D), dtype=dtype, device=q.device)
        qot, qoh = Hq * D, D
    else:
        qot, qoh = _heads("q_out", q_out, T, D, dev, dtype)
        if q_out.shape[1] != Hq:
            raise ValueError("q_out: q's shape is expected")
    Hk = kt = kh = kot = koh = 0
    kp = kop = None
    if k is not None:
        kt, kh = _heads("k", k, T, D, dev, dtype)
        Hk, kp = k.shape[1], k.data_ptr()
        if k_out is None:
            k_out = _empty((T, Hk, D), dtype=dtype, device=q.device)
            kot, koh = Hk * D, D
        else:
            kot, koh = _heads("k_out", k_out, T, D, dev, dtype)
            if k_out.shape[1] != Hk:
                raise ValueError("k_out: k's shape is expected")
        kop = k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    st = (_fns or _lib()).kda_rotary(q.data_ptr(), qt, qh, Hq, kp, kt, kh, Hk, pp, T, D, 2 * n, fp, amplitude, (1 if interleaved else 0) | (2 if inverse else 0),
                           dt, q_out.data_ptr(), qot, qoh, kop, kot, koh, _current_raw_stream(dev))
    if st:
        _fail(st, "kda_rotary")
    return q_out, k_out
