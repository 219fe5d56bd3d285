"""Paged 4-bit key/value cache of a hybrid decoder's attention layers.

Thin ctypes binding of ``include/kda_kv4.h``, with the C names (the layout of the
cache, the rounding and the errors are stated there):

* ``kda_page_map(cached_lens, new_lens, block_table, free_pages, free_start,
  page_size, num_tokens)`` -> ``(cu_seqlens, seq_lens, slot_map, positions,
  free_next)``: block tables (updated in place) and slot maps from request lengths;
* ``kda_kv4_cache(num_pages, num_kv_heads, page_size, head_dim)`` -> an empty cache,
  uint8 ``[pages, kv heads, page_size / 16, 17 * head_dim]``;
* ``kda_kv4_append(k, v, slot_map, cache)``: new tokens into the cache;
* ``kda_kv4_gather(cache, slot_map, dtype)`` -> ``(k, v)``: tokens read back;
* ``kda_kv4_attention(q, cache, block_table, seq_lens, ...)`` -> ``o`` or ``(o, lse)``:
  softmax attention of each sequence's newest tokens over its cached ones.

Tensors are CUDA tensors of one device; a ``stream`` (default: the current one) is
a ``torch.cuda.Stream`` or a raw handle, and what a function allocates itself
belongs to that stream.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

__all__ = ["kda_page_map", "kda_kv4_cache", "kda_kv4_append", "kda_kv4_gather", "kda_kv4_attention",
           "kda_kv4_attention_workspace_size"]

_UNIT = 16          # tokens of a unit of the cache
_UNIT_BYTES = 17    # bytes of a unit per channel

_fns = None


def _lib():
    global _fns
    if _fns is None:
        from . import load_library
        lib = load_library()
        vp, i32, i64, sz, c = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int
        lib.kda_kv4_cache_bytes.argtypes = [i64, i32, i32, i32]
        lib.kda_kv4_cache_bytes.restype = sz
        lib.kda_page_map.argtypes = [vp, vp, i32, vp, i32, vp, i64, vp, i32, i64, vp, vp, vp, vp, vp, vp]
        lib.kda_page_map.restype = c
        lib.kda_kv4_append.argtypes = [vp, vp, vp, i64, i32, i32, i64, i64, i64, i64, c, vp, i64, i32, vp]
        lib.kda_kv4_append.restype = c
        lib.kda_kv4_gather.argtypes = [vp, i64, i32, vp, i64, i32, i32, c, vp, vp, vp]
        lib.kda_kv4_gather.restype = c
        lib.kda_kv4_attention_workspace_size.argtypes = [i64, i32, i32, i32, i32, i32, c]
        lib.kda_kv4_attention_workspace_size.restype = sz
        lib.kda_kv4_attention.argtypes = [vp, i64, i64, vp, i64, i32, vp, i32, vp, vp, i64, i32, i32, i32, i32, i32,
                                          ctypes.c_float, c, vp, vp, vp, sz, vp]
        lib.kda_kv4_attention.restype = c
        _fns = lib
    return _fns


def _check(status: int, where: str):
    if status != 0:
        from . import KdaError
        raise KdaError(status, where)


def _dtype(dt: torch.dtype) -> int:
    from . import _DT
    if dt not in _DT:
        raise TypeError(f"unsupported dtype {dt} (float32 or bfloat16)")
    return _DT[dt]


def _i32(name: str, t: torch.Tensor, dev: int, n: Optional[int] = None, dim: int = 1) -> int:
    """Data pointer of a dense int32 tensor of device ``dev`` with ``dim`` dimensions
    (and n entries)."""
    if t.dtype is not torch.int32:
        raise TypeError(f"{name}: int32 expected, got {t.dtype}")
    if t.get_device() != dev or not t.is_contiguous() or t.dim() != dim or (n is not None and t.numel() != n):
        raise ValueError(f"{name}: a contiguous {dim}-dimensional tensor{'' if n is None else f' of {n} entries'} on "
                         f"cuda:{dev} expected, got {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _device(name: str, t: torch.Tensor, dtype: Optional[torch.dtype] = None) -> int:
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name}: {dtype} expected, got {t.dtype}")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    return dev


# The handle alone: no Stream object per call.  A PyTorch without CUDA does not have it, and has no tensor that gets as far.
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(dev: int, stream, f):
    """f(handle of the stream) with device ``dev`` current, and the caller's stream for
    what f allocates."""
    if stream is None and dev == torch.cuda.current_device():
        return f(_current_raw_stream(dev))
    with torch.cuda.device(dev):
        if stream is None:
            return f(_current_raw_stream(dev))
        if not hasattr(stream, "cuda_stream"):
            stream = torch.cuda.ExternalStream(int(stream), device=torch.device("cuda", dev))
        with torch.cuda.stream(stream):
            return f(stream.cuda_stream)


def _dims(cache: torch.Tensor) -> Tuple[int, int, int, int]:
    """(pages, kv heads, page size, head dim) of a cache."""
    if cache.dtype is not torch.uint8 or cache.dim() != 4:
        raise ValueError("cache: uint8 [pages, kv heads, page_size / 16, 17 * head_dim] is expected")
    pages, heads, units, width = cache.shape
    if width % _UNIT_BYTES != 0:
        raise ValueError("cache: uint8 [pages, kv heads, page_size / 16, 17 * head_dim] is expected")
    if not cache.is_cuda or not cache.is_contiguous():
        raise ValueError("cache: a contiguous CUDA tensor is expected")
    return pages, heads, units * _UNIT, width // _UNIT_BYTES


def kda_kv4_cache(num_pages: int, num_kv_heads: int, page_size: int, head_dim: int, device="cuda") -> torch.Tensor:
    """An empty cache (zeros)."""
    if _lib().kda_kv4_cache_bytes(num_pages, num_kv_heads, page_size, head_dim) == (1 << 64) - 1:
        _check(1, "kda_kv4_cache")
    return torch.zeros((num_pages, num_kv_heads, page_size // _UNIT, _UNIT_BYTES * head_dim), dtype=torch.uint8,
                       device=device)


def kda_page_map(cached_lens: torch.Tensor, new_lens: torch.Tensor, block_table: torch.Tensor,
                 free_pages: torch.Tensor, free_start: torch.Tensor, page_size: int, num_tokens: int,
                 stream=None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]:
    """Block tables and slot maps of a step.  cached_lens, new_lens ``[N]``,
    block_table ``[N, max_pages]`` (updated in place), free_pages ``[F]``,
    free_start ``[1]``, all int32; ``num_tokens`` new tokens at most.  Returns int32
    ``(cu_seqlens [N + 1], seq_lens [N], slot_map [num_tokens], positions
    [num_tokens], free_next [1])``."""
    lib = _lib()
    dev = _device("cached_lens", cached_lens, torch.int32)
    N = cached_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != N:
        raise ValueError(f"block_table: [{N}, max_pages] expected, got {tuple(block_table.shape)}")
    if num_tokens < 0:
        raise ValueError("num_tokens < 0")
    max_pages = block_table.shape[1]
    args = (_i32("cached_lens", cached_lens, dev), _i32("new_lens", new_lens, dev, N), N,
            _i32("block_table", block_table, dev, dim=2), max_pages, _i32("free_pages", free_pages, dev),
            free_pages.numel(), _i32("free_start", free_start, dev, 1), page_size, num_tokens)
    pad = -num_tokens & 3   # one allocation; slot_map and positions begin on 16-byte boundaries
    room = num_tokens + pad

    def call(st):
        buf = cached_lens.new_empty(2 * room + 2 * N + 2)
        p = buf.data_ptr()
        _check(lib.kda_page_map(*args, p + 8 * room, p + 4 * (2 * room + N + 1), p, p + 4 * room,
                                p + 4 * (2 * room + 2 * N + 1), st), "kda_page_map")
        if pad:
            slots, _, pos, _, cu, lens, nxt = buf.split_with_sizes((num_tokens, pad, num_tokens, pad, N + 1, N, 1))
        else:
            slots, pos, cu, lens, nxt = buf.split_with_sizes((num_tokens, num_tokens, N + 1, N, 1))
        return cu, lens, slots, pos, nxt

    return _run(dev, stream, call)


def _strided(name: str, t: torch.Tensor, heads: int, dim: int, dev: int) -> Tuple[int, int]:
    """Token and head strides of [tokens, heads, dim] with contiguous channels."""
    if t.dim() != 3 or t.get_device() != dev:
        raise ValueError(f"{name}: [tokens, {heads}, {dim}] on cuda:{dev} expected, got {tuple(t.shape)} on {t.device}")
    T, H, D = t.shape
    ts, hs, cs = t.stride()
    if H != heads or D != dim or cs != 1:
        raise ValueError(f"{name}: [tokens, {heads}, {dim}] with contiguous channels expected, got {tuple(t.shape)}")
    return ts if T > 1 else 0, hs if H > 1 else 0   # a stride over one entry has no meaning


def kda_kv4_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, cache: torch.Tensor,
                   stream=None) -> None:
    """Writes k, v ``[T, kv heads, head dim]`` (token and head strides of 16-byte
    steps, such as parts of a fused projection) into the cache at slot_map ``[T]``
    int32; tokens with a negative slot are left out."""
    lib = _lib()
    dev = _device("k", k)
    pages, H, ps, D = _dims(cache)
    (kt, kh), (vt, vh) = _strided("k", k, H, D, dev), _strided("v", v, H, D, dev)
    T = k.shape[0]
    if v.dtype is not k.dtype or v.shape[0] != T or cache.get_device() != dev:
        raise ValueError("k, v and the cache differ in type, length or device")
    args = (k.data_ptr(), v.data_ptr(), _i32("slot_map", slot_map, dev, T), T, H, D, kt, kh, vt, vh, _dtype(k.dtype),
            cache.data_ptr(), pages, ps)
    _run(dev, stream, lambda st: _check(lib.kda_kv4_append(*args, st), "kda_kv4_append"))


def kda_kv4_gather(cache: torch.Tensor, slot_map: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cache's values at slot_map ``[T]`` int32: k, v ``[T, kv heads, head dim]``
    of ``dtype``, zeros at negative slots."""
    lib = _lib()
    pages, H, ps, D = _dims(cache)
    dev = cache.get_device()
    dt, sl, T = _dtype(dtype), _i32("slot_map", slot_map, dev), slot_map.numel()

    def call(st):
        k, v = cache.new_empty((2, T, H, D), dtype=dtype).unbind(0)
        _check(lib.kda_kv4_gather(cache.data_ptr(), pages, ps, sl, T, H, D, dt, k.data_ptr(), v.data_ptr(), st),
               "kda_kv4_gather")
        return k, v

    return _run(dev, stream, call)


def kda_kv4_attention_workspace_size(num_tokens: int, num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int,
                                     max_q_len: int, dtype: torch.dtype) -> int:
    """Bytes of workspace for ``kda_kv4_attention`` with these sizes."""
    n = _lib().kda_kv4_attention_workspace_size(num_tokens, num_seqs, num_heads, num_kv_heads, head_dim, max_q_len,
                                                _dtype(dtype))
    if n == (1 << 64) - 1:
        _check(1, "kda_kv4_attention_workspace_size")
    return int(n)


def kda_kv4_attention(q: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
                      cu_seqlens: Optional[torch.Tensor] = None, max_q_len: int = 1,
                      sm_scale: Optional[float] = None, return_lse: bool = False, o: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of the newest tokens of N sequences over their cached tokens.

    q ``[T, heads, head dim]`` (token and head strides of 16-byte steps), block_table
    ``[N, max_pages]``, seq_lens ``[N]`` (cached tokens, the new ones among them),
    cu_seqlens ``[N + 1]`` (int32; None: one query token per sequence), at most
    ``max_q_len`` query tokens per sequence; ``sm_scale`` defaults to head_dim^-1/2.
    Returns o ``[T, heads, head dim]``, and with ``return_lse`` the log of each row's
    sum of exponentials, fp32 ``[T, heads]``."""
    lib = _lib()
    dev = _device("q", q)
    pages, H, ps, D = _dims(cache)
    T, Hq = q.shape[0], q.shape[1]
    qt, qh = _strided("q", q, Hq, D, dev)
    if block_table.dim() != 2 or cache.get_device() != dev:
        raise ValueError(f"block_table [N, max_pages] and the cache are expected on cuda:{dev}")
    N, max_pages = block_table.shape
    dt = _dtype(q.dtype)
    bt, ln = _i32("block_table", block_table, dev, dim=2), _i32("seq_lens", seq_lens, dev, N)
    cu = None if cu_seqlens is None else _i32("cu_seqlens", cu_seqlens, dev, N + 1)
    if o is not None and (o.dtype is not q.dtype or o.shape != q.shape or not o.is_contiguous() or o.get_device() != dev):
        raise ValueError("o: a contiguous tensor of q's type, shape and device is expected")
    if workspace is not None and (not workspace.is_contiguous() or workspace.get_device() != dev):
        raise ValueError(f"workspace: a contiguous tensor on cuda:{dev} is expected")
    scale = D ** -0.5 if sm_scale is None else sm_scale

    def call(st):
        out = q.new_empty((T, Hq, D)) if o is None else o
        lse = q.new_empty((T, Hq), dtype=torch.float32) if return_lse else None
        if workspace is None:
            n = lib.kda_kv4_attention_workspace_size(T, N, Hq, H, D, max_q_len, dt)
            ws = cache.new_empty(256 if n == (1 << 64) - 1 else n)
        else:
            ws, n = workspace, workspace.numel() * workspace.element_size()
        _check(lib.kda_kv4_attention(q.data_ptr(), qt, qh, cache.data_ptr(), pages, ps, bt, max_pages, ln, cu, T, N, Hq, H,
                                     D, max_q_len, scale, dt, out.data_ptr(), lse.data_ptr() if return_lse else None,
                                     ws.data_ptr(), n, st), "kda_kv4_attention")
        return (out, lse) if return_lse else out

    return _run(dev, stream, call)
