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

import contextlib
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


def _i32(name: str, t: torch.Tensor, shape: Optional[tuple] = None) -> int:
    """Data pointer of a dense int32 CUDA tensor (of the given shape)."""
    if t.dtype is not torch.int32:
        raise TypeError(f"{name}: int32 expected, got {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{name}: a CUDA tensor is expected")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor is expected")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name}: shape {shape} expected, got {tuple(t.shape)}")
    return t.data_ptr()


def _same_device(*ts: Optional[torch.Tensor]):
    dev = None
    for t in ts:
        if t is None:
            continue
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"tensors on {dev} and {t.device}")
    return dev


@contextlib.contextmanager
def _on(device, stream):
    """The device made current, and the caller's stream for what is allocated
    inside; yields the stream's handle."""
    with contextlib.ExitStack() as st:
        if device.index is not None and device.index != torch.cuda.current_device():
            st.enter_context(torch.cuda.device(device))
        if stream is not None:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=device)
            st.enter_context(torch.cuda.stream(stream))
            yield stream.cuda_stream
        else:
            yield torch.cuda.current_stream().cuda_stream


def _dims(cache: torch.Tensor) -> Tuple[int, int, int, int]:
    """(pages, kv heads, page size, head dim) of a cache."""
    if cache.dtype is not torch.uint8 or cache.dim() != 4 or cache.shape[3] % _UNIT_BYTES != 0:
        raise ValueError("cache: uint8 [pages, kv heads, page_size / 16, 17 * head_dim] is expected")
    if not cache.is_cuda or not cache.is_contiguous():
        raise ValueError("cache: a contiguous CUDA tensor is expected")
    return cache.shape[0], cache.shape[1], cache.shape[2] * _UNIT, cache.shape[3] // _UNIT_BYTES


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
    if cached_lens.dim() != 1 or block_table.dim() != 2 or free_pages.dim() != 1:
        raise ValueError("cached_lens [N], block_table [N, max_pages], free_pages [F] are expected")
    N, max_pages = cached_lens.shape[0], block_table.shape[1]
    args = (_i32("cached_lens", cached_lens), _i32("new_lens", new_lens, (N,)), N,
            _i32("block_table", block_table, (N, max_pages)), max_pages, _i32("free_pages", free_pages),
            free_pages.shape[0], _i32("free_start", free_start, (1,)), page_size, num_tokens)
    dev = _same_device(cached_lens, new_lens, block_table, free_pages, free_start)
    if num_tokens < 0:
        raise ValueError("num_tokens < 0")
    with _on(dev, stream) as st:
        # one allocation; slot_map and positions begin on 16-byte boundaries
        room = (num_tokens + 3) & ~3
        buf = torch.empty(2 * room + 2 * N + 2, dtype=torch.int32, device=dev)
        slots, pos, cu, lens, nxt, _ = buf.split_with_sizes([room, room, N + 1, N, 1, 0])
        p = buf.data_ptr()
        _check(lib.kda_page_map(*args, p + 8 * room, p + 4 * (2 * room + N + 1), p, p + 4 * room,
                                p + 4 * (2 * room + 2 * N + 1), st), "kda_page_map")
    if room != num_tokens:
        slots, pos = slots[:num_tokens], pos[:num_tokens]
    return cu, lens, slots, pos, nxt


def _strided(name: str, t: torch.Tensor, heads: int, dim: int):
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != dim:
        raise ValueError(f"{name}: [tokens, {heads}, {dim}] expected, got {tuple(t.shape)}")
    if not t.is_cuda or (t.stride(2) != 1 and dim > 1):
        raise ValueError(f"{name}: a CUDA tensor with contiguous channels is expected")
    # a stride over one entry has no meaning
    return t.stride(0) if t.shape[0] > 1 else 0, t.stride(1) if heads > 1 else 0


def kda_kv4_append(k: torch.Tensor, v: torch.Tensor, slot_map: torch.Tensor, cache: torch.Tensor,
                   stream=None) -> None:
    """Writes k, v ``[T, kv heads, head dim]`` (token and head strides of 16-byte
    steps, such as parts of a fused projection) into the cache at slot_map ``[T]``
    int32; tokens with a negative slot are left out."""
    lib = _lib()
    pages, H, ps, D = _dims(cache)
    T = k.shape[0]
    (kt, kh), (vt, vh) = _strided("k", k, H, D), _strided("v", v, H, D)
    if v.dtype is not k.dtype or v.shape[0] != T:
        raise ValueError("k and v differ in type or length")
    dev = _same_device(k, v, slot_map, cache)
    dt, sl = _dtype(k.dtype), _i32("slot_map", slot_map, (T,))
    with _on(dev, stream) as st:
        _check(lib.kda_kv4_append(k.data_ptr(), v.data_ptr(), sl, T, H, D, kt, kh, vt, vh, dt, cache.data_ptr(),
                                  pages, ps, st), "kda_kv4_append")


def kda_kv4_gather(cache: torch.Tensor, slot_map: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                   stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The cache's values at slot_map ``[T]`` int32: k, v ``[T, kv heads, head dim]``
    of ``dtype``, zeros at negative slots."""
    lib = _lib()
    pages, H, ps, D = _dims(cache)
    if slot_map.dim() != 1:
        raise ValueError("slot_map: [T] is expected")
    T = slot_map.shape[0]
    dev = _same_device(cache, slot_map)
    dt, sl = _dtype(dtype), _i32("slot_map", slot_map)
    with _on(dev, stream) as st:
        k = torch.empty((T, H, D), dtype=dtype, device=dev)
        v = torch.empty((T, H, D), dtype=dtype, device=dev)
        _check(lib.kda_kv4_gather(cache.data_ptr(), pages, ps, sl, T, H, D, dt, k.data_ptr(), v.data_ptr(), st),
               "kda_kv4_gather")
    return k, v


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
    pages, H, ps, D = _dims(cache)
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError(f"q: [tokens, heads, {D}] expected, got {tuple(q.shape)}")
    T, Hq = q.shape[0], q.shape[1]
    if block_table.dim() != 2:
        raise ValueError("block_table: [N, max_pages] is expected")
    N, max_pages = block_table.shape
    qt, qh = _strided("q", q, Hq, D)
    dt = _dtype(q.dtype)
    bt, ln = _i32("block_table", block_table), _i32("seq_lens", seq_lens, (N,))
    cu = None if cu_seqlens is None else _i32("cu_seqlens", cu_seqlens, (N + 1,))
    dev = _same_device(q, cache, block_table, seq_lens, cu_seqlens, o, workspace)
    if o is not None and (o.dtype is not q.dtype or o.shape != q.shape or not o.is_contiguous()):
        raise ValueError("o: a contiguous tensor of q's type and shape is expected")
    need = lib.kda_kv4_attention_workspace_size(T, N, Hq, H, D, max_q_len, dt)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor is expected")
    with _on(dev, stream) as st:
        if o is None:
            o = torch.empty((T, Hq, D), dtype=q.dtype, device=dev)
        lse = torch.empty((T, Hq), dtype=torch.float32, device=dev) if return_lse else None
        if workspace is None:
            workspace = torch.empty(256 if need == (1 << 64) - 1 else need, dtype=torch.uint8, device=dev)
        _check(lib.kda_kv4_attention(q.data_ptr(), qt, qh, cache.data_ptr(), pages, ps, bt, max_pages, ln, cu, T, N, Hq, H,
                                     D, max_q_len, D ** -0.5 if sm_scale is None else sm_scale, dt, o.data_ptr(),
                                     None if lse is None else lse.data_ptr(), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), st), "kda_kv4_attention")
    return (o, lse) if return_lse else o
