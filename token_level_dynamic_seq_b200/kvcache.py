"""The 8-bit key/value cache and the decode step over it (``include/logo_cache8.h``).

Keys and values are held as e4m3 or int8 codes with one fp32 scale for every
block of tokens and key/value head; the last two blocks of every sequence are
kept in bf16 as well, so that the cache depends on its tokens alone, however
they were appended.  A serving loop is::

    cache = logo.cache8(B, Hkv, Lmax, d, device)
    ws = logo.decode8_workspace(cache, Hq)
    logo.cache8_append(cache, k, v, start, ws=ws)                   # the prompts, start = 0
    logo.cache8_append(cache, k1, v1, length, ws=ws, new_len=held)  # each step: one new token,
    out, selected = logo.decode8(q, cache, held, gate, tau, window, ws=ws)

As in the rest of the binding, only pointers are marshalled here; tensors have
to lie on the current device.  Device-side errors go to the workspace's status
word (:func:`check`): a call without ``ws`` makes one of its own, and its errors
are not seen.  A ``stream`` that is not the current one has to be ordered behind
what made the inputs, and they have to be kept until it is done with them.
"""
from __future__ import annotations

import ctypes

import torch

import token_level_dynamic_seq_b200 as _logo

_TYPES = {torch.float8_e4m3fn: 0, torch.int8: 1}


class Cache8:
    """One layer's cache: codes ``k``, ``v`` [B, Hkv, Lmax, d] (float8_e4m3fn or int8), ``k_scale``,
    ``v_scale`` fp32 [B, Hkv, ceil(Lmax / block)], ``k_tail``, ``v_tail`` bf16 [B, Hkv, 2, block, d].
    The tensors are the caller's; :func:`cache8` allocates a set."""

    __slots__ = ("k", "v", "k_scale", "v_scale", "k_tail", "v_tail", "B", "Hkv", "Lmax", "d", "block", "device",
                 "index", "_desc", "_ref")

    def __init__(self, k, v, k_scale, v_scale, k_tail, v_tail):
        if k.dim() != 4 or k_tail.dim() != 5:
            raise ValueError("expected codes [B, Hkv, Lmax, d] and tails [B, Hkv, 2, block, d]")
        if k.dtype not in _TYPES:
            raise TypeError(f"expected float8_e4m3fn or int8 codes, got {k.dtype}")
        B, H, L, d = k.shape
        block = k_tail.shape[3]
        nblk = -(-L // block) if block else 0
        for name, t, dtype, shape in (("v", v, k.dtype, (B, H, L, d)),
                                      ("k_scale", k_scale, torch.float32, (B, H, nblk)),
                                      ("v_scale", v_scale, torch.float32, (B, H, nblk)),
                                      ("k_tail", k_tail, torch.bfloat16, (B, H, 2, block, d)),
                                      ("v_tail", v_tail, torch.bfloat16, (B, H, 2, block, d))):
            if t.dtype != dtype:
                raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
            if tuple(t.shape) != shape:
                raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")
        tensors = (k, v, k_scale, v_scale, k_tail, v_tail)
        for t in tensors:
            if not t.is_contiguous():
                raise ValueError("expected contiguous tensors")
            if t.device != k.device:
                raise ValueError("the cache's tensors lie on different devices")
        self.k, self.v, self.k_scale, self.v_scale, self.k_tail, self.v_tail = tensors
        self.B, self.Hkv, self.Lmax, self.d, self.block, self.device = B, H, L, d, block, k.device
        self.index = k.get_device() if k.is_cuda else -1
        self._desc = _logo.Cache8Desc(B, H, L, d, block, _TYPES[k.dtype], *(t.data_ptr() for t in tensors))
        self._ref = ctypes.byref(self._desc)

    @property
    def dtype(self):
        return self.k.dtype


def cache8(B: int, Hkv: int, Lmax: int, d: int, device, dtype=torch.float8_e4m3fn, block: int = 64) -> Cache8:
    """Allocates a cache.  Nothing in it has to be initialised (its contents are not)."""
    new = lambda shape, t: torch.empty(shape, dtype=t, device=device)  # noqa: E731
    code, scale, tail = (B, Hkv, Lmax, d), (B, Hkv, -(-Lmax // block)), (B, Hkv, 2, block, d)
    return Cache8(new(code, dtype), new(code, dtype), new(scale, torch.float32), new(scale, torch.float32),
                  new(tail, torch.bfloat16), new(tail, torch.bfloat16))


def _lib_on(cache: Cache8):
    """The library, for a cache on the current device."""
    if cache.index < 0:
        raise ValueError("expected a cache of CUDA tensors")
    if cache.index != torch.cuda.current_device():
        raise ValueError(f"the cache lies on {cache.device}, the current device is cuda:{torch.cuda.current_device()}")
    return _logo._lib or _logo.load_library()


def _at(cache: Cache8, t, dtype, count: int, name: str):
    """Address of a tensor that a call takes: of its type, contiguous, on the cache's device, with `count` elements."""
    if t.dtype is dtype and t.get_device() == cache.index and t.is_contiguous() and t.numel() >= count:
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != cache.index:
        raise ValueError(f"{name} lies on {t.device}, the cache on {cache.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    raise ValueError(f"{name}: expected {count} elements, got {t.numel()}")


def _queue(cache: Cache8, stream):
    """The stream's handle; the current stream's without making an object of it."""
    return torch._C._cuda_getCurrentRawStream(cache.index) if stream is None else stream.cuda_stream


def _new(stream, make):
    """A tensor that a call on `stream` writes.  It is allocated there: memory that the current stream gave back may
    still be in use by what is queued on it.  The caller goes on with the tensor on the current stream."""
    if stream is None:
        return make()
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream):
        t = make()
    t.record_stream(here)
    return t


def _new_ws(cache: Cache8, size: int, stream):
    ws = _new(stream, lambda: torch.empty(size, dtype=torch.uint8, device=cache.device))
    _logo._raise(_logo.load_library().logo_workspace_init(ws.data_ptr(), size, _logo._stream(stream)))
    return ws


def _rows_shape(cache: Cache8, rows: int, cu_seqlens, max_seqlen):
    if cu_seqlens is None:
        return _logo.Shape(cache.B, cache.Hkv, cache.Hkv, rows, cache.d, None, cache.B, rows)
    if max_seqlen is None:
        raise ValueError("max_seqlen is required with cu_seqlens (the library never reads device data on the host)")
    if cu_seqlens.numel() != cache.B + 1:
        raise ValueError(f"cu_seqlens: expected {cache.B + 1} offsets, got {cu_seqlens.numel()}")
    cu = _at(cache, cu_seqlens, torch.int32, 0, "cu_seqlens")
    return _logo.Shape(1, cache.Hkv, cache.Hkv, rows, cache.d, cu, cache.B, int(max_seqlen))


def cache8_append(cache: Cache8, k, v, start, ws=None, cu_seqlens=None, max_seqlen=None, new_len=None, stream=None):
    """Quantises new rows into the cache at positions ``start`` (int32 [B], device) onwards.

    ``k``, ``v``: bf16 [B, Hkv, n, d], or packed [1, Hkv, T, d] with ``cu_seqlens`` int32 [B + 1] and
    ``max_seqlen``.  ``start[b]`` may be the sequence's length so far, an earlier multiple of the block, or a
    position in the sequence's latest append (its last two blocks): rejected drafts are appended over.
    ``new_len`` (int32 [B]) receives start + n."""
    lib = _lib_on(cache)
    B, H, d = cache.B, cache.Hkv, cache.d
    n = k.shape[2] if k.dim() == 4 else -1
    want = (B if cu_seqlens is None else 1, H, n, d)
    if tuple(k.shape) != want or v.shape != k.shape:
        raise ValueError(f"k, v: expected {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
    ws = _new_ws(cache, 256, stream) if ws is None else ws
    shape = _rows_shape(cache, n, cu_seqlens, max_seqlen)
    _logo._raise(lib.logo_cache8_append(
        cache._ref, _at(cache, k, torch.bfloat16, 0, "k"), _at(cache, v, torch.bfloat16, 0, "v"), shape,
        _at(cache, start, torch.int32, B, "start"),
        None if new_len is None else _at(cache, new_len, torch.int32, B, "new_len"),
        _at(cache, ws, torch.uint8, 0, "ws"), ws.numel(), _queue(cache, stream)))


def cache8_read(cache: Cache8, start, rows: int, ws=None, cu_seqlens=None, max_seqlen=None, out=None, stream=None):
    """Reads ``rows`` positions from ``start`` (int32 [B], device) on back as bf16: (k, v) [B, Hkv, rows, d].

    With ``cu_seqlens`` int32 [B + 1] and ``max_seqlen`` the rows of all sequences come packed,
    [1, Hkv, rows, d] (``rows`` is their total).  ``out`` = (k, v) to write into."""
    lib = _lib_on(cache)
    rows = int(rows)
    want = (cache.B if cu_seqlens is None else 1, cache.Hkv, rows, cache.d)
    if out is None:
        out = _new(stream, lambda: cache.k_tail.new_empty((2,) + want)).unbind(0)
    k, v = out
    if tuple(k.shape) != want or tuple(v.shape) != want:
        raise ValueError(f"out: expected {want}, got {tuple(k.shape)} and {tuple(v.shape)}")
    ws = _new_ws(cache, 256, stream) if ws is None else ws
    shape = _rows_shape(cache, rows, cu_seqlens, max_seqlen)
    _logo._raise(lib.logo_cache8_read(
        cache._ref, _at(cache, start, torch.int32, cache.B, "start"), shape, _at(cache, k, torch.bfloat16, 0, "k_out"),
        _at(cache, v, torch.bfloat16, 0, "v_out"), _at(cache, ws, torch.uint8, 0, "ws"), ws.numel(),
        _queue(cache, stream)))
    return k, v


def decode8_workspace(cache: Cache8, Hq: int, n: int = 1, stream=None) -> torch.Tensor:
    """Workspace of :func:`decode8` for ``Hq`` query heads and ``n`` new tokens a sequence."""
    size = _logo.load_library().logo_decode8_workspace_size(cache._ref, int(Hq), int(n))
    if size == 0:
        raise _logo.LogoError(2, _logo.load_library().logo_last_error().decode())
    _lib_on(cache)
    return _new_ws(cache, size, stream)


def decode8(q, cache: Cache8, cache_len, gate, tau, window: int, ws=None, scale: float = 0.0, out=None, selected=None,
            stream=None):
    """Decode step over the cache: ``q`` bf16 [B, Hq, n, d] (or [B, Hq, d] for one token), ``cache_len`` int32 [B]
    (the new tokens included), ``gate`` fp32 [B, n], ``tau`` fp32 [1].  Returns (out, like q; selected int32 [B, n]).
    A given ``selected`` has gate's shape; either may be [B] for one token."""
    B, Hq, *n, d = q.shape
    if len(n) > 1 or B != cache.B or d != cache.d:
        raise ValueError(f"q: expected [{cache.B}, Hq, n, {cache.d}], got {tuple(q.shape)}")
    n = n[0] if n else 1
    # read by n from one sequence to the next: a longer buffer would give them each other's
    for name, t in (("gate", gate), ("selected", selected)):
        if t is not None and t.shape != (B, n) and not (n == 1 and t.shape == (B,)):
            raise ValueError(f"{name}: expected [{B}, {n}], got {list(t.shape)}")
    if tau.numel() != 1:
        raise ValueError(f"tau: expected one element, got {tau.numel()}")
    lib = _lib_on(cache)
    if ws is None:
        ws = decode8_workspace(cache, Hq, n, stream)
    if out is None:
        out = _new(stream, lambda: torch.empty_like(q))
    elif out.shape != q.shape:
        raise ValueError(f"out: expected {tuple(q.shape)}, got {tuple(out.shape)}")
    if selected is None:
        selected = _new(stream, lambda: cache_len.new_empty((B, n)))
    _logo._raise(lib.logo_decode8(
        _at(cache, q, torch.bfloat16, 0, "q"), cache._ref, _at(cache, cache_len, torch.int32, B, "cache_len"),
        _at(cache, gate, torch.float32, B * n, "gate"), _at(cache, tau, torch.float32, 1, "tau"), Hq, n, min(int(window), 0x7fffffff),
        float(scale), _at(cache, out, torch.bfloat16, 0, "out"), _at(cache, selected, torch.int32, B * n, "selected"),
        _at(cache, ws, torch.uint8, 0, "ws"), ws.numel(), _queue(cache, stream)))
    return out, selected
