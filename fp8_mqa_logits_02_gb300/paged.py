"""Paged caches: the operators of a serving step around the prefill logits.

``cache_write`` quantises new rows into pages of e4m3 values with one scale per row and head,
``cache_read`` packs sequences back out of them, ``logits_paged`` scores the newest tokens
straight from the pages (its result goes to ``topk``), and ``attention_paged`` attends to a
paged cache, all of it or the positions that ``topk`` selected.  Argument marshalling only, as
in the rest of the binding; layouts and limits are stated in ``include/fp8_mqa_logits.h``.

A cache is a tensor ``data [pages, page_size, heads, dim]`` (float8_e4m3fn, or for
``attention_paged`` also bfloat16 or float16) and, for e4m3, ``scale [pages, page_size, heads]``
float32.  Strides are free but for the last of ``data``, which is 1.
"""
from __future__ import annotations

import struct

import torch

from . import DIM, HEADS, Fp8MqaError, _entry, _on, _raw_stream, _stream_ptr

_E4M3 = torch.float8_e4m3fn
_TYPE = {_E4M3: 0, torch.bfloat16: 1, torch.float16: 2, torch.float32: 3}
_pack_cache = struct.Struct("@PPqiiiiqqqqqq").pack  # struct fp8mqa_cache


# A call's checks and its launch cost about the same, so each check reads an attribute once and finds
# out what is wrong only after it knows that something is.
def _cuda(t, name):
    """The device of a CUDA tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    return t.device


def _on_device(t, name, device):
    if not isinstance(t, torch.Tensor) or t.device != device:
        _cuda(t, name)
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _ints(t, name, device, *shape):
    """Checks an int32 tensor of ``shape`` (None: any size) whose last dimension is contiguous."""
    if isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.device == device:
        got = t.shape
        if len(got) == len(shape) and (shape[0] is None or got[0] == shape[0]):
            if t.stride(-1) == 1 or got[-1] < 2:
                return
            raise ValueError(f"{name} must be contiguous in its last dimension")
        raise ValueError(f"{name} must be {['any' if n is None else n for n in shape]}, got {list(got)}")
    _on_device(t, name, device)
    raise TypeError(f"{name} must be int32, got {t.dtype}")


def _cache(data, scale, name, device, other=None):
    """(the packed fp8mqa_cache, the data's shape); e4m3, or the type ``other``."""
    _on_device(data, f"{name} data", device)
    dtype, shape, stride = data.dtype, data.shape, data.stride()
    if len(shape) != 4:
        raise ValueError(f"{name} data must be [pages, page_size, heads, dim], got {list(shape)}")
    pages, page, heads, dim = shape
    x, y, z, one = stride
    if one != 1:
        raise ValueError(f"{name} data must be contiguous in its last dimension")
    if dtype is _E4M3:
        _on_device(scale, f"{name} scale", device)
        if scale.dtype is not torch.float32 or scale.shape != (pages, page, heads):
            raise ValueError(f"{name} scale must be float32 {[pages, page, heads]}")
        a, b, c = scale.stride()
        return _pack_cache(data.data_ptr(), scale.data_ptr(), pages, page, heads, dim, 0, x, y, z, a, b, c), shape
    if dtype is not other:
        raise TypeError(f"{name} data must be {_E4M3}{'' if other is None else f' or {other}'}, got {dtype}")
    if scale is not None:
        raise ValueError(f"{name} scale goes with float8_e4m3fn data only")
    return _pack_cache(data.data_ptr(), 0, pages, page, heads, dim, _TYPE[dtype], x, y, z, 0, 0, 0), shape


_current = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(name, device, stream, *args):
    index = device.index
    if stream is None and _raw_stream is not None and _current() == index:
        rc = _entry(name)(*args, _raw_stream(index))
    else:
        rc = _on(device, _entry(name), *args, _stream_ptr(stream, device))
    if rc != 0:
        raise Fp8MqaError(rc, name)


def _empty(shape, dtype, device, stream):
    """A new tensor, owned by the stream that the call goes to."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _rows(x, name, device, shape, dtype=None):
    """x [tokens, heads, dim] for cache_write: its address and strides."""
    _on_device(x, name, device)
    if x.dtype not in _TYPE or x.dtype == _E4M3 or (dtype is not None and x.dtype != dtype):
        raise TypeError(f"{name} must be bfloat16, float16 or float32"
                        f"{'' if dtype is None else ' as k is'}, got {x.dtype}")
    if x.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(x.shape)}")
    stride = x.stride()
    if stride[2] != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return x.data_ptr(), stride[0], stride[1]


def cache_write(slots: torch.Tensor, k: torch.Tensor, k_data: torch.Tensor, k_scale: torch.Tensor,
                v: torch.Tensor | None = None, v_data: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None, stream=None) -> None:
    """Quantise rows into one cache, or keys and values into two, in one launch.

    slots: int32 [T], page * page_size + row; a slot outside the cache is skipped (padding).
    k (and v, of the same type): bfloat16, float16 or float32 [T, heads, dim]; tokens and heads
    may be strided.  Each row gets the scale max|x| / 448 (at least 1e-30 / 448) and the e4m3
    values nearest to x / scale; a row with a NaN or an infinity reads back as NaN.
    """
    dev = _cuda(k_data, "k data")
    cache, shape = _cache(k_data, k_scale, "k", dev)
    _ints(slots, "slots", dev, None)
    rows = (slots.shape[0], shape[2], shape[3])
    x = _rows(k, "k", dev, rows)
    if (v is None) != (v_data is None) or (v is None) != (v_scale is None):
        raise ValueError("v, v_data and v_scale go together")
    if v is None:
        x2, cache2 = (None, 0, 0), None
    else:
        cache2, shape2 = _cache(v_data, v_scale, "v", dev)
        if shape2[1:] != shape[1:]:
            raise ValueError(f"v data must be {list(shape[1:])} a page, as k data is")
        x2 = _rows(v, "v", dev, rows, k.dtype)
    _call("fp8_mqa_cache_write", dev, stream, slots.data_ptr(), rows[0], _TYPE[k.dtype], *x, cache,
          *x2, cache2)


def cache_read(data: torch.Tensor, scale: torch.Tensor, table: torch.Tensor, starts: torch.Tensor,
               total: int, dtype: torch.dtype = _E4M3, stream=None):
    """Pack the sequences of a page table, one after the other, out of an e4m3 cache.

    table: int32 [B, columns] page ids; starts: int32 [B + 1], sequence b goes to rows
    starts[b] .. starts[b + 1] - 1; total: the number of output rows (starts[B]; it is not read
    back from the device).  With ``dtype`` float8_e4m3fn returns (rows [total, heads, dim],
    scales float32 [total, heads]), for one head the ``k`` and ``kv_scale`` of fp8_mqa_logits
    after ``squeeze(1)``; otherwise rows of ``dtype``, values times scale.  Rows whose page is not
    there are zero.
    """
    dev = _cuda(data, "data")
    cache, shape = _cache(data, scale, "cache", dev)
    _ints(table, "table", dev, None, None)
    rows, cols = table.shape
    _ints(starts, "starts", dev, rows + 1)
    if dtype not in _TYPE:
        raise TypeError(f"dtype must be one of {list(_TYPE)}, got {dtype}")
    total = int(total)
    if total < 0:
        raise ValueError("total must not be negative")
    out = _empty((total, shape[2], shape[3]), dtype, dev, stream)
    scales = _empty((total, shape[2]), torch.float32, dev, stream) if dtype == _E4M3 else None
    _call("fp8_mqa_cache_read", dev, stream, cache, table.data_ptr(), table.stride(0), cols,
          starts.data_ptr(), rows, total, _TYPE[dtype], out.data_ptr(),
          None if scales is None else scales.data_ptr())
    return out if scales is None else (out, scales)


def logits_paged(q: torch.Tensor, data: torch.Tensor, scale: torch.Tensor, w: torch.Tensor,
                 table: torch.Tensor, lens: torch.Tensor, max_len: int | None = None,
                 out: torch.Tensor | None = None, clean_logits: bool = True,
                 stream=None) -> torch.Tensor:
    """Indexer logits of each sequence's newest tokens against its own paged keys.

    q: float8_e4m3fn [B, T, 32, 128], the T newest tokens of each sequence; w: float32 [B, T, 32];
    data, scale: the keys' cache with one head of width 128; table: int32 [B, columns]; lens:
    int32 [B], lengths with the new tokens included.  Token t sees positions
    n < lens[b] - (T - 1 - t).  Returns float32 [B * T, max_len] (default: all that the table can
    hold), -inf outside (left as they are with ``clean_logits=False``); ``out`` may have strided rows.
    """
    dev = _cuda(q, "q")
    got = q.shape
    if q.dtype != _E4M3 or len(got) != 4 or got[2] != HEADS or got[3] != DIM or not q.is_contiguous():
        raise ValueError(f"q must be contiguous float8_e4m3fn [B, T, {HEADS}, {DIM}]")
    B, T = got[0], got[1]
    _on_device(w, "w", dev)
    if w.dtype != torch.float32 or w.shape != (B, T, HEADS) or not w.is_contiguous():
        raise ValueError(f"w must be contiguous float32 [{B}, {T}, {HEADS}]")
    cache, shape = _cache(data, scale, "key", dev)
    if shape[2] != 1 or shape[3] != DIM:
        raise ValueError(f"key data must be [pages, page_size, 1, {DIM}]")
    _ints(table, "table", dev, B, None)
    _ints(lens, "lens", dev, B)
    cols = table.shape[1]
    N = cols * shape[1] if max_len is None else int(max_len)
    if N < 0:
        raise ValueError("max_len must not be negative")
    if out is None:
        out, ld = _empty((B * T, N), torch.float32, dev, stream), N
    else:
        _on_device(out, "out", dev)
        if out.dtype != torch.float32 or out.shape != (B * T, N) or (N > 1 and out.stride(1) != 1):
            raise ValueError(f"out must be float32 [{B * T}, {N}] with contiguous rows")
        ld = out.stride(0) if B * T > 1 else N
    _call("fp8_mqa_logits_paged", dev, stream, q.data_ptr(), w.data_ptr(), B, T, HEADS, DIM, cache,
          table.data_ptr(), table.stride(0), cols, lens.data_ptr(), out.data_ptr(), ld, N,
          1 if clean_logits else 0)
    return out


# Workspace bytes by (device, query heads, key heads, width): they depend on nothing else.
_workspace = {}


def attention_paged(q: torch.Tensor, k_data: torch.Tensor, v_data: torch.Tensor,
                    table: torch.Tensor, lens: torch.Tensor, sm_scale: float | None = None,
                    k_scale: torch.Tensor | None = None, v_scale: torch.Tensor | None = None,
                    indices: torch.Tensor | None = None, return_lse: bool = False, stream=None):
    """Attention of one new token per row over a paged key and value cache.

    q: bfloat16 or float16 [B, q_heads, dim] (rows and heads may be strided); k_data, v_data:
    caches of float8_e4m3fn (with k_scale and v_scale) or of q's type, q_heads a multiple of
    their heads; table: int32 [B, columns] (an expanded row shares one sequence); lens: int32 [B];
    sm_scale: default dim ** -0.5.  ``indices``: int32 [B, S], the positions that each row attends
    to instead of all, in any order, as ``topk`` returns them; entries outside [0, lens[b]) are
    ignored.  Returns out [B, q_heads, dim] in q's type, and with ``return_lse`` the float32
    [B, q_heads] log of the softmax's sum.  A row with nothing to attend to gives 0 and -inf.
    """
    dev, dtype = _cuda(q, "q"), q.dtype
    if dtype != torch.bfloat16 and dtype != torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    if q.dim() != 3 or q.stride(2) != 1:
        raise ValueError("q must be [B, q_heads, dim], contiguous in its last dimension")
    B, heads, dim = q.shape
    k, shape = _cache(k_data, k_scale, "k", dev, dtype)
    v, shape2 = _cache(v_data, v_scale, "v", dev, dtype)
    if shape != shape2 or k_data.dtype != v_data.dtype:
        raise ValueError("k data and v data must have one shape and type")
    kv_heads = shape[2]
    if shape[3] != dim or heads == 0 or kv_heads == 0 or heads % kv_heads:
        raise ValueError(f"q {list(q.shape)} does not go with a cache of {list(shape)}")
    _ints(table, "table", dev, B, None)
    _ints(lens, "lens", dev, B)
    if indices is None:
        at, by, n = None, 0, -1
    else:
        _ints(indices, "indices", dev, B, None)
        at, by, n = indices.data_ptr(), indices.stride(0), indices.shape[1]
    key = (dev.index, heads, kv_heads, dim)
    need = _workspace.get(key)
    if need is None:
        need = _on(dev, _entry("fp8_mqa_attention_paged_workspace_bytes"), heads, kv_heads, dim)
        if need:
            _workspace[key] = need
    out = _empty((B, heads, dim), dtype, dev, stream)
    lse = _empty((B, heads), torch.float32, dev, stream) if return_lse else None
    space = _empty((need,), torch.uint8, dev, stream)
    _call("fp8_mqa_attention_paged", dev, stream, q.data_ptr(), _TYPE[dtype], B, heads,
          q.stride(0), q.stride(1), k, v, table.data_ptr(), table.stride(0), table.shape[1],
          lens.data_ptr(), at, by, n, dim ** -0.5 if sm_scale is None else float(sm_scale),
          out.data_ptr(), None if lse is None else lse.data_ptr(), space.data_ptr(), need)
    return (out, lse) if return_lse else out
