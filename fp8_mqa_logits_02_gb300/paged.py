"""Paged caches: the operators of a serving step around the prefill logits.

``cache_write`` quantises new rows into pages of e4m3 values with one scale per row and head,
``cache_read`` packs sequences back out of them, ``logits_paged`` scores the newest tokens
straight from the pages (its result goes to ``topk``), and ``attention_paged`` attends to a
paged cache, all of it or the positions that ``topk`` selected.  Argument marshalling only, as
in the rest of the binding, but compiled (``csrc/paged_binding.cpp``: a serving step makes these
calls for every layer and token); layouts and limits are stated in ``include/fp8_mqa_logits.h``.

A cache is a tensor ``data [pages, page_size, heads, dim]`` (float8_e4m3fn, or for
``attention_paged`` also bfloat16 or float16) and, for e4m3, ``scale [pages, page_size, heads]``
float32.  Strides are free but for the last of ``data``, which is 1.

``stream`` (default: the current one of the tensors' device) is a stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
import sys

import torch

from . import Fp8MqaError, nvcc_build, _entry

_E4M3 = torch.float8_e4m3fn
_package = sys.modules[__package__]
_compiled = None
_bound = None  # which library build the compiled binding calls


def _binding():
    """The compiled binding, calling the library build that is in use; raises if either has not
    been built."""
    global _compiled, _bound
    if _bound is not _package._debug:
        entries = [ctypes.cast(_entry(f"fp8_mqa_{name}"), ctypes.c_void_p).value
                   for name in ("cache_write", "cache_read", "logits_paged",
                                "attention_paged_workspace_bytes", "attention_paged")]
        if _compiled is None:
            if not os.path.exists(nvcc_build.BINDING):
                raise RuntimeError(
                    f"{nvcc_build.BINDING} is missing: build it with "
                    "`python -m fp8_mqa_logits_02_gb300.nvcc_build` (there is no fallback)")
            spec = importlib.util.spec_from_file_location("_paged_binding", nvcc_build.BINDING)
            _compiled = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(_compiled)
        _compiled.bind(*entries, Fp8MqaError)
        _bound = _package._debug
    return _compiled


def _on(stream, like):
    """The context of a call on ``stream``.  Its kernels go to the device of the call's tensors (``like`` is
    one), so a stream of another device is refused."""
    device = getattr(like, "device", None)
    if device is not None and device.type == "cuda" and stream.device != device:
        raise ValueError(f"stream is on {stream.device}, expected {device}")
    return torch.cuda.stream(stream)


def load() -> None:
    """Load the compiled binding (the first call of any operator does the same)."""
    _binding()


def cache_write(slots: torch.Tensor, k: torch.Tensor, k_data: torch.Tensor, k_scale: torch.Tensor,
                v: torch.Tensor | None = None, v_data: torch.Tensor | None = None,
                v_scale: torch.Tensor | None = None, stream=None) -> None:
    """Quantise rows into one cache, or keys and values into two, in one launch.

    slots: int32 [T], page * page_size + row; a slot outside the cache is skipped (padding).
    k (and v, of the same type): bfloat16, float16 or float32 [T, heads, dim]; tokens and heads
    may be strided.  Each row gets the scale max|x| / 448 (at least 1e-30 / 448) and the e4m3
    values nearest to x / scale; a row with a NaN or an infinity reads back as NaN.
    """
    call = _binding().cache_write
    if stream is not None:
        with _on(stream, k_data):
            return call(slots, k, k_data, k_scale, v, v_data, v_scale)
    return call(slots, k, k_data, k_scale, v, v_data, v_scale)


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
    call = _binding().cache_read
    if stream is not None:
        with _on(stream, data):
            return call(data, scale, table, starts, total, dtype)
    return call(data, scale, table, starts, total, dtype)


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
    call = _binding().logits_paged
    if stream is not None:
        with _on(stream, q):
            return call(q, data, scale, w, table, lens, max_len, out, clean_logits)
    return call(q, data, scale, w, table, lens, max_len, out, clean_logits)


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
    The work is laid out for rows as long as the table is wide: with a table that was made for much
    longer rows, pass ``table[:, :columns]``.
    """
    call = _binding().attention_paged
    if stream is not None:
        with _on(stream, q):
            return call(q, k_data, v_data, table, lens, sm_scale, k_scale, v_scale, indices, return_lse)
    return call(q, k_data, v_data, table, lens, sm_scale, k_scale, v_scale, indices, return_lse)

