"""Attention layers beside the state-space layers: the paged key/value cache.

Python binding of ``ssd_kv_append_ex``, ``ssd_kv_read_ex`` and
``ssd_paged_attention_ex`` (include/ssd.h): argument marshalling only, like
:mod:`state_space_model_gb300.ssd` (compiled, in ``_attn_ext``).  Every step
of the computation runs in the CUDA kernels of ``libssd_gb300.so`` on the
current torch stream.

The cache is two pools of pages, ``k_cache`` and ``v_cache`` [pages, Hkv, ps,
D], bf16 or f32, or ``torch.float8_e4m3fn`` with scales ``k_scale`` and
``v_scale`` [pages, Hkv, ps] f32 (an element stands for code * scale), or
``torch.float4_e2m1fn_x2`` [pages, Hkv, ps, D/2] (two 4-bit codes a byte, the even
place in the low bits) with those scales and ``k_group_scale`` and
``v_group_scale`` [pages, Hkv, ps, D/16] float8_e4m3fn besides (an element stands
for code * group scale * scale; make them as uint8 and ``view`` them, torch has few
operations for these types).  Slot s
is token s % ps of page s // ps; ``page_table`` [B, M] int32 names each
sequence's pages in order.  Memory laid out [pages, ps, Hkv, D] is passed as
``pool.transpose(1, 2)``, one allocation [pages, 2, Hkv, ps, D] as
``pool.unbind(1)``.
"""
from __future__ import annotations

import ctypes
import threading

import torch

from . import _native

_CODES = {torch.float32: _native.SSD_F32, torch.bfloat16: _native.SSD_BF16,
          torch.float8_e4m3fn: _native.SSD_F8E4M3}
if hasattr(torch, "float4_e2m1fn_x2"):       # torch 2.8; without it there are the other pools
    _CODES[torch.float4_e2m1fn_x2] = _native.SSD_F4E2M1X2
_OF_CODES = (_native.SSD_F8E4M3, _native.SSD_F4E2M1X2)

_ext_module = None
_lock = threading.Lock()


def _load():
    """The compiled marshalling (binding/attn_ext.cpp), bound to the loaded library."""
    global _ext_module
    with _lock:
        if _ext_module is None:
            lib = _native.load()
            try:
                from . import _attn_ext
            except ImportError as e:
                raise RuntimeError(f"the attention binding is not built ({e}); run `python -m "
                                   "state_space_model_gb300.build` (or __graft_entry__.build()) "
                                   "first") from e
            _attn_ext.bind(*[ctypes.cast(f, ctypes.c_void_p).value for f in (
                lib.ssd_kv_append_ex, lib.ssd_kv_read_ex, lib.ssd_paged_attention_ex,
                lib.ssd_paged_attention_workspace_size)])
            _ext_module = _attn_ext
    return _ext_module


def kv_append(q, k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None,
              k_group_scale=None, v_group_scale=None, positions=None, cos=None, sin=None,
              sections=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6, out=None):
    """Norms, rotates and caches new tokens in one pass (``ssd_kv_append_ex``).

    q [T,Hq,D], k and v [T,Hkv,D] (views of one projection's output do); each
    query and key head gets an RMS norm with ``q_weight`` / ``k_weight`` [D]
    f32 (None: no norm) and is rotated by row ``positions[t]`` of ``cos`` and
    ``sin`` [S,R/2] f32 (None: not rotated) in pairs (i, i + R/2), or (2i, 2i +
    1) if ``interleaved``.  ``sections`` (with ``positions`` [A,T], A of 2 to 4
    axes such as time, height and width): lengths of runs of pairs, which sum to
    R/2 and go round the axes; the pairs of run j turn by ``positions[j % A][t]``,
    so (16, 24, 24) gives each of three axes one run and (1,) * 60 + (4,) deals
    the pairs out in turn.  Key and value go to slot ``slots[t]`` of the pools,
    quantised with one scale for each token and head if those are float8, with
    one for each 16 places besides if they are float4.  A
    token whose slot or (any) position is out of range (-1, say) is padding: nothing
    is written for it.  Returns the queries [T,Hq,D] (``out`` if given)."""
    r = (_ext_module or _load()).kv_append(q, k, v, slots, positions, cos, sin, q_weight, k_weight,
                                           eps, interleaved, k_cache, v_cache, k_scale, v_scale,
                                           k_group_scale, v_group_scale, sections, out)
    if type(r) is int:
        _native.check(r, "ssd_kv_append_ex")
    return r


def kv_read(k_cache, v_cache, page_table, cu_lens, tokens, *, starts=None, k_scale=None,
            v_scale=None, k_group_scale=None, v_group_scale=None, dtype=None, out=None):
    """Cached keys and values as contiguous rows (``ssd_kv_read_ex``).

    Row i of sequence b (``cu_lens[b] <= i < cu_lens[b + 1]``) is its position
    ``starts[b] + i - cu_lens[b]`` (``starts`` None: 0).  Returns k and v
    [tokens,Hkv,D] (or the pair ``out``) in the dtype of the pools; for float8 and
    float4 pools in ``dtype``, bf16 (default) or f32, as code * scale or code *
    group scale * scale."""
    if out is not None:
        k, v = out
    else:
        k = v = None
        if dtype is not None and dtype is not k_cache.dtype and (
                _CODES.get(k_cache.dtype) not in _OF_CODES
                or dtype not in (torch.bfloat16, torch.float32)):
            raise ValueError(f"rows of {k_cache.dtype} pools cannot be read as {dtype}")
    r = (_ext_module or _load()).kv_read(k_cache, v_cache, k_scale, v_scale, k_group_scale,
                                         v_group_scale, page_table, cu_lens, starts, tokens,
                                         dtype == torch.float32, k, v)
    if type(r) is int:
        _native.check(r, "ssd_kv_read_ex")
    return r


def paged_attention_workspace_size(batch, tokens, q_heads, kv_heads, headdim,
                                   cache_dtype=torch.bfloat16) -> int:
    """Bytes of workspace :func:`paged_attention` needs for this problem."""
    need = ctypes.c_size_t(0)
    st = _native.load().ssd_paged_attention_workspace_size(
        batch, tokens, q_heads, kv_heads, headdim, _CODES.get(cache_dtype, 99), ctypes.byref(need))
    _native.check(st, "ssd_paged_attention_workspace_size")
    return int(need.value)


def paged_attention(q, k_cache, v_cache, page_table, lens, *, k_scale=None, v_scale=None,
                    k_group_scale=None, v_group_scale=None, scale=None, window=0, sinks=0,
                    return_lse=False, out=None, workspace=None):
    """Attention of T new tokens of each sequence over the cache
    (``ssd_paged_attention_ex``).

    q [B,T,Hq,D]: the rows that :func:`kv_append` returned for the last T of
    the ``lens[b]`` tokens that the cache holds of sequence b (their keys
    included).  Row t sees its own and earlier positions, with ``window`` > 0
    only the last ``window`` of them and the sequence's first ``sinks``; pages in between
    are not looked at.  ``scale`` defaults to D ** -0.5.  Returns
    out [B,T,Hq,D], or (out, lse) with lse [B,T,Hq] f32, the log of each row's
    sum of exponentials; a row that sees nothing gives 0 and -inf.
    ``workspace`` may give a uint8 buffer of
    :func:`paged_attention_workspace_size` bytes."""
    r = (_ext_module or _load()).paged_attention(q, k_cache, v_cache, k_scale, v_scale,
                                                 k_group_scale, v_group_scale, page_table, lens,
                                                 scale, window, sinks, return_lse, out, workspace)
    if type(r) is int:
        _native.check(r, "ssd_paged_attention_ex")
    return r
