"""Attention layers beside the state-space layers: the paged key/value cache.

Python binding of ``ssd_kv_append``, ``ssd_kv_read`` and
``ssd_paged_attention`` (include/ssd.h): argument marshalling only, like
:mod:`state_space_model_gb300.ssd`.  Every step of the computation runs in
the CUDA kernels of ``libssd_gb300.so`` on the current torch stream.

The cache is two pools of pages, ``k_cache`` and ``v_cache`` [pages, Hkv, ps,
D], bf16 or f32, or ``torch.float8_e4m3fn`` with scales ``k_scale`` and
``v_scale`` [pages, Hkv, ps] f32 (an element stands for code * scale).  Slot s
is token s % ps of page s // ps; ``page_table`` [B, M] int32 names each
sequence's pages in order.  Memory laid out [pages, ps, Hkv, D] is passed as
``pool.transpose(1, 2)``.
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch

from . import _native

_CODES = {torch.float32: _native.SSD_F32, torch.bfloat16: _native.SSD_BF16,
          torch.int32: _native.SSD_I32, torch.float8_e4m3fn: _native.SSD_F8E4M3}

# One ssd_tensor of the C ABI: pointer, dtype, ndim, five extents, five strides.
_PACK = struct.Struct("@Pii10q")
assert _PACK.size == ctypes.sizeof(_native.SsdTensor)
_MOST = 16
_PAD = tuple((0,) * (5 - n) for n in range(6))


class _Descriptors(threading.local):
    """Room for the descriptors of one call, for each thread."""

    def __init__(self):
        self.room = ctypes.create_string_buffer(_MOST * _PACK.size)
        self.base = ctypes.addressof(self.room)


_local = _Descriptors()


def _describe(tensors):
    """Addresses of ssd_tensor descriptors of ``tensors`` (None -> None), valid
    until this thread's next call, and the tensors' device."""
    room, base, size = _local.room, _local.base, _PACK.size
    out, device, at = [], None, 0
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"expected a torch.Tensor, got {type(t).__name__}")
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (the library takes device pointers)")
        if device is None:
            device = t.device
        elif t.device != device:
            raise ValueError(f"tensors on different devices: {device} and {t.device}")
        shape = t.shape
        n = len(shape)
        if n > 5:
            raise ValueError("tensors of more than 5 dimensions are not supported")
        pad = _PAD[n]
        _PACK.pack_into(room, at, t.data_ptr(), _CODES.get(t.dtype, 99), n, *shape, *pad,
                        *t.stride(), *pad)
        out.append(base + at)
        at += size
    return out, device


def _stream(device):
    return torch.cuda.current_stream(device).cuda_stream


def kv_append(q, k, v, slots, k_cache, v_cache, *, k_scale=None, v_scale=None, positions=None,
              cos=None, sin=None, interleaved=False, q_weight=None, k_weight=None, eps=1e-6,
              out=None):
    """Norms, rotates and caches new tokens in one pass (``ssd_kv_append``).

    q [T,Hq,D], k and v [T,Hkv,D] (views of one projection's output do); each
    query and key head gets an RMS norm with ``q_weight`` / ``k_weight`` [D]
    f32 (None: no norm) and is rotated by row ``positions[t]`` of ``cos`` and
    ``sin`` [S,R/2] f32 (None: not rotated) in pairs (i, i + R/2), or (2i, 2i +
    1) if ``interleaved``.  Key and value go to slot ``slots[t]`` of the pools,
    quantised with one scale for each token and head if those are float8.  A
    token whose slot or position is out of range (-1, say) is padding: nothing
    is written for it.  Returns the queries [T,Hq,D] (``out`` if given)."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lib = _native.load()
    (dq, dk, dv, dslots, dpos, dcos, dsin, dqw, dkw, dkc, dvc, dks, dvs, dout), dev = _describe(
        (q, k, v, slots, positions, cos, sin, q_weight, k_weight, k_cache, v_cache, k_scale,
         v_scale, out))
    st = lib.ssd_kv_append(dq, dk, dv, dslots, dpos, dcos, dsin, dqw, dkw, eps,
                           1 if interleaved else 0, dkc, dvc, dks, dvs, dout, _stream(dev))
    if st:
        _native.check(st, "ssd_kv_append")
    return out


def kv_read(k_cache, v_cache, page_table, cu_lens, tokens, *, starts=None, k_scale=None,
            v_scale=None, dtype=None, out=None):
    """Cached keys and values as contiguous rows (``ssd_kv_read``).

    Row i of sequence b (``cu_lens[b] <= i < cu_lens[b + 1]``) is its position
    ``starts[b] + i - cu_lens[b]`` (``starts`` None: 0).  Returns k and v
    [tokens,Hkv,D] (or the pair ``out``) in the dtype of the pools; for float8
    pools in ``dtype``, bf16 (default) or f32, as code * scale."""
    if out is None:
        if dtype is None:
            dtype = torch.bfloat16 if k_cache.dtype == torch.float8_e4m3fn else k_cache.dtype
        shape = (tokens, k_cache.shape[1], k_cache.shape[3])
        out = (torch.empty(shape, dtype=dtype, device=k_cache.device),
               torch.empty(shape, dtype=dtype, device=k_cache.device))
    k, v = out
    lib = _native.load()
    d, dev = _describe((k_cache, v_cache, k_scale, v_scale, page_table, cu_lens, starts, k, v))
    st = lib.ssd_kv_read(*d, _stream(dev))
    if st:
        _native.check(st, "ssd_kv_read")
    return k, v


def paged_attention_workspace_size(batch, tokens, q_heads, kv_heads, headdim,
                                   cache_dtype=torch.bfloat16) -> int:
    """Bytes of workspace :func:`paged_attention` needs for this problem."""
    need = ctypes.c_size_t(0)
    st = _native.load().ssd_paged_attention_workspace_size(
        batch, tokens, q_heads, kv_heads, headdim, _CODES.get(cache_dtype, 99), ctypes.byref(need))
    _native.check(st, "ssd_paged_attention_workspace_size")
    return int(need.value)


def paged_attention(q, k_cache, v_cache, page_table, lens, *, k_scale=None, v_scale=None,
                    scale=None, window=0, return_lse=False, out=None, workspace=None):
    """Attention of T new tokens of each sequence over the cache
    (``ssd_paged_attention``).

    q [B,T,Hq,D]: the rows that :func:`kv_append` returned for the last T of
    the ``lens[b]`` tokens that the cache holds of sequence b (their keys
    included).  Row t sees its own and earlier positions, with ``window`` > 0
    only the last ``window`` of them; ``scale`` defaults to D ** -0.5.  Returns
    out [B,T,Hq,D], or (out, lse) with lse [B,T,Hq] f32, the log of each row's
    sum of exponentials; a row that sees nothing gives 0 and -inf.
    ``workspace`` may give a uint8 buffer of
    :func:`paged_attention_workspace_size` bytes."""
    Bn, T, Hq, D = q.shape
    if out is None:
        out = torch.empty((Bn, T, Hq, D), dtype=q.dtype, device=q.device)
    lse = torch.empty((Bn, T, Hq), dtype=torch.float32, device=q.device) if return_lse else None
    if workspace is None:
        need = paged_attention_workspace_size(Bn, T, Hq, k_cache.shape[1], D, k_cache.dtype)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    lib = _native.load()
    d, dev = _describe((q, k_cache, v_cache, k_scale, v_scale, page_table, lens, out, lse))
    if workspace is None:
        ws, ws_bytes = None, 0
    else:
        if workspace.device != dev:
            raise ValueError(f"tensors on different devices: {dev} and {workspace.device}")
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    st = lib.ssd_paged_attention(*d[:7], D ** -0.5 if scale is None else scale, window, d[7], d[8],
                                 ws, ws_bytes, _stream(dev))
    if st:
        _native.check(st, "ssd_paged_attention")
    return (out, lse) if return_lse else out
