"""Python binding of ``include/kva.h``: appending to and attending over the
paged cache.

Argument marshalling only, like :mod:`gqa_kv_cache_mla_gb300.kvw`, whose
library, cache descriptor (:func:`kvw.paged_cache`), status codes and error
type these calls share.  Tensors are passed as they are; their shapes give
the sizes unless keyword arguments override them.
"""
from __future__ import annotations

import ctypes
import os
import re

from . import kvw
from .kvw import HEADER as _KVW_HEADER
from .kvw import PagedCacheT, _done, _ptr, lib

HEADER = os.path.join(os.path.dirname(_KVW_HEADER), "kva.h")


def _declare(L):
    vp, u32, i64, u64, f32, i = (ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64,
                                 ctypes.c_uint64, ctypes.c_float, ctypes.c_int)
    pc, pu64 = ctypes.POINTER(PagedCacheT), ctypes.POINTER(ctypes.c_uint64)
    for name, args in {
        "kva_append_qkv_paged": [vp, i64, vp, i64, vp, u32, u32, u32, vp, vp, f32, f32, vp, u32,
                                 u32, vp, i, vp, pc, f32, u32, vp, vp],
        "kva_gqa_decode_paged": [vp, vp, vp, i64, vp, u32, u32, u32, pc, f32, u32, f32, f32, u32,
                                 vp, vp, u64, vp, vp],
        "kva_gqa_decode_workspace": [u32, u32, u32, pu64],
        "kva_mla_decode_paged": [vp, vp, vp, i64, vp, i64, vp, u32, u32, u32, pc, u32, f32, vp,
                                 u64, vp, vp],
        "kva_mla_decode_workspace": [u32, pu64],
    }.items():
        f = getattr(L, name)
        f.restype, f.argtypes = i, args


_declare(lib)


_raw_stream = None  # torch's current stream of a device, as a number


def _stream(stream):
    """The stream's handle; None means torch's current stream.  A small call's
    time is the host's: a number is had in 0.2 us, a Stream object in 3."""
    global _raw_stream
    if stream is not None:
        return kvw._stream(stream)
    if _raw_stream is None:
        import torch

        if not (torch.cuda.is_initialized() and hasattr(torch._C, "_cuda_getCurrentRawStream")
                and hasattr(torch._C, "_cuda_getDevice")):
            return kvw._stream(None)
        raw, device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        _raw_stream = lambda: raw(device())
    return _raw_stream()


def header_functions():
    """Names of the functions ``include/kva.h`` declares."""
    return sorted(set(re.findall(r"^\s*int\s+(kva_\w+)\s*\(", open(HEADER).read(), re.M)))


def _size(t):
    """Bytes of a workspace tensor."""
    return t.numel() * t.element_size()


def kva_append_qkv_paged(q_out, qkv, input_row_offsets, cache: PagedCacheT, freqs_cis,
                         layer_idx: int, q_gamma=None, k_gamma=None, epsilon: float = 1e-6,
                         weight_offset: float = 0.0, v_scale: float = 1.0, position_ids=None,
                         interleaved: bool = False, mrope_section=None, err_flags=None,
                         stream=None, *, num_batches=None, tot_seq_len=None, num_q_heads=None,
                         q_out_row_stride=None, qkv_row_stride=None, freqs_rows=None,
                         rope_dim=None, check=True) -> int:
    """``q_out`` [tokens, heads, head_size] (or None for no query heads), or any
    [tokens, ...] tensor with ``num_q_heads`` given; ``qkv`` [tokens, columns]."""
    B = input_row_offsets.shape[0] - 1 if num_batches is None else num_batches
    T = qkv.shape[0] if tot_seq_len is None else tot_seq_len
    if num_q_heads is None:
        num_q_heads = 0 if q_out is None else q_out.shape[1]
    qs = qkv.stride(0) if qkv_row_stride is None else qkv_row_stride
    if q_out_row_stride is None:
        q_out_row_stride = 0 if q_out is None else q_out.stride(0)
    if freqs_rows is None:
        freqs_rows = 0 if freqs_cis is None else freqs_cis.shape[0]
    if rope_dim is None:
        rope_dim = 0 if freqs_cis is None else freqs_cis.shape[1]
    sec = None
    if mrope_section is not None:
        sec = ctypes.cast((ctypes.c_uint32 * 3)(*[int(v) for v in mrope_section]),
                          ctypes.c_void_p)
    st = lib.kva_append_qkv_paged(
        _ptr(q_out), q_out_row_stride, _ptr(qkv), qs, _ptr(input_row_offsets), B, T, num_q_heads,
        _ptr(q_gamma), _ptr(k_gamma), epsilon, weight_offset, _ptr(freqs_cis), freqs_rows,
        rope_dim, _ptr(position_ids), int(bool(interleaved)), sec, ctypes.byref(cache), v_scale,
        layer_idx, _ptr(err_flags), _stream(stream))
    return _done(st, "kva_append_qkv_paged", check)


def kva_gqa_decode_workspace(num_q_heads: int, num_kv_heads: int, head_size: int) -> int:
    """Bytes of workspace :func:`kva_gqa_decode_paged` needs."""
    n = ctypes.c_uint64()
    _done(lib.kva_gqa_decode_workspace(num_q_heads, num_kv_heads, head_size, ctypes.byref(n)),
          "kva_gqa_decode_workspace", True)
    return n.value


def kva_gqa_decode_paged(out, q, input_row_offsets, cache: PagedCacheT, layer_idx: int,
                         sm_scale: float, workspace, lse=None, v_scale: float = 1.0,
                         softcap: float = 0.0, window: int = 0, alibi_slopes=None,
                         err_flags=None, stream=None, *, num_batches=None, tot_seq_len=None,
                         num_q_heads=None, q_row_stride=None, workspace_bytes=None,
                         check=True) -> int:
    """``out``, ``q`` [tokens, heads, head_size]; ``workspace`` any tensor of
    :func:`kva_gqa_decode_workspace` bytes."""
    B = input_row_offsets.shape[0] - 1 if num_batches is None else num_batches
    T = q.shape[0] if tot_seq_len is None else tot_seq_len
    H = q.shape[1] if num_q_heads is None else num_q_heads
    qs = q.stride(0) if q_row_stride is None else q_row_stride
    nb = _size(workspace) if workspace_bytes is None else workspace_bytes
    st = lib.kva_gqa_decode_paged(
        _ptr(out), _ptr(lse), _ptr(q), qs, _ptr(input_row_offsets), B, T, H, ctypes.byref(cache),
        v_scale, layer_idx, sm_scale, softcap, window, _ptr(alibi_slopes), _ptr(workspace), nb,
        _ptr(err_flags), _stream(stream))
    return _done(st, "kva_gqa_decode_paged", check)


def kva_mla_decode_workspace(num_heads: int) -> int:
    """Bytes of workspace :func:`kva_mla_decode_paged` needs."""
    n = ctypes.c_uint64()
    _done(lib.kva_mla_decode_workspace(num_heads, ctypes.byref(n)), "kva_mla_decode_workspace",
          True)
    return n.value


def kva_mla_decode_paged(out, q_latent, q_rope, input_row_offsets, cache: PagedCacheT,
                         layer_idx: int, sm_scale: float, workspace, lse=None, err_flags=None,
                         stream=None, *, num_batches=None, tot_seq_len=None, num_heads=None,
                         q_latent_row_stride=None, q_rope_row_stride=None, workspace_bytes=None,
                         check=True) -> int:
    """``out``, ``q_latent`` [tokens, heads, 512], ``q_rope`` [tokens, heads, 64]."""
    B = input_row_offsets.shape[0] - 1 if num_batches is None else num_batches
    T = q_latent.shape[0] if tot_seq_len is None else tot_seq_len
    H = q_latent.shape[1] if num_heads is None else num_heads
    ls = q_latent.stride(0) if q_latent_row_stride is None else q_latent_row_stride
    rs = q_rope.stride(0) if q_rope_row_stride is None else q_rope_row_stride
    nb = _size(workspace) if workspace_bytes is None else workspace_bytes
    st = lib.kva_mla_decode_paged(
        _ptr(out), _ptr(lse), _ptr(q_latent), ls, _ptr(q_rope), rs, _ptr(input_row_offsets), B, T,
        H, ctypes.byref(cache), layer_idx, sm_scale, _ptr(workspace), nb, _ptr(err_flags),
        _stream(stream))
    return _done(st, "kva_mla_decode_paged", check)
