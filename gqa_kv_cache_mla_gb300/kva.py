"""Python binding of ``include/kva.h``: appending to and attending over the
paged cache, also one held in 4 bits, and the page tables of a step.

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
DTYPE_INT4 = 3  # of a descriptor for the *_int4 calls
GROUP = 64      # columns that share a scale


class GroupScalesT(ctypes.Structure):
    """Mirror of ``kva_group_scales_t``."""

    _fields_ = [("data", ctypes.c_void_p)] + [
        ("stride_" + d, ctypes.c_int64) for d in ("page", "kv", "layer", "head")]


def _declare(L):
    vp, u32, i64, u64, f32, i = (ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64,
                                 ctypes.c_uint64, ctypes.c_float, ctypes.c_int)
    pc, pu64 = ctypes.POINTER(PagedCacheT), ctypes.POINTER(ctypes.c_uint64)
    ps = ctypes.POINTER(GroupScalesT)
    for name, args in {
        "kva_append_qkv_paged": [vp, i64, vp, i64, vp, u32, u32, u32, vp, vp, f32, f32, vp, u32,
                                 u32, vp, i, vp, pc, f32, u32, vp, vp],
        "kva_gqa_decode_paged": [vp, vp, vp, i64, vp, u32, u32, u32, pc, f32, u32, f32, f32, u32,
                                 vp, vp, u64, vp, vp],
        "kva_gqa_decode_workspace": [u32, u32, u32, pu64],
        "kva_mla_decode_paged": [vp, vp, vp, i64, vp, i64, vp, u32, u32, u32, pc, u32, f32, vp,
                                 u64, vp, vp],
        "kva_mla_decode_workspace": [u32, pu64],
        "kva_append_qkv_int4": [vp, i64, vp, i64, vp, u32, u32, u32, vp, vp, f32, f32, vp, u32,
                                u32, vp, i, vp, pc, ps, u32, vp, vp],
        "kva_gather_kv_int4": [vp, vp, i64, pc, ps, u32, vp, vp, u32, u32, vp, vp],
        "kva_gqa_decode_int4": [vp, vp, vp, i64, vp, u32, u32, u32, pc, ps, u32, f32, f32, u32, vp,
                                vp, u64, vp, vp],
        "kva_extend_page_tables": [vp, u32, vp, vp, u32, u32, u32, u32, vp, u32, vp, vp, vp, vp,
                                   vp],
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


def _check_integers(name, t, size=4):
    """ValueError unless t holds integers of `size` bytes (or is an address)."""
    d = getattr(t, "dtype", None)
    if d is not None and (d.itemsize != size or d.is_floating_point or d.is_complex):
        raise ValueError("%s: integers of %d bits, not %s" % (name, 8 * size, d))


def _append(call, place, q_out, qkv, input_row_offsets, cache, freqs_cis, layer_idx, q_gamma,
            k_gamma, epsilon, weight_offset, position_ids, interleaved, mrope_section, err_flags,
            stream, num_batches, tot_seq_len, num_q_heads, q_out_row_stride, qkv_row_stride,
            freqs_rows, rope_dim):
    """The two appends' status; ``place`` is what stands between cache and layer."""
    B = input_row_offsets.shape[0] - 1 if num_batches is None else num_batches
    T = qkv.shape[0] if tot_seq_len is None else tot_seq_len
    if num_q_heads is None:
        num_q_heads = 0 if q_out is None else q_out.shape[1]
    qs = qkv.stride(0) if qkv_row_stride is None else qkv_row_stride
    if q_out_row_stride is None:
        q_out_row_stride = 0 if q_out is None else q_out.stride(0)
    if freqs_rows is None or rope_dim is None:
        size = (0, 0) if freqs_cis is None else freqs_cis.shape
        freqs_rows = size[0] if freqs_rows is None else freqs_rows
        rope_dim = size[1] if rope_dim is None else rope_dim
    sec = None
    if mrope_section is not None:
        sec = ctypes.cast((ctypes.c_uint32 * 3)(*[int(v) for v in mrope_section]),
                          ctypes.c_void_p)
    return call(
        _ptr(q_out), q_out_row_stride, _ptr(qkv), qs, _ptr(input_row_offsets), B, T, num_q_heads,
        _ptr(q_gamma), _ptr(k_gamma), epsilon, weight_offset, _ptr(freqs_cis), freqs_rows,
        rope_dim, _ptr(position_ids), 1 if interleaved else 0, sec, ctypes.byref(cache), place,
        layer_idx, _ptr(err_flags), _stream(stream))


def kva_append_qkv_paged(q_out, qkv, input_row_offsets, cache: PagedCacheT, freqs_cis,
                         layer_idx: int, q_gamma=None, k_gamma=None, epsilon: float = 1e-6,
                         weight_offset: float = 0.0, v_scale: float = 1.0, position_ids=None,
                         interleaved: bool = False, mrope_section=None, err_flags=None,
                         stream=None, *, num_batches=None, tot_seq_len=None, num_q_heads=None,
                         q_out_row_stride=None, qkv_row_stride=None, freqs_rows=None,
                         rope_dim=None, check=True) -> int:
    """``q_out`` [tokens, heads, head_size] (or None for no query heads), or any
    [tokens, ...] tensor with ``num_q_heads`` given; ``qkv`` [tokens, columns]."""
    st = _append(lib.kva_append_qkv_paged, v_scale, q_out, qkv, input_row_offsets, cache,
                 freqs_cis, layer_idx, q_gamma, k_gamma, epsilon, weight_offset, position_ids,
                 interleaved, mrope_section, err_flags, stream, num_batches, tot_seq_len,
                 num_q_heads, q_out_row_stride, qkv_row_stride, freqs_rows, rope_dim)
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


# ------------------------------------------------------------------ 4 bits

def group_scales(data, strides) -> GroupScalesT:
    """Fill a ``kva_group_scales_t``; ``strides`` = (page, kv, layer, head) in elements."""
    s = GroupScalesT()
    s.data = _ptr(data)
    s.stride_page, s.stride_kv, s.stride_layer, s.stride_head = strides
    return s


def int4_cache(codes, scales, page_table, cache_lengths):
    """The two descriptors of a cache held in 4 bits, for ``codes`` uint8
    [pages, 2, layers, heads, page_size, head_size / 2] and ``scales`` bf16
    [pages, 2, layers, heads, groups, page_size], views whose last two
    dimensions are dense, an int32 page table and int32 lengths."""
    import torch

    _check_integers("page_table", page_table)
    _check_integers("cache_lengths", cache_lengths)
    pages, planes, layers, heads, page_size, half = codes.shape
    d, groups = 2 * half, -(-2 * half // GROUP)
    if planes != 2 or tuple(scales.shape) != (pages, 2, layers, heads, groups, page_size) \
            or codes.element_size() != 1 or scales.dtype != torch.bfloat16 \
            or tuple(codes.stride()[4:]) != (half, 1) \
            or scales.stride()[5] != 1 or (groups > 1 and scales.stride()[4] != page_size):
        raise ValueError("codes %s %s and scales %s %s are not those of a cache in 4 bits"
                         % (tuple(codes.shape), codes.dtype, tuple(scales.shape), scales.dtype))
    st = codes.stride()
    cache = kvw.paged_cache(codes, DTYPE_INT4, page_table, cache_lengths, pages, layers, page_size,
                            heads, d, (2 * st[0], 2 * st[1], 2 * st[2], d, 2 * st[3]))
    return cache, group_scales(scales, scales.stride()[:4])


def kva_append_qkv_int4(q_out, qkv, input_row_offsets, cache: PagedCacheT, scales: GroupScalesT,
                        freqs_cis, layer_idx: int, q_gamma=None, k_gamma=None,
                        epsilon: float = 1e-6, weight_offset: float = 0.0, position_ids=None,
                        interleaved: bool = False, mrope_section=None, err_flags=None, stream=None,
                        *, num_batches=None, tot_seq_len=None, num_q_heads=None,
                        q_out_row_stride=None, qkv_row_stride=None, freqs_rows=None, rope_dim=None,
                        check=True) -> int:
    """:func:`kva_append_qkv_paged` to a cache held in 4 bits."""
    st = _append(lib.kva_append_qkv_int4, ctypes.byref(scales), q_out, qkv, input_row_offsets,
                 cache, freqs_cis, layer_idx, q_gamma, k_gamma, epsilon, weight_offset,
                 position_ids, interleaved, mrope_section, err_flags, stream, num_batches,
                 tot_seq_len, num_q_heads, q_out_row_stride, qkv_row_stride, freqs_rows, rope_dim)
    return _done(st, "kva_append_qkv_int4", check)


def kva_gather_kv_int4(k_out, v_out, ctx_offsets, cache: PagedCacheT, scales: GroupScalesT,
                       layer_idx: int, first_positions=None, err_flags=None, stream=None, *,
                       num_batches=None, total_rows=None, out_row_stride=None, check=True) -> int:
    """``k_out``, ``v_out`` [rows, heads, head_size], of the same row stride;
    either may be None."""
    one = v_out if k_out is None else k_out
    B = ctx_offsets.shape[0] - 1 if num_batches is None else num_batches
    R = (0 if one is None else one.shape[0]) if total_rows is None else total_rows
    try:
        wide = (k_out is None or k_out.element_size() == 2) \
            and (v_out is None or v_out.element_size() == 2)
    except AttributeError:  # addresses among them
        wide = True
    if not wide:
        raise ValueError("rows are written in bf16")
    if out_row_stride is None:
        out_row_stride = 0 if one is None else one.stride(0)
        if k_out is not None and v_out is not None and v_out.stride(0) != out_row_stride:
            raise ValueError("k_out and v_out have different row strides")
    st = lib.kva_gather_kv_int4(
        _ptr(k_out), _ptr(v_out), out_row_stride, ctypes.byref(cache), ctypes.byref(scales),
        layer_idx, _ptr(ctx_offsets), _ptr(first_positions), B, R, _ptr(err_flags),
        _stream(stream))
    return _done(st, "kva_gather_kv_int4", check)


def kva_gqa_decode_int4(out, q, input_row_offsets, cache: PagedCacheT, scales: GroupScalesT,
                        layer_idx: int, sm_scale: float, workspace, lse=None, softcap: float = 0.0,
                        window: int = 0, alibi_slopes=None, err_flags=None, stream=None, *,
                        num_batches=None, tot_seq_len=None, num_q_heads=None, q_row_stride=None,
                        workspace_bytes=None, check=True) -> int:
    """``out``, ``q`` [tokens, heads, head_size]; ``workspace`` any tensor of
    :func:`kva_gqa_decode_workspace` bytes."""
    B = input_row_offsets.shape[0] - 1 if num_batches is None else num_batches
    T = q.shape[0] if tot_seq_len is None else tot_seq_len
    H = q.shape[1] if num_q_heads is None else num_q_heads
    qs = q.stride(0) if q_row_stride is None else q_row_stride
    nb = _size(workspace) if workspace_bytes is None else workspace_bytes
    st = lib.kva_gqa_decode_int4(
        _ptr(out), _ptr(lse), _ptr(q), qs, _ptr(input_row_offsets), B, T, H, ctypes.byref(cache),
        ctypes.byref(scales), layer_idx, sm_scale, softcap, window, _ptr(alibi_slopes),
        _ptr(workspace), nb, _ptr(err_flags), _stream(stream))
    return _done(st, "kva_gqa_decode_int4", check)


# ------------------------------------------------------------------ page tables

_int32 = _int64 = object()  # torch's types, once a call has looked


def _check_tables(*tensors):
    """The types of a call's tensors, the slot map last."""
    global _int32, _int64
    import torch

    _int32, _int64 = torch.int32, torch.int64
    for name, t in zip(("page_table", "cache_lengths", "input_row_offsets", "free_pages", "taken",
                        "taken_out"), tensors):
        _check_integers(name, t)
    _check_integers("slot_map", tensors[-1], 8)


def kva_extend_page_tables(page_table, cache_lengths, input_row_offsets, free_pages, taken,
                           taken_out, page_size: int, num_pages: int, slot_map=None,
                           err_flags=None, stream=None, *, num_batches=None, tot_seq_len=None,
                           max_pages_per_seq=None, num_free=None, check=True) -> int:
    """``page_table`` int32 [requests, width], ``free_pages`` int32 ids,
    ``taken``, ``taken_out`` int32 [1], ``slot_map`` int64 [tokens] or None
    (then ``tot_seq_len`` is needed).  Other types are refused: ids of 64 bits
    would be read as two each."""
    # (a small call's time is the host's: comparisons of identity, 0.2 us in all)
    try:
        right = page_table.dtype is cache_lengths.dtype is input_row_offsets.dtype \
            is free_pages.dtype is taken.dtype is taken_out.dtype is _int32 \
            and (slot_map is None or slot_map.dtype is _int64)
    except AttributeError:  # addresses among them
        right = False
    if not right:
        _check_tables(page_table, cache_lengths, input_row_offsets, free_pages, taken, taken_out,
                      slot_map)
    B = input_row_offsets.numel() - 1 if num_batches is None else num_batches
    if tot_seq_len is None:
        if slot_map is None:
            raise ValueError("without a slot map the number of tokens has to be given")
        tot_seq_len = slot_map.numel()
    width = page_table.shape[-1] if max_pages_per_seq is None else max_pages_per_seq
    nf = free_pages.numel() if num_free is None else num_free
    st = lib.kva_extend_page_tables(
        _ptr(page_table), width, _ptr(cache_lengths), _ptr(input_row_offsets), B, tot_seq_len,
        page_size, num_pages, _ptr(free_pages), nf, _ptr(taken), _ptr(taken_out), _ptr(slot_map),
        _ptr(err_flags), _stream(stream))
    return _done(st, "kva_extend_page_tables", check)
