"""What the Python bindings take as a device address, and what they refuse before
the library sees it (no device needed)."""
import ctypes

import numpy as np
import pytest
import torch

from gqa_kv_cache_mla_gb300 import kva, kvw


def test_device_addresses():
    t = torch.zeros(4)
    assert kvw._ptr(t) == t.data_ptr() and kvw._ptr(None) is None
    assert kvw._ptr(0x10000) == 0x10000 and kvw._ptr(0) == 0


# ctypes would pass the first three on as addresses of host memory
@pytest.mark.parametrize("other", [b"bytes", "text", (ctypes.c_uint32 * 4)(),
                                   bytearray(8), [1, 2], (), 1.0, np.zeros(4), np.int64(16)],
                         ids=lambda x: type(x).__name__)
def test_nothing_else_is_a_device_address(other):
    with pytest.raises((AttributeError, TypeError)):
        kvw._ptr(other)
    offsets = torch.zeros(2, dtype=torch.int32)
    cache = kvw.paged_cache(0x10000, kva.DTYPE_INT4, 0x10000, 0x10000, 1, 1, 16, 1, 64,
                            (2048, 1024, 1024, 64, 1024), max_pages_per_seq=1)
    scales = kva.group_scales(0x10000, (64, 32, 32, 32))
    with pytest.raises((AttributeError, TypeError)):
        kva.kva_gqa_decode_int4(0x10000, 0x10000, offsets, cache, scales, 0, 1.0, other,
                                num_batches=1, tot_seq_len=0, num_q_heads=1, q_row_stride=64,
                                workspace_bytes=1 << 30, stream=0)
    with pytest.raises((AttributeError, TypeError)):
        kvw.paged_cache(other, kva.DTYPE_INT4, 0x10000, 0x10000, 1, 1, 16, 1, 64,
                        (2048, 1024, 1024, 64, 1024), max_pages_per_seq=1)


# ------------------------------------------------------------------ a cache in 4 bits

def test_types_of_a_cache_in_4_bits():
    codes = torch.zeros(5, 2, 3, 4, 32, 48, dtype=torch.uint8)
    scales = torch.zeros(5, 2, 3, 4, 2, 32, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 7, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    kva.int4_cache(codes, scales, table, lens)
    kva.int4_cache(codes, scales, table.view(torch.uint32), lens.data_ptr())
    for bad in (scales.half(), scales.view(torch.int16), scales.view(torch.uint16)):
        with pytest.raises(ValueError):  # their bits are not those of bf16 numbers
            kva.int4_cache(codes, bad, table, lens)
    for bad in (table.long(), table.short(), table.float()):
        with pytest.raises(ValueError):
            kva.int4_cache(codes, scales, bad, lens)
        with pytest.raises(ValueError):
            kva.int4_cache(codes, scales, table, bad[0])


# ------------------------------------------------------------------ page tables

NAMES = ["page_table", "cache_lengths", "input_row_offsets", "free_pages", "taken", "taken_out"]


def tables(**kw):
    """A call of no tokens, which launches nothing."""
    a = {n: torch.zeros(2, dtype=torch.int32) for n in NAMES}
    a["page_table"] = torch.zeros(1, 7, dtype=torch.int32)
    a.update(kw)
    return kva.kva_extend_page_tables(*[a[n] for n in NAMES], 16, 8, stream=0,
                                      slot_map=a.get("slot_map"), tot_seq_len=0, num_free=2,
                                      num_batches=1, max_pages_per_seq=7)


def test_page_tables_take_tensors_and_addresses():
    assert tables() == tables(slot_map=torch.zeros(0, dtype=torch.int64)) == kvw.KVW_OK
    assert tables(**{n: torch.zeros(2, 7, dtype=torch.uint32) for n in NAMES}) == kvw.KVW_OK
    assert tables(**{n: 0x10000 for n in NAMES}, slot_map=0x10000) == kvw.KVW_OK


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("dtype", [torch.int64, torch.int16, torch.uint8, torch.float32])
def test_page_tables_are_of_32_bits(name, dtype):
    """torch.arange gives 64-bit ids, of which every second word would be an id 0."""
    with pytest.raises(ValueError):
        tables(**{name: torch.zeros(2, 7, dtype=dtype)})


@pytest.mark.parametrize("dtype", [torch.int32, torch.float64])
def test_slots_are_of_64_bits(dtype):
    """A narrower buffer would be written past its end."""
    with pytest.raises(ValueError):
        tables(slot_map=torch.zeros(4, dtype=dtype))


# ------------------------------------------------------------------ rows of such a cache

@pytest.mark.parametrize("dtype", [torch.uint8, torch.float8_e4m3fn, torch.float32])
def test_rows_are_of_16_bits(dtype):
    """A narrower buffer would be written past its end.  (With no requests the
    library refuses the call before it launches anything.)"""
    cache = kvw.paged_cache(0x10000, kva.DTYPE_INT4, 0x10000, 0x10000, 1, 1, 16, 1, 64,
                            (2048, 1024, 1024, 64, 1024), max_pages_per_seq=1)
    scales = kva.group_scales(0x10000, (64, 32, 32, 32))
    off, bad = torch.zeros(1, dtype=torch.int32), torch.zeros(3, 1, 64, dtype=dtype)
    good = bad.to(torch.bfloat16)
    for k, v in ((bad, None), (None, bad), (good, bad), (bad, good)):
        with pytest.raises(ValueError):
            kva.kva_gather_kv_int4(k, v, off, cache, scales, 0, stream=0)
    with pytest.raises(kvw.KvwError):
        kva.kva_gather_kv_int4(good, good, off, cache, scales, 0, stream=0)
