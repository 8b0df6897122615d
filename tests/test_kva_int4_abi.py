"""The calls on a cache held in 4 bits and on page tables: their refusals
(argument errors are found on the host before any CUDA call, so these run
without a device)."""
import ctypes

import pytest
import torch

from gqa_kv_cache_mla_gb300 import kva, kvw
from test_kva_abi import FAKE, ODD, ODD4, append, gqa, mla

INVAL, UNSUP, OK = kvw.KVW_EINVAL, kvw.KVW_EUNSUPPORTED, kvw.KVW_OK
HEADS, HEAD, PAGE, LAYERS = 8, 128, 16, 2
ROWS = PAGE * HEAD  # codes of a head in a page
CODES = (2 * LAYERS * HEADS * ROWS, LAYERS * HEADS * ROWS, HEADS * ROWS, HEAD, ROWS)
SCALES = (2 * LAYERS * HEADS * 32, LAYERS * HEADS * 32, HEADS * 32, 32)


def cache(**kw):
    d = dict(data=FAKE, dtype=kva.DTYPE_INT4, page_table=FAKE, cache_lengths=FAKE, num_pages=8,
             num_layers=LAYERS, page_size=PAGE, num_heads=HEADS, head_size=HEAD, strides=CODES,
             max_pages_per_seq=4, scale=float("nan"))  # the scale is not used
    d.update(kw)
    return kvw.paged_cache(**d)


def group_scales(data=FAKE, strides=SCALES):
    return kva.group_scales(data, strides)


def swapped(strides, at, value):
    return strides[:at] + (value,) + strides[at + 1:]


# (cache arguments, scales arguments, status), of every call on such a cache
FAULTS = [
    ({"data": None}, {}, INVAL), ({"data": ODD}, {}, INVAL), ({}, {"data": None}, INVAL),
    ({}, {"data": ODD}, INVAL), ({"page_table": None}, {}, INVAL),
    ({"page_table": ODD4}, {}, INVAL), ({"cache_lengths": None}, {}, INVAL),
    ({"cache_lengths": ODD4}, {}, INVAL), ({"dtype": kvw.DTYPE_BF16}, {}, UNSUP),
    ({"dtype": kvw.DTYPE_FP8_E4M3}, {}, UNSUP), ({"dtype": kvw.DTYPE_F32}, {}, UNSUP),
    ({"num_pages": 0}, {}, INVAL), ({"page_size": 0}, {}, INVAL), ({"num_layers": 1}, {}, INVAL),
    ({"max_pages_per_seq": 0}, {}, INVAL), ({"num_heads": 0}, {}, INVAL),
    ({"head_size": 0}, {}, INVAL), ({"page_size": 8}, {}, UNSUP), ({"page_size": 24}, {}, UNSUP),
    ({"strides": swapped(CODES, 3, HEAD + 32)}, {}, INVAL),
    ({"strides": swapped(CODES, 3, 0)}, {}, INVAL),
] + [({"head_size": d, "strides": swapped(CODES, 3, d)}, {}, UNSUP)
     for d in (16, 32, 80, 112, 160, 192, 512)] + [
    ({"strides": swapped(CODES, at, CODES[at] + 16)}, {}, INVAL) for at in (0, 1, 2, 4)] + [
    ({}, {"strides": swapped(SCALES, at, SCALES[at] + 4)}, INVAL) for at in range(4)]


def append4(c, s, **kw):
    a = dict(q_out=FAKE + 16, qs=4096, qkv=FAKE, qkvs=6144, off=FAKE, B=2, T=0, Hq=32, gq=FAKE,
             gk=FAKE, eps=1e-6, wo=0.0, freqs=FAKE, rows=64, rope=128, pos=None, il=0, sec=None,
             layer=1, err=None)
    a.update(kw)
    sec = a["sec"]
    if sec is not None:
        sec = ctypes.cast((ctypes.c_uint32 * 3)(*sec), ctypes.c_void_p)
    return kva.lib.kva_append_qkv_int4(
        a["q_out"], a["qs"], a["qkv"], a["qkvs"], a["off"], a["B"], a["T"], a["Hq"], a["gq"],
        a["gk"], a["eps"], a["wo"], a["freqs"], a["rows"], a["rope"], a["pos"], a["il"], sec,
        None if c is None else ctypes.byref(c), None if s is None else ctypes.byref(s), a["layer"],
        a["err"], 0)


def gather4(c, s, **kw):
    a = dict(k=FAKE, v=FAKE, stride=HEADS * HEAD, off=FAKE, first=None, B=2, rows=0, layer=1,
             err=None)
    a.update(kw)
    return kva.lib.kva_gather_kv_int4(
        a["k"], a["v"], a["stride"], None if c is None else ctypes.byref(c),
        None if s is None else ctypes.byref(s), a["layer"], a["off"], a["first"], a["B"], a["rows"],
        a["err"], 0)


def gqa4(c, s, **kw):
    a = dict(out=FAKE, lse=None, q=FAKE, qs=4096, off=FAKE, B=2, T=0, Hq=32, layer=1, scale=0.1,
             cap=0.0, window=0, slopes=None, ws=FAKE, nbytes=1 << 30, err=None)
    a.update(kw)
    return kva.lib.kva_gqa_decode_int4(
        a["out"], a["lse"], a["q"], a["qs"], a["off"], a["B"], a["T"], a["Hq"],
        None if c is None else ctypes.byref(c), None if s is None else ctypes.byref(s), a["layer"],
        a["scale"], a["cap"], a["window"], a["slopes"], a["ws"], a["nbytes"], a["err"], 0)


CALLS = [append4, gather4, gqa4]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("cache_kw,scales_kw,want", FAULTS)
def test_cache_refusals(call, cache_kw, scales_kw, want):
    assert call(cache(**cache_kw), group_scales(**scales_kw)) == want


@pytest.mark.parametrize("call", CALLS)
def test_both_descriptors_are_needed(call):
    assert call(cache(), group_scales()) == OK
    assert call(None, group_scales()) == INVAL and call(cache(), None) == INVAL
    assert call(cache(), group_scales(), layer=2) == INVAL


@pytest.mark.parametrize("call", CALLS)
def test_a_dimension_of_one_index_needs_no_stride(call):
    for at, name, scales_at in ((0, "num_pages", 0), (2, "num_layers", 2), (4, "num_heads", 3)):
        kw = {name: 1, "strides": swapped(CODES, at, 7)}
        layer = {"layer": 0} if name == "num_layers" else {}
        if call is append4 and name == "num_heads":
            layer["Hq"] = 32
        s = group_scales(strides=swapped(SCALES, scales_at, 3))
        assert call(cache(**kw), s, **layer) == OK


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("call", CALLS)
def test_head_sizes(call, head):
    kw = {gqa4: {"qs": 32 * head}, append4: {"qs": 32 * head, "qkvs": 48 * head, "rope": 64},
          gather4: {"stride": HEADS * head}}[call]
    rows = PAGE * head
    st = (2 * LAYERS * HEADS * rows, LAYERS * HEADS * rows, HEADS * rows, head, rows)
    assert call(cache(head_size=head, strides=st), group_scales(strides=(8 * x for x in SCALES)),
                **kw) == OK


@pytest.mark.parametrize("call_kw,want", [
    ({}, OK), ({"Hq": 0, "q_out": None, "qs": 0}, OK), ({"rope": 0, "freqs": None, "rows": 0}, OK),
    ({"q_out": FAKE, "qs": 6144}, OK),  # in place
    ({"pos": FAKE, "sec": (16, 24, 24)}, OK), ({"q_out": None}, INVAL), ({"q_out": ODD}, INVAL),
    ({"qkv": None}, INVAL), ({"qkv": ODD}, INVAL), ({"q_out": FAKE, "qs": 4104}, INVAL),
    ({"off": None}, INVAL), ({"off": ODD4}, INVAL), ({"B": 0}, INVAL), ({"B": 8193}, UNSUP),
    ({"qkvs": 6136}, INVAL), ({"qkvs": 6148}, INVAL), ({"qs": 4088}, INVAL), ({"qs": 4100}, INVAL),
    ({"gq": ODD}, INVAL), ({"gk": ODD}, INVAL), ({"freqs": ODD}, INVAL), ({"freqs": None}, INVAL),
    ({"rows": 0}, INVAL), ({"rope": 120}, INVAL), ({"rope": 144}, INVAL), ({"eps": -1.0}, INVAL),
    ({"eps": float("nan")}, INVAL), ({"wo": float("inf")}, INVAL), ({"sec": (16, 24, 24)}, INVAL),
    ({"pos": FAKE, "sec": (16, 24, 23)}, INVAL), ({"pos": ODD4}, INVAL), ({"err": ODD4}, INVAL),
    ({"Hq": 4090, "qs": 1 << 20, "qkvs": 1 << 20}, UNSUP), ({"T": 1 << 28}, UNSUP),
])
def test_append_refusals(call_kw, want):
    assert append4(cache(), group_scales(), **call_kw) == want


@pytest.mark.parametrize("call_kw,want", [
    ({}, OK), ({"k": None}, OK), ({"v": None}, OK), ({"first": FAKE}, OK),
    ({"stride": HEADS * HEAD + 8}, OK), ({"k": None, "v": None}, INVAL), ({"k": ODD}, INVAL),
    ({"v": ODD}, INVAL), ({"stride": HEADS * HEAD - 8}, INVAL),
    ({"stride": HEADS * HEAD + 4}, INVAL), ({"off": None}, INVAL), ({"off": ODD4}, INVAL),
    ({"first": ODD4}, INVAL), ({"err": ODD4}, INVAL), ({"B": 0}, INVAL), ({"B": 8193}, UNSUP),
    ({"rows": (1 << 31) + 1}, UNSUP),
])
def test_gather_refusals(call_kw, want):
    assert gather4(cache(), group_scales(), **call_kw) == want


def test_gather_most_heads():
    st = tuple(512 * x if i < 3 else x for i, x in enumerate(CODES))
    for heads, want in ((2048, OK), (2049, UNSUP)):
        assert gather4(cache(num_heads=heads, strides=st), group_scales(),
                       stride=heads * HEAD) == want


@pytest.mark.parametrize("call_kw,want", [
    ({}, OK), ({"lse": FAKE, "slopes": FAKE, "window": 7, "cap": 2.0}, OK), ({"out": None}, INVAL),
    ({"out": ODD}, INVAL), ({"q": None}, INVAL), ({"q": ODD}, INVAL), ({"lse": ODD4}, INVAL),
    ({"slopes": ODD4}, INVAL), ({"off": None}, INVAL), ({"err": ODD4}, INVAL),
    ({"qs": 4088}, INVAL), ({"qs": 4100}, INVAL), ({"B": 0}, INVAL), ({"B": 8193}, UNSUP),
    ({"T": (1 << 20) + 1}, UNSUP), ({"Hq": 0}, INVAL), ({"Hq": 33, "qs": 8192}, INVAL),
    ({"Hq": 4104, "qs": 1 << 20}, UNSUP), ({"scale": 0.0}, INVAL), ({"scale": float("nan")}, INVAL),
    ({"scale": float("inf")}, INVAL), ({"cap": -1.0}, INVAL), ({"cap": float("nan")}, INVAL),
    ({"cap": float("inf")}, INVAL), ({"ws": None}, INVAL), ({"ws": ODD}, INVAL),
    ({"nbytes": 1000}, INVAL),
])
def test_gqa_refusals(call_kw, want):
    assert gqa4(cache(), group_scales(), **call_kw) == want


def test_gqa_workspace_is_exact():
    n = kva.kva_gqa_decode_workspace(32, HEADS, HEAD)
    assert gqa4(cache(), group_scales(), nbytes=n) == OK
    assert gqa4(cache(), group_scales(), nbytes=n - 1) == INVAL


# a copy of the cache walks pages, planes and heads with positive strides below
# 2^40 bytes: 2^41 codes, 2^39 scales
@pytest.mark.parametrize("at,value,want", [
    (0, -65536, INVAL), (0, 0, INVAL), (0, 1 << 41, INVAL), (0, (1 << 41) - 32, OK),
    (1, -65536, INVAL), (1, 0, INVAL), (1, 1 << 41, INVAL), (4, -2048, INVAL), (4, 0, INVAL),
    (4, 1 << 41, INVAL), (2, -65536, OK), (2, 0, OK), (2, 1 << 45, OK)])
def test_gqa_strides_of_codes(at, value, want):
    assert gqa4(cache(strides=swapped(CODES, at, value)), group_scales()) == want


@pytest.mark.parametrize("at,value,want", [
    (0, -64, INVAL), (0, 0, INVAL), (0, 1 << 39, INVAL), (0, (1 << 39) - 8, OK), (1, -64, INVAL),
    (1, 0, INVAL), (1, 1 << 39, INVAL), (3, -64, INVAL), (3, 0, INVAL), (3, 1 << 39, INVAL),
    (2, -64, OK), (2, 0, OK)])
def test_gqa_strides_of_scales(at, value, want):
    assert gqa4(cache(), group_scales(strides=swapped(SCALES, at, value))) == want


@pytest.mark.parametrize("name", ["num_pages", "page_size"])
def test_most_pages_and_rows(name):
    for count, want in ((1 << 31, OK), ((1 << 31) + 16, UNSUP)):
        assert gqa4(cache(**{name: count}), group_scales()) == want
        assert append4(cache(**{name: count}), group_scales()) == OK


def test_the_other_calls_refuse_it():
    c = cache(strides=(65536, 32768, 16384, 1024, 128))
    assert append(c, q_out=FAKE + 16) == UNSUP
    assert gqa(c) == UNSUP
    assert mla(cache(num_heads=1, head_size=576, strides=(2 * 16 * 576, 0, 16 * 576, 576, 576))) \
        == UNSUP


def tables(**kw):
    a = dict(table=FAKE, width=4, lens=FAKE, off=FAKE, B=2, T=0, page=16, pages=8, free=FAKE, nf=4,
             taken=FAKE, out=FAKE, slots=FAKE, err=None)
    a.update(kw)
    return kva.lib.kva_extend_page_tables(
        a["table"], a["width"], a["lens"], a["off"], a["B"], a["T"], a["page"], a["pages"],
        a["free"], a["nf"], a["taken"], a["out"], a["slots"], a["err"], 0)


@pytest.mark.parametrize("call_kw,want", [
    ({}, OK), ({"slots": None}, OK), ({"free": None, "nf": 0}, OK), ({"table": None}, INVAL),
    ({"table": ODD4}, INVAL), ({"width": 0}, INVAL), ({"lens": None}, INVAL),
    ({"lens": ODD4}, INVAL), ({"off": None}, INVAL), ({"off": ODD4}, INVAL), ({"B": 0}, INVAL),
    ({"B": 8193}, UNSUP), ({"T": (1 << 31) + 1}, UNSUP), ({"page": 0}, INVAL),
    ({"pages": 0}, INVAL), ({"free": None}, INVAL), ({"free": ODD4}, INVAL),
    ({"taken": None}, INVAL), ({"taken": ODD4}, INVAL), ({"out": None}, INVAL),
    ({"out": ODD4}, INVAL), ({"slots": FAKE + 4}, INVAL), ({"err": ODD4}, INVAL),
])
def test_tables_refusals(call_kw, want):
    assert tables(**call_kw) == want


def test_descriptors_of_dense_tensors():
    codes = torch.zeros(5, 2, 3, 4, 32, 48, dtype=torch.uint8)
    scales = torch.zeros(5, 2, 3, 4, 2, 32, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 7, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    c, s = kva.int4_cache(codes, scales, table, lens)
    assert (c.dtype, c.num_pages, c.num_layers, c.page_size, c.num_heads, c.head_size,
            c.max_pages_per_seq) == (3, 5, 3, 32, 4, 96, 7)
    row = 32 * 96
    assert (c.stride_page, c.stride_kv, c.stride_layer, c.stride_token, c.stride_head) == \
        (24 * row, 12 * row, 4 * row, 96, row)
    assert (s.stride_page, s.stride_kv, s.stride_layer, s.stride_head) == (1536, 768, 256, 64)
    for bad in (codes[..., :40], codes.transpose(3, 4), codes[:, :, :2], codes[:, :1],
                codes.short()):
        with pytest.raises(ValueError):
            kva.int4_cache(bad, scales, table, lens)
    with pytest.raises(ValueError):
        kva.int4_cache(codes, scales[..., :1, :], table, lens)
    with pytest.raises(ValueError):
        kva.int4_cache(codes, scales.float(), table, lens)


def test_wrapper_checks():
    one, two = torch.zeros(3, 2, 8), torch.zeros(3, 2, 16)
    with pytest.raises(ValueError):
        kva.kva_gather_kv_int4(one, two, torch.zeros(2), cache(), group_scales(), 0)
    with pytest.raises(ValueError):
        kva.kva_extend_page_tables(one, one, torch.zeros(2), one, one, one, 16, 8)
    with pytest.raises(kvw.KvwError):
        kva.kva_gather_kv_int4(None, None, torch.zeros(2), cache(), group_scales(), 0, stream=0)
