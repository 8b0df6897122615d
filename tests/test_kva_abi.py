"""include/kva.h: exported, bound, usable from C, and its refusals (argument
errors are found on the host before any CUDA call, so these run without a
device)."""
import ctypes
import os
import re
import shutil
import subprocess

import pytest

from gqa_kv_cache_mla_gb300 import kva, kvw

FAKE, ODD, ODD4 = 0x10000, 0x10008, 0x10002


def test_exports_every_header_function():
    names = kva.header_functions()
    out = subprocess.run(["nm", "-D", "--defined-only", kvw.LIB_PATH], capture_output=True,
                         text=True).stdout
    assert set(re.findall(r"\bT (kva_\w+)", out)) == set(names) and names
    for n in names:
        assert hasattr(kva.lib, n) and hasattr(kva, n)


def test_header_compiles_as_c(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    src = tmp_path / "use.c"
    src.write_text('#include "kva.h"\nint main(void) { uint64_t n = 0;\n'
                   '  return kva_gqa_decode_workspace(32, 8, 128, &n) != KVW_OK || n == 0 ||\n'
                   '         kva_mla_decode_workspace(128, &n) != KVW_OK; }\n')
    exe, where = str(tmp_path / "use"), os.path.dirname(kvw.LIB_PATH)
    subprocess.run([nvcc, str(src), "-I", os.path.dirname(kva.HEADER), "-L", where, "-lkvw",
                    "-Xlinker", "-rpath=" + where, "-o", exe], check=True, capture_output=True)
    assert subprocess.run([exe]).returncode == 0


def cache(**kw):
    d = dict(data=FAKE, dtype=kvw.DTYPE_BF16, page_table=FAKE, cache_lengths=FAKE, num_pages=8,
             num_layers=2, page_size=16, num_heads=8, head_size=128,
             strides=(2 * 2 * 16 * 8 * 128, 2 * 16 * 8 * 128, 16 * 8 * 128, 8 * 128, 128),
             max_pages_per_seq=4)
    d.update(kw)
    return kvw.paged_cache(**d)


CACHE_FAULTS = [
    ({"data": None}, kvw.KVW_EINVAL), ({"data": ODD}, kvw.KVW_EINVAL),
    ({"page_table": None}, kvw.KVW_EINVAL), ({"cache_lengths": None}, kvw.KVW_EINVAL),
    ({"page_table": ODD4}, kvw.KVW_EINVAL), ({"cache_lengths": ODD4}, kvw.KVW_EINVAL),
    ({"dtype": kvw.DTYPE_F32}, kvw.KVW_EUNSUPPORTED), ({"dtype": 7}, kvw.KVW_EUNSUPPORTED),
    ({"num_pages": 0}, kvw.KVW_EINVAL), ({"page_size": 0}, kvw.KVW_EINVAL),
    ({"num_layers": 1}, kvw.KVW_EINVAL),  # layer 1 of one
    ({"max_pages_per_seq": 0}, kvw.KVW_EINVAL),
    ({"dtype": kvw.DTYPE_FP8_E4M3, "scale": 0.0}, kvw.KVW_EINVAL),
    ({"dtype": kvw.DTYPE_FP8_E4M3, "scale": float("nan")}, kvw.KVW_EINVAL),
    ({"dtype": kvw.DTYPE_FP8_E4M3, "scale": float("inf")}, kvw.KVW_EINVAL),
]
GQA_CACHE_FAULTS = CACHE_FAULTS + [
    ({"num_heads": 0}, kvw.KVW_EINVAL), ({"head_size": 0}, kvw.KVW_EINVAL),
    ({"head_size": 72}, kvw.KVW_EUNSUPPORTED),
    ({"strides": (65536, 32768, 16384, 1020, 128)}, kvw.KVW_EINVAL),
    ({"strides": (65536, 32768, 16384, 1024, 132)}, kvw.KVW_EINVAL),
    ({"strides": (65536, 32764, 16384, 1024, 128)}, kvw.KVW_EINVAL),
    ({"strides": (65532, 32768, 16384, 1024, 128)}, kvw.KVW_EINVAL),
    ({"strides": (65536, 32768, 16380, 1024, 128)}, kvw.KVW_EINVAL),
    ({"dtype": kvw.DTYPE_FP8_E4M3, "strides": (65536, 32768, 16384, 1024, 136)}, kvw.KVW_EINVAL),
]


def append(c, **kw):
    a = dict(q_out=FAKE, qs=4096, qkv=FAKE, qkvs=6144, off=FAKE, B=2, T=0, Hq=32, gq=FAKE, gk=FAKE,
             eps=1e-6, wo=0.0, freqs=FAKE, rows=64, rope=128, pos=None, il=0, sec=None, vs=1.0,
             layer=1, err=None)
    a.update(kw)
    sec = a["sec"]
    if sec is not None:
        sec = ctypes.cast((ctypes.c_uint32 * 3)(*sec), ctypes.c_void_p)
    return kva.lib.kva_append_qkv_paged(
        a["q_out"], a["qs"], a["qkv"], a["qkvs"], a["off"], a["B"], a["T"], a["Hq"], a["gq"],
        a["gk"], a["eps"], a["wo"], a["freqs"], a["rows"], a["rope"], a["pos"], a["il"], sec,
        None if c is None else ctypes.byref(c), a["vs"], a["layer"], a["err"], 0)


@pytest.mark.parametrize("call_kw,want", [
    ({}, kvw.KVW_OK),  # no tokens: nothing is launched
    ({"Hq": 0, "q_out": None, "qs": 0}, kvw.KVW_OK),
    ({"rope": 0, "freqs": None, "rows": 0}, kvw.KVW_OK),
    ({"q_out": FAKE, "qs": 6144}, kvw.KVW_OK),  # in place
    ({"pos": FAKE, "sec": (16, 24, 24)}, kvw.KVW_OK),
    ({"q_out": None}, kvw.KVW_EINVAL), ({"q_out": ODD}, kvw.KVW_EINVAL),
    ({"qkv": None}, kvw.KVW_EINVAL), ({"qkv": ODD}, kvw.KVW_EINVAL),
    ({"qkv": FAKE, "q_out": FAKE, "qs": 4104}, kvw.KVW_EINVAL),  # in place, other stride
    ({"off": None}, kvw.KVW_EINVAL), ({"off": ODD4}, kvw.KVW_EINVAL),
    ({"B": 0}, kvw.KVW_EINVAL), ({"B": 8193}, kvw.KVW_EUNSUPPORTED),
    ({"qkvs": 6136}, kvw.KVW_EINVAL), ({"qkvs": 6148}, kvw.KVW_EINVAL),
    ({"q_out": FAKE + 16, "qs": 4088}, kvw.KVW_EINVAL),
    ({"q_out": FAKE + 16, "qs": 4100}, kvw.KVW_EINVAL),
    ({"gq": ODD}, kvw.KVW_EINVAL), ({"gk": ODD}, kvw.KVW_EINVAL),
    ({"freqs": ODD}, kvw.KVW_EINVAL), ({"freqs": None}, kvw.KVW_EINVAL),
    ({"rows": 0}, kvw.KVW_EINVAL), ({"rope": 120}, kvw.KVW_EINVAL),
    ({"rope": 144}, kvw.KVW_EINVAL), ({"eps": -1.0}, kvw.KVW_EINVAL),
    ({"eps": float("nan")}, kvw.KVW_EINVAL), ({"wo": float("inf")}, kvw.KVW_EINVAL),
    ({"sec": (16, 24, 24)}, kvw.KVW_EINVAL),  # no position ids
    ({"pos": FAKE, "sec": (16, 24, 23)}, kvw.KVW_EINVAL),
    ({"pos": FAKE, "sec": (64, 1, 2 ** 32 - 1)}, kvw.KVW_EINVAL),  # the sum wraps in 32 bits
    ({"pos": ODD4}, kvw.KVW_EINVAL), ({"err": ODD4}, kvw.KVW_EINVAL),
    ({"Hq": 4090, "qs": 1 << 20, "qkvs": 1 << 20}, kvw.KVW_EUNSUPPORTED),
    ({"T": 1 << 28}, kvw.KVW_EUNSUPPORTED), ({"layer": 2}, kvw.KVW_EINVAL),
])
def test_append_refusals(call_kw, want):
    if call_kw == {} or "qs" not in call_kw and "q_out" not in call_kw:
        call_kw = {"q_out": FAKE + 16, **call_kw}
    assert append(cache(), **call_kw) == want


@pytest.mark.parametrize("cache_kw,want", GQA_CACHE_FAULTS + [
    ({"head_size": 528}, kvw.KVW_EUNSUPPORTED)])
def test_append_cache_refusals(cache_kw, want):
    assert append(cache(**cache_kw), q_out=FAKE + 16, qs=1 << 20, qkvs=1 << 20) == want


def test_append_value_scale():
    fp8 = cache(dtype=kvw.DTYPE_FP8_E4M3)
    for vs in (0.0, -1.0, float("nan"), float("inf")):
        assert append(fp8, q_out=FAKE + 16, vs=vs) == kvw.KVW_EINVAL
        assert append(cache(), q_out=FAKE + 16, vs=vs) == kvw.KVW_OK  # bf16 ignores it
    assert append(None, q_out=FAKE + 16) == kvw.KVW_EINVAL


def gqa(c, **kw):
    a = dict(out=FAKE, lse=None, q=FAKE, qs=4096, off=FAKE, B=2, T=0, Hq=32, vs=1.0, layer=1,
             scale=0.1, cap=0.0, window=0, slopes=None, ws=FAKE, nbytes=1 << 30, err=None)
    a.update(kw)
    return kva.lib.kva_gqa_decode_paged(
        a["out"], a["lse"], a["q"], a["qs"], a["off"], a["B"], a["T"], a["Hq"],
        None if c is None else ctypes.byref(c), a["vs"], a["layer"], a["scale"], a["cap"],
        a["window"], a["slopes"], a["ws"], a["nbytes"], a["err"], 0)


@pytest.mark.parametrize("call_kw,want", [
    ({}, kvw.KVW_OK), ({"lse": FAKE, "slopes": FAKE, "window": 7, "cap": 2.0}, kvw.KVW_OK),
    ({"out": None}, kvw.KVW_EINVAL), ({"out": ODD}, kvw.KVW_EINVAL),
    ({"q": None}, kvw.KVW_EINVAL), ({"q": ODD}, kvw.KVW_EINVAL),
    ({"lse": ODD4}, kvw.KVW_EINVAL), ({"slopes": ODD4}, kvw.KVW_EINVAL),
    ({"off": None}, kvw.KVW_EINVAL), ({"err": ODD4}, kvw.KVW_EINVAL),
    ({"qs": 4088}, kvw.KVW_EINVAL), ({"qs": 4100}, kvw.KVW_EINVAL),
    ({"B": 0}, kvw.KVW_EINVAL), ({"B": 8193}, kvw.KVW_EUNSUPPORTED),
    ({"T": (1 << 20) + 1}, kvw.KVW_EUNSUPPORTED),
    ({"Hq": 0}, kvw.KVW_EINVAL), ({"Hq": 33, "qs": 8192}, kvw.KVW_EINVAL),
    ({"Hq": 4104, "qs": 1 << 20}, kvw.KVW_EUNSUPPORTED),
    ({"scale": 0.0}, kvw.KVW_EINVAL), ({"scale": float("nan")}, kvw.KVW_EINVAL),
    ({"scale": float("inf")}, kvw.KVW_EINVAL), ({"cap": -1.0}, kvw.KVW_EINVAL),
    ({"cap": float("nan")}, kvw.KVW_EINVAL), ({"cap": float("inf")}, kvw.KVW_EINVAL),
    ({"ws": None}, kvw.KVW_EINVAL), ({"ws": ODD}, kvw.KVW_EINVAL),
    ({"nbytes": 1000}, kvw.KVW_EINVAL), ({"layer": 2}, kvw.KVW_EINVAL),
])
def test_gqa_refusals(call_kw, want):
    assert gqa(cache(), **call_kw) == want


@pytest.mark.parametrize("cache_kw,want", GQA_CACHE_FAULTS + [
    ({"head_size": 272}, kvw.KVW_EUNSUPPORTED)])
def test_gqa_cache_refusals(cache_kw, want):
    assert gqa(cache(**cache_kw), qs=1 << 20) == want


def test_gqa_workspace_is_exact():
    n = kva.kva_gqa_decode_workspace(32, 8, 128)
    assert gqa(cache(), nbytes=n) == kvw.KVW_OK and gqa(cache(), nbytes=n - 1) == kvw.KVW_EINVAL
    assert kva.lib.kva_gqa_decode_workspace(32, 8, 128, None) == kvw.KVW_EINVAL
    for args in ((32, 0, 128), (0, 8, 128), (30, 8, 128), (32, 8, 0), (32, 8, 40), (32, 8, 272)):
        with pytest.raises(kvw.KvwError):
            kva.kva_gqa_decode_workspace(*args)
    assert gqa(None) == kvw.KVW_EINVAL
    assert gqa(cache(dtype=kvw.DTYPE_FP8_E4M3), vs=0.0) == kvw.KVW_EINVAL


def mla_cache(**kw):
    d = dict(num_heads=1, head_size=576, strides=(2 * 16 * 576, 0, 16 * 576, 576, 576))
    d.update(kw)
    return cache(**d)


def mla(c, **kw):
    a = dict(out=FAKE, lse=None, ql=FAKE, qls=16 * 512, qr=FAKE, qrs=16 * 64, off=FAKE, B=2, T=0,
             H=16, layer=1, scale=0.1, ws=FAKE, nbytes=1 << 30, err=None)
    a.update(kw)
    return kva.lib.kva_mla_decode_paged(
        a["out"], a["lse"], a["ql"], a["qls"], a["qr"], a["qrs"], a["off"], a["B"], a["T"], a["H"],
        None if c is None else ctypes.byref(c), a["layer"], a["scale"], a["ws"], a["nbytes"],
        a["err"], 0)


@pytest.mark.parametrize("call_kw,want", [
    ({}, kvw.KVW_OK), ({"lse": FAKE}, kvw.KVW_OK), ({"qls": 16 * 512 + 8, "qrs": 4096}, kvw.KVW_OK),
    ({"out": None}, kvw.KVW_EINVAL), ({"out": ODD}, kvw.KVW_EINVAL),
    ({"ql": None}, kvw.KVW_EINVAL), ({"ql": ODD}, kvw.KVW_EINVAL),
    ({"qr": None}, kvw.KVW_EINVAL), ({"qr": ODD}, kvw.KVW_EINVAL),
    ({"lse": ODD4}, kvw.KVW_EINVAL), ({"off": None}, kvw.KVW_EINVAL),
    ({"err": ODD4}, kvw.KVW_EINVAL), ({"qls": 16 * 512 - 8}, kvw.KVW_EINVAL),
    ({"qls": 16 * 512 + 4}, kvw.KVW_EINVAL), ({"qrs": 16 * 64 - 8}, kvw.KVW_EINVAL),
    ({"qrs": 16 * 64 + 4}, kvw.KVW_EINVAL), ({"qls": 1 << 39}, kvw.KVW_EINVAL),
    ({"B": 0}, kvw.KVW_EINVAL), ({"B": 8193}, kvw.KVW_EUNSUPPORTED),
    ({"T": (1 << 20) + 1}, kvw.KVW_EUNSUPPORTED), ({"H": 0}, kvw.KVW_EINVAL),
    ({"H": 1025, "qls": 1 << 20, "qrs": 1 << 20}, kvw.KVW_EUNSUPPORTED),
    ({"scale": 0.0}, kvw.KVW_EINVAL), ({"scale": float("nan")}, kvw.KVW_EINVAL),
    ({"ws": None}, kvw.KVW_EINVAL), ({"ws": ODD}, kvw.KVW_EINVAL),
    ({"nbytes": 1000}, kvw.KVW_EINVAL), ({"layer": 2}, kvw.KVW_EINVAL),
])
def test_mla_refusals(call_kw, want):
    assert mla(mla_cache(), **call_kw) == want


@pytest.mark.parametrize("cache_kw,want", CACHE_FAULTS + [
    ({"num_heads": 2}, kvw.KVW_EUNSUPPORTED), ({"head_size": 512}, kvw.KVW_EUNSUPPORTED),
    ({"strides": (2 * 16 * 576, 0, 16 * 576, 580, 576)}, kvw.KVW_EINVAL),
    ({"strides": (2 * 16 * 576, 0, 16 * 576, -576, 576)}, kvw.KVW_EINVAL),
    ({"strides": (1 << 39, 0, 16 * 576, 576, 576)}, kvw.KVW_EINVAL),
])
def test_mla_cache_refusals(cache_kw, want):
    assert mla(mla_cache(**cache_kw)) == want


def test_mla_workspace_is_exact():
    for heads in (1, 16, 128):
        n = kva.kva_mla_decode_workspace(heads)
        kw = dict(H=heads, qls=heads * 512, qrs=heads * 64)
        assert n % 16 == 0
        assert mla(mla_cache(), nbytes=n, **kw) == kvw.KVW_OK
        assert mla(mla_cache(), nbytes=n - 1, **kw) == kvw.KVW_EINVAL
    assert kva.kva_mla_decode_workspace(64) == kva.kva_mla_decode_workspace(1024)
    for heads in (0, 1025):
        with pytest.raises(kvw.KvwError):
            kva.kva_mla_decode_workspace(heads)
    assert mla(None) == kvw.KVW_EINVAL


# (page, kv, layer, token, head): a copy of the cache walks page, plane, token
# and head with positive strides below 2^40 bytes; one index needs no stride
@pytest.mark.parametrize("at,stride,want", [
    (0, -65536, kvw.KVW_EINVAL), (0, 0, kvw.KVW_EINVAL), (0, 1 << 39, kvw.KVW_EINVAL),
    (1, -32768, kvw.KVW_EINVAL), (1, 0, kvw.KVW_EINVAL), (1, 1 << 39, kvw.KVW_EINVAL),
    (3, -1024, kvw.KVW_EINVAL), (3, 0, kvw.KVW_EINVAL), (3, 1 << 39, kvw.KVW_EINVAL),
    (4, -128, kvw.KVW_EINVAL), (4, 0, kvw.KVW_EINVAL), (4, 1 << 39, kvw.KVW_EINVAL),
    (2, -16384, kvw.KVW_OK), (2, 0, kvw.KVW_OK), (2, 1 << 45, kvw.KVW_OK),
    (0, (1 << 39) - 8, kvw.KVW_OK),
])
def test_gqa_strides(at, stride, want):
    strides = [65536, 32768, 16384, 1024, 128]
    strides[at] = stride
    assert gqa(cache(strides=tuple(strides))) == want
    one = {0: "num_pages", 4: "num_heads"}.get(at)
    if one and stride % 8 == 0:
        assert gqa(cache(strides=tuple(strides), **{one: 1})) == kvw.KVW_OK


def test_query_strides():
    top = 1 << 39  # bytes of a row stride of the latent queries stay below 2^40
    assert mla(mla_cache(), qls=top - 8, qrs=top - 8) == kvw.KVW_OK
    assert mla(mla_cache(), qls=top - 8, qrs=top) == kvw.KVW_EINVAL
    assert gqa(cache(), qs=1 << 45) == kvw.KVW_OK


# the copies' coordinates are signed 32-bit
@pytest.mark.parametrize("name", ["num_pages", "page_size"])
def test_most_pages_and_rows(name):
    for count, want in ((1 << 31, kvw.KVW_OK), ((1 << 31) + 1, kvw.KVW_EUNSUPPORTED),
                        (2 ** 32 - 1, kvw.KVW_EUNSUPPORTED)):
        assert gqa(cache(**{name: count})) == want
        assert mla(mla_cache(**{name: count})) == want
        assert append(cache(**{name: count}), q_out=FAKE + 16) == kvw.KVW_OK
