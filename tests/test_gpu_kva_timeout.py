"""A bounded device-side wait of the attention calls that runs out (GPU).

Every wait in the attention kernels is bounded; at its limit the kernel sets
KVW_ERR_TIMEOUT, gives up its work and returns.  As in the tests of the write
kernels, the sources are compiled a second time with -DKVW_TEST_HOOKS into a
library of this test's own, whose entry points announce the first copy of
every CTA on its barrier but never issue it, so that the wait for it can only
end at its limit (a few milliseconds here).  The call has to return, set the
flag, and leave the output and the cache as they were, and the product entry
point then has to match the 64-bit evaluation in the same context.
"""
import ctypes
import time

import pytest
import torch

import kva_reference as R
from test_gpu_timeout import KVW_ERR_TIMEOUT, WAIT_NS, _hook_library

pytestmark = pytest.mark.gpu

VP, U32, I64, U64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64, ctypes.c_uint64


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def hook(tmp_path_factory, source, name, args):
    f = getattr(_hook_library(tmp_path_factory, source), name)
    f.restype, f.argtypes = ctypes.c_int, args
    return f


@pytest.fixture(scope="module")
def gqa_hook(kva, tmp_path_factory):
    from gqa_kv_cache_mla_gb300 import kvw

    return hook(tmp_path_factory, "gqa_decode_paged.cu", "kva_test_gqa_decode_withheld",
                [VP, VP, I64, VP, U32, U32, U32, ctypes.POINTER(kvw.PagedCacheT), U32, VP, U64, VP,
                 VP, U64])


@pytest.fixture(scope="module")
def mla_hook(kva, tmp_path_factory):
    from gqa_kv_cache_mla_gb300 import kvw

    return hook(tmp_path_factory, "mla_decode_paged.cu", "kva_test_mla_decode_withheld",
                [VP, VP, I64, VP, I64, VP, U32, U32, U32, ctypes.POINTER(kvw.PagedCacheT), U32, VP,
                 U64, VP, VP, U64])


def runs_out(call, out, flags, store, c):
    before = out.clone()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert call(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(flags) & KVW_ERR_TIMEOUT
    assert torch.equal(out, before)
    assert torch.equal(store.cpu().view(torch.uint8), c.store.view(torch.uint8))
    flags.zero_()


# one long context, so that every piece has more tiles than its ring, and
# short ones, whose pieces have one
CONTEXTS = [1, 2, 0, 1, 1], [40000, 900, 3, 0, 64]


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [64, 12])
def test_gqa_withheld_copy(kva, gqa_hook, dtype, page):
    c = R.Paged(90, *CONTEXTS, kv_heads=2, head=128, dtype=dtype, page=page, layers=1,
                layer=0).fill()
    heads = 8
    desc, store, keep = c.on()
    q = c.normal(c.T, heads, 128)
    dq, out = q.cuda(), torch.full((c.T, heads, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_gqa_decode_workspace(heads, 2, 128),), 0xFF, dtype=torch.uint8,
                       device="cuda")
    runs_out(lambda stream: gqa_hook(out.data_ptr(), dq.data_ptr(), heads * 128,
                                     keep[3].data_ptr(), c.B, c.T, heads, ctypes.byref(desc), 0,
                                     space.data_ptr(), space.numel(), flags.data_ptr(), stream,
                                     WAIT_NS), out, flags, store, c)
    want, _, tol, _ = R.gqa(c, q, 0.1)
    kva.kva_gqa_decode_paged(out, dq, keep[3], desc, 0, 0.1, space, v_scale=c.v_scale,
                             err_flags=flags)
    assert int(flags) == 0
    R.check(out, want, tol)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("page", [64, 12])
def test_mla_withheld_copy(kva, mla_hook, dtype, heads, page):
    c = R.Paged(91, *CONTEXTS, kv_heads=1, head=576, planes=1, dtype=dtype, page=page, layers=1,
                layer=0).fill()
    desc, store, keep = c.on()
    q = c.normal(c.T, heads, 512), c.normal(c.T, heads, 64)
    dl, dr = q[0].cuda(), q[1].cuda()
    out = torch.full((c.T, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_mla_decode_workspace(heads),), 0xFF, dtype=torch.uint8,
                       device="cuda")
    runs_out(lambda stream: mla_hook(out.data_ptr(), dl.data_ptr(), heads * 512, dr.data_ptr(),
                                     heads * 64, keep[3].data_ptr(), c.B, c.T, heads,
                                     ctypes.byref(desc), 0, space.data_ptr(), space.numel(),
                                     flags.data_ptr(), stream, WAIT_NS), out, flags, store, c)
    want, _, tol, _ = R.mla(c, *q, 0.1)
    kva.kva_mla_decode_paged(out, dl, dr, keep[3], desc, 0, 0.1, space, err_flags=flags)
    assert int(flags) == 0
    R.check(out, want, tol)
