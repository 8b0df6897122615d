"""A CTA of the attention calls ends only when its copies have landed (GPU).

In the test build the consumers leave at once, as those do whose wait ran out,
so nobody waits for what the feeding warps have issued: all of a piece that
fits their ring, or the ring's fill of a longer one.  The feeding warps then
count the places whose last copy is still under way when they leave."""
import ctypes

import pytest
import torch

import kva_reference as R
from test_gpu_kva_timeout import I64, KVW_ERR_TIMEOUT, U32, U64, VP, WAIT_NS, hook

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def check_abandoned(call, flags, out, store, c):
    assert call(ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert int(flags[0]) & KVW_ERR_TIMEOUT
    assert int(flags[1]) == 0
    assert bool((out == 7.0).all())
    assert torch.equal(store.cpu().view(torch.uint8), c.store.view(torch.uint8))


CONTEXTS = [([1, 1, 1], [60, 100, 300]), ([1, 2, 0, 1, 1], [40000, 900, 3, 0, 64])]


@pytest.fixture(scope="module")
def gqa_abandoned(kva, tmp_path_factory):
    from gqa_kv_cache_mla_gb300 import kvw

    return hook(tmp_path_factory, "gqa_decode_paged.cu", "kva_test_gqa_decode_abandoned",
                [VP, VP, I64, VP, U32, U32, U32, ctypes.POINTER(kvw.PagedCacheT), U32, VP, U64, VP,
                 VP, U64])


@pytest.fixture(scope="module")
def mla_abandoned(kva, tmp_path_factory):
    from gqa_kv_cache_mla_gb300 import kvw

    return hook(tmp_path_factory, "mla_decode_paged.cu", "kva_test_mla_decode_abandoned",
                [VP, VP, I64, VP, I64, VP, U32, U32, U32, ctypes.POINTER(kvw.PagedCacheT), U32, VP,
                 U64, VP, VP, U64])


@pytest.mark.parametrize("new,prior", CONTEXTS)
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [64, 12])
def test_gqa(kva, gqa_abandoned, dtype, page, new, prior):
    c = R.Paged(92, new, prior, kv_heads=2, head=128, dtype=dtype, page=page, layers=1,
                layer=0).fill()
    desc, store, keep = c.on()
    q = c.normal(c.T, 8, 128)
    dq, out = q.cuda(), torch.full((c.T, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    space = torch.empty(kva.kva_gqa_decode_workspace(8, 2, 128), dtype=torch.uint8, device="cuda")
    check_abandoned(lambda stream: gqa_abandoned(
        out.data_ptr(), dq.data_ptr(), 8 * 128, keep[3].data_ptr(), c.B, c.T, 8,
        ctypes.byref(desc), 0, space.data_ptr(), space.numel(), flags.data_ptr(), stream,
        WAIT_NS), flags, out, store, c)


@pytest.mark.parametrize("new,prior", CONTEXTS)
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [64, 12])
def test_mla(kva, mla_abandoned, dtype, page, new, prior):
    heads = 80
    c = R.Paged(93, new, prior, kv_heads=1, head=576, planes=1, dtype=dtype, page=page, layers=1,
                layer=0).fill()
    desc, store, keep = c.on()
    dl, dr = c.normal(c.T, heads, 512).cuda(), c.normal(c.T, heads, 64).cuda()
    out = torch.full((c.T, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    space = torch.empty(kva.kva_mla_decode_workspace(heads), dtype=torch.uint8, device="cuda")
    check_abandoned(lambda stream: mla_abandoned(
        out.data_ptr(), dl.data_ptr(), heads * 512, dr.data_ptr(), heads * 64,
        keep[3].data_ptr(), c.B, c.T, heads, ctypes.byref(desc), 0, space.data_ptr(),
        space.numel(), flags.data_ptr(), stream, WAIT_NS), flags, out, store, c)
