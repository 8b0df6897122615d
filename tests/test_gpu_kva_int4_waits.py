"""Bounded waits of the attention over a cache held in 4 bits that run out while
the ring has come round several times (GPU): every piece has three rings of
tiles, which test_gpu_kva_int4_steps.py's contexts do not reach."""
import ctypes
import time

import pytest
import torch

import kva_int4_reference as Q
from test_gpu_kva_int4 import Call, kva  # noqa: F401 (fixture)
from test_gpu_kva_int4_paths import tiles_wanted
from test_gpu_kva_int4_steps import hook  # noqa: F401 (fixture)
from test_gpu_timeout import KVW_ERR_TIMEOUT, WAIT_NS

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [64, 48, 16])
@pytest.mark.parametrize("abandoned", [False, True])
def test_waits_that_run_out_in_a_full_ring(kva, hook, head, page, abandoned):
    period = 13 * (64 if page == 16 else page)
    c = Q.Int4(226, [1, 2, 0, 1, 1], [period - 1, 900, 3, 0, 64], head=head, page=page, layers=1,
               layer=0, table_extra=0).fill()
    # the first request's context goes through the same pages over and over
    times = -(-tiles_wanted(head) * 64 // period)
    mine = period // page
    c.table = torch.nn.functional.pad(c.table, (0, mine * times - c.table.shape[1]), value=-1)
    c.table[0] = c.table[0, :mine].repeat(times)
    c.lens[0] = period * times - 1
    x = Call(kva, c, 8, sm_scale=0.1)
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0
    whole = x.out.clone()
    x.out.fill_(7.0)
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    assert hook(x.out.data_ptr(), x.dq.data_ptr(), 8 * head, x.keep[4].data_ptr(), c.B, c.T, 8,
                ctypes.byref(x.cache), ctypes.byref(x.scales), 0, x.space.data_ptr(),
                x.space.numel(), flags.data_ptr(),
                ctypes.c_void_p(torch.cuda.current_stream().cuda_stream),
                WAIT_NS, int(abandoned)) == 0
    torch.cuda.synchronize()
    assert time.perf_counter() - t0 < 5.0
    assert int(flags[0]) & KVW_ERR_TIMEOUT
    assert int(flags[1]) == 0  # no copy was under way when its CTA went
    assert bool((x.out == 7.0).all())
    # the context is as good as before
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0 and torch.equal(x.out, whole)
