"""A cache held in 4 bits as a serving loop uses it (GPU): page tables, append,
gather and attention one after another, captured into CUDA graphs, on other
streams, with workspaces shared or not, and bounded waits that run out."""
import ctypes
import math
import time

import pytest
import torch

import kva_int4_reference as Q
import kva_reference as R
from test_gpu_kva_int4 import Call, gather, lengths
from test_gpu_timeout import KVW_ERR_TIMEOUT, WAIT_NS, _hook_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


MAKE = [lambda k, s: Call(k, Q.Int4(s, [1, 2, 1], [300, 63, 5000], head=64).fill(), 8),
        lambda k, s: Call(k, Q.Int4(s, *lengths(90, 1500), head=128, page=64).fill(), 32),
        lambda k, s: Call(k, Q.Int4(s, [1, 3], [700, 20], kv_heads=1, head=256).fill(), 5)]


def captured(call):
    """One eager call, then a graph of one."""
    call()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        call(stream=s)
    return g


@pytest.mark.parametrize("make", MAKE)
def test_captured_and_replayed(kva, make):
    x = make(kva, 180)
    g = captured(x.call)
    eager = x.out.clone()
    for _ in range(3):
        x.out.fill_(7.0)
        x.space.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.out, eager)
    x.check()
    # the graph reads the lengths and the tables when it is replayed
    x.keep[3].sub_(15)
    x.c.prior = [p - 15 for p in x.c.prior]
    g.replay()
    x.check()


def test_graphs_with_workspaces_of_their_own_replay_together(kva):
    xs = [make(kva, 181 + i) for i, make in enumerate(MAKE)] + [MAKE[1](kva, 185)]
    graphs = [captured(x.call) for x in xs]
    eager = [x.out.clone() for x in xs]
    for x in xs:
        x.out.fill_(7.0)
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for x, e in zip(xs, eager):
        assert torch.equal(x.out, e)
        x.check()


def test_calls_of_one_stream_share_a_workspace(kva):
    xs = [make(kva, 186 + i) for i, make in enumerate(MAKE)]
    n = max(x.space.numel() for x in xs)
    space = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for x in xs:
            x.call(stream=s, space=space)
    s.synchronize()
    for x in xs:
        x.check()


@pytest.mark.parametrize("make", MAKE)
def test_on_the_current_stream_behind_other_work(kva, make):
    """stream=None is torch's current stream; the kernels may be launched early,
    what they read may not be."""
    x = make(kva, 189)
    s = torch.cuda.Stream()
    real = [k.clone() for k in (*x.keep[:2], x.dq)]
    for t in (*x.keep[:2], x.dq):
        t.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        for t, r in zip((*x.keep[:2], x.dq), real):
            t.copy_(r)
        x.call()
        for t in x.keep[:2]:
            t.zero_()
    s.synchronize()
    for t, r in zip(x.keep[:2], real):
        t.copy_(r)
    x.check()


def test_most_requests(kva):
    n = 8192
    new, prior = [(i * 5) % 3 % 2 for i in range(n)], [(i * 7) % 5 for i in range(n)]
    c = Q.Int4(190, new, prior, kv_heads=1, layers=1, layer=0, table_extra=0).fill()
    x = Call(kva, c, 2)
    x.call()
    x.check()


def test_requests_share_pages(kva):
    """A common prefix: the same pages in several tables, and twice in one."""
    c = Q.Int4(191, [1, 1, 2], [200, 150, 170], page=16).fill()
    c.table[1, :6] = c.table[0, :6]
    c.table[2, 2:5] = c.table[0, 3:6]
    c.table[2, 7] = c.table[2, 1]
    x = Call(kva, c, 8)
    x.call()
    x.check()
    gather(kva, c, [201, 151, 172])


@pytest.mark.parametrize("page", [16, 64])
def test_pages_past_32_bit_offsets(kva, page):
    """The same pages at the far end of a cache of more than 2^32 bytes of codes
    give the same bits; appending to them writes the same rows."""
    x = Call(kva, Q.Int4(192, [1, 2], [150, 700], head=128, page=page, layers=1, layer=0).fill(), 8)
    c = x.c
    one = [s[0].numel() for s in (c.code_store, c.scale_store)]
    pages = (1 << 32) // one[0] + 8 + c.pages
    far = pages - c.pages
    big = [torch.empty((pages, n), dtype=s.dtype, device="cuda")
           for n, s in zip(one, (c.code_store, c.scale_store))]
    for b, k in zip(big, x.keep):
        b[far:] = k
    table = torch.where(x.keep[2] >= 0, x.keep[2] + far, x.keep[2])
    views = [torch.as_strided(b, (pages, *sh[1:]), st) for b, sh, st in
             zip(big, (c.code_shape, c.scale_shape), (c.code_stride, c.scale_stride))]
    cache, scales = kva.int4_cache(*views, table, x.keep[3])
    qkv, freqs = c.normal(c.T, 12 * 128).cuda(), R.freqs_table(1024, 128).cuda()
    q = [torch.empty(c.T, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    rows = [torch.empty(853, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    off = torch.tensor([0, 151, 853], dtype=torch.int32, device="cuda")
    for i, (y, d) in enumerate(zip(q, ((x.cache, x.scales), (cache, scales)))):
        kva.kva_append_qkv_int4(y, qkv, x.keep[4], *d, freqs, 0, err_flags=x.flags)
        kva.kva_gather_kv_int4(rows[2 * i], rows[2 * i + 1], off, *d, 0, err_flags=x.flags)
    assert torch.equal(*q)
    assert torch.equal(rows[0], rows[2]) and torch.equal(rows[1], rows[3])
    for b, k in zip(big, x.keep):
        assert torch.equal(b[far:].view(torch.uint8), k.view(torch.uint8))
    x.call()
    near = x.out.clone()
    x.out.fill_(7.0)
    x.cache, x.scales = cache, scales
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0 and torch.equal(x.out, near)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("head,page", [(96, 48), (128, 64)])
def test_whole_steps(kva, graph, head, page):
    """A prefill and decode steps of a small model's layer, from page tables that
    are empty at first: tables, append, gather of what was appended, attention."""
    heads, kv_heads, rope = 6, 2, head // 2
    news = [[20, 1, 90]] + [[1, 1, 1]] * 40
    lens = [0, 0, 0]
    c = Q.Int4(193, [70, 70, 140], lens, kv_heads=kv_heads, head=head, page=page, spare_pages=5)
    free = torch.randperm(c.pages, generator=c.gen).to(torch.int32)
    c.table[:] = R.UNMAPPED
    width = c.table.shape[1]
    cache, scales, keep = c.on()
    table, dlens = keep[2], keep[3]
    freqs = R.freqs_table(256, rope)
    gamma = [(1 + 0.1 * torch.randn(head, generator=c.gen)).bfloat16() for _ in range(2)]
    dfree, dfreqs, dg = free.cuda(), freqs.cuda(), [x.cuda() for x in gamma]
    taken = torch.zeros(1, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_gqa_decode_workspace(heads, kv_heads, head),), 0xFF,
                       dtype=torch.uint8, device="cuda")
    step_graph = None
    for step, new in enumerate(news):
        T = sum(new)
        off = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32).cuda()
        qkv = (2 * torch.randn(T, (heads + 2 * kv_heads) * head, generator=c.gen)).bfloat16()
        if step < 2:
            doff, dqkv = off, qkv.cuda()
            slots = torch.empty(T, dtype=torch.int64, device="cuda")
            q = torch.empty(T, heads, head, dtype=torch.bfloat16, device="cuda")
            out, back = torch.empty_like(q), [
                torch.empty(T, kv_heads, head, dtype=torch.bfloat16, device="cuda")
                for _ in range(2)]
        else:
            dqkv.copy_(qkv)
        before = keep[0].cpu(), keep[1].cpu()

        def work(stream=None):
            kva.kva_extend_page_tables(table, dlens, doff, dfree, taken, taken, page, c.pages,
                                       slot_map=slots, err_flags=flags, stream=stream)
            kva.kva_append_qkv_int4(q, dqkv, doff, cache, scales, dfreqs, c.layer, q_gamma=dg[0],
                                    k_gamma=dg[1], err_flags=flags, stream=stream)
            kva.kva_gather_kv_int4(*back, doff, cache, scales, c.layer, first_positions=dlens,
                                   err_flags=flags, stream=stream)
            kva.kva_gqa_decode_int4(out, q, doff, cache, scales, c.layer, 0.1, space,
                                    err_flags=flags, stream=stream)

        if graph and step >= 2:
            if step_graph is None:
                step_graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.graph(step_graph, stream=side):
                    work(stream=side)
            step_graph.replay()
        else:
            work()
        torch.cuda.synchronize()
        assert int(flags) == 0
        s = Q.Int4(0, new, lens, kv_heads=kv_heads, head=head, page=page)
        s.table, s.pages, s.code_shape, s.scale_shape = (table.cpu(), c.pages, c.code_shape,
                                                         c.scale_shape)
        s.code_stride, s.scale_stride = c.code_stride, c.scale_stride
        s.see(keep[0], keep[1])
        # ids are distinct, and taken in the order of the list
        used = s.table[s.table >= 0]
        need = sum(-(-(p + n) // page) for p, n in zip(lens, new))
        assert len(used) == len(used.unique()) == need == int(taken)
        assert set(used.tolist()) == set(free[:need].tolist())
        want, err = R.append(s, qkv, heads, freqs, q_gamma=gamma[0], k_gamma=gamma[1])
        R.check(q, want[0], R.HALF_STEP[R.BF16] * want[0].abs() * (1 + 2.0 ** -8) + err[0], "q")
        where = slots.cpu()
        for t, b, pos in s.tokens():
            p, row = int(s.table[b, pos // page]), pos % page
            assert int(where[t]) == p * page + row
            u, by = s.rows(torch.tensor([p]), torch.tensor([row]))
            for plane in range(2):
                Q.check_held(u[0, plane].long(), s.scales[p, plane, s.layer, :, :, row],
                             want[1 + plane][t], err[1 + plane][t])
                assert torch.equal(back[plane][t].cpu(), ((u - 8) * by)[0, plane].bfloat16())
        # the other layer is left alone
        assert torch.equal(s.codes[:, :, 0], torch.as_strided(before[0], s.code_shape,
                                                              s.code_stride)[:, :, 0])
        # attention: exact over the queries and the cache as they were stored
        wo, _, tol, _ = Q.gqa(s, q.cpu(), 0.1)
        R.check(out, wo, tol, "out")
        lens = [p + n for p, n in zip(lens, new)]
        dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        assert width == table.shape[1]


# ------------------------------------------------------------------ waits that run out

@pytest.fixture(scope="module")
def hook(kva, tmp_path_factory):
    """The kernel with its first tile of every CTA announced but never copied, or
    with consumers that leave at once (a library of this test's own)."""
    from gqa_kv_cache_mla_gb300 import kvw

    vp, u32, i64, u64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_int64, ctypes.c_uint64
    f = _hook_library(tmp_path_factory, "gqa_decode_int4.cu").kva_test_gqa_int4
    f.restype = ctypes.c_int
    f.argtypes = [vp, vp, i64, vp, u32, u32, u32, ctypes.POINTER(kvw.PagedCacheT),
                  ctypes.POINTER(kva.GroupScalesT), u32, vp, u64, vp, vp, u64, ctypes.c_int]
    return f


@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("page", [64, 48])
@pytest.mark.parametrize("abandoned", [False, True])
def test_waits_that_run_out(kva, hook, head, page, abandoned):
    # one long context, so that every piece has more tiles than its ring, and
    # short ones, whose pieces have one
    c = Q.Int4(194, [1, 2, 0, 1, 1], [40000, 900, 3, 0, 64], head=head, page=page, layers=1,
               layer=0).fill()
    x = Call(kva, c, 8, sm_scale=0.1)
    flags = torch.zeros(2, dtype=torch.int32, device="cuda")
    before = x.out.clone()
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
    assert torch.equal(x.out, before)
    # the context is as good as before
    x.call()
    x.check()
