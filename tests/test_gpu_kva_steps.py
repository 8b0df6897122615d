"""The calls of include/kva.h as a serving loop uses them (GPU): steps of
append and attention one after another, captured into CUDA graphs, on other
streams, with workspaces shared or not."""
import math

import numpy as np
import pytest
import torch

import kva_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def space_of(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns


class Gqa:
    """A batch with everything a call needs on the device."""

    def __init__(self, kva, seed, new, prior, heads=8, kv_heads=2, head=64, dtype=R.BF16, **kw):
        self.kva, self.heads = kva, heads
        self.c = c = R.Paged(seed, new, prior, kv_heads=kv_heads, head=head, dtype=dtype,
                             **kw).fill()
        self.desc, self.store, self.keep = c.on()
        self.q = c.normal(c.T, heads, head)
        self.scale = 1 / math.sqrt(head)
        self.dq = self.q.cuda()
        self.out = torch.full((c.T, heads, head), 7.0, dtype=torch.bfloat16, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.space = space_of(kva.kva_gqa_decode_workspace(heads, kv_heads, head))

    def call(self, stream=None, space=None):
        self.kva.kva_gqa_decode_paged(self.out, self.dq, self.keep[3], self.desc, self.c.layer,
                                      self.scale, self.space if space is None else space,
                                      v_scale=self.c.v_scale, err_flags=self.flags, stream=stream)

    def check(self):
        want, _, tol, _ = R.gqa(self.c, self.q, self.scale)
        assert int(self.flags) == 0
        R.check(self.out, want, tol)


class Mla:
    def __init__(self, kva, seed, new, prior, heads=16, dtype=R.BF16, **kw):
        self.kva, self.heads = kva, heads
        self.c = c = R.Paged(seed, new, prior, kv_heads=1, head=576, planes=1, dtype=dtype,
                             **kw).fill()
        self.desc, self.store, self.keep = c.on()
        self.q = c.normal(c.T, heads, 512), c.normal(c.T, heads, 64)
        self.scale = 1 / math.sqrt(192)
        self.dq = [x.cuda() for x in self.q]
        self.out = torch.full((c.T, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.space = space_of(kva.kva_mla_decode_workspace(heads))

    def call(self, stream=None, space=None):
        self.kva.kva_mla_decode_paged(self.out, *self.dq, self.keep[3], self.desc, self.c.layer,
                                      self.scale, self.space if space is None else space,
                                      err_flags=self.flags, stream=stream)

    def check(self):
        want, _, tol, _ = R.mla(self.c, *self.q, self.scale)
        assert int(self.flags) == 0
        R.check(self.out, want, tol)


MAKE = [lambda k, s, d: Gqa(k, s, [1, 2, 1], [300, 63, 5000], dtype=d),
        lambda k, s, d: Mla(k, s, [1, 2, 1], [300, 63, 2500], dtype=d),
        lambda k, s, d: Mla(k, s, [1, 1], [90, 1500], heads=128, dtype=d)]


def captured(call):
    """One eager call, then a graph of one."""
    call()
    torch.cuda.synchronize()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        call(stream=s)
    return g


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("make", MAKE)
def test_captured_and_replayed(kva, make, dtype):
    x = make(kva, 80, dtype)
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
    lens = x.keep[2].clone()
    x.keep[2].sub_(50)
    x.c.prior = [p - 50 for p in x.c.prior]
    g.replay()
    torch.cuda.synchronize()
    x.check()
    x.keep[2].copy_(lens)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_graphs_with_workspaces_of_their_own_replay_together(kva, dtype):
    xs = [make(kva, 81 + i, dtype) for i, make in enumerate(MAKE)] + [MAKE[0](kva, 85, dtype)]
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


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("make", MAKE)
def test_captured_behind_other_work(kva, make, joined):
    """A call that follows a copy on its stream, and one that follows a join
    with another stream, inside a graph and outside: the kernels may be
    launched early, what they read may not."""
    x = make(kva, 95, R.BF16)
    real, queries = x.store.clone(), x.dq if isinstance(x.dq, list) else [x.dq]
    given = [q.clone() for q in queries]
    s, side = torch.cuda.Stream(), torch.cuda.Stream()

    def work():
        x.store.copy_(real)
        if joined:
            side.wait_stream(s)
            with torch.cuda.stream(side):
                for q, g in zip(queries, given):
                    torch.add(g, 0, out=q)
            s.wait_stream(side)
        x.call(stream=s)
        x.store.zero_()
        for q in queries:
            if joined:
                q.zero_()

    with torch.cuda.stream(s):
        work()
    torch.cuda.synchronize()
    x.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work()
    for _ in range(3):
        x.out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        x.check()


def test_append_captured_behind_other_work(kva):
    c = R.Paged(96, [40, 1], [0, 9], kv_heads=2, head=64)
    desc, store, keep = c.on()
    qkv, freqs = c.normal(c.T, 8 * 64), R.freqs_table(64, 64)
    (wq, wk, wv), (eq, ek, ev) = R.append(c, qkv, 4, freqs)
    real, dqkv, dfreqs = qkv.cuda(), torch.zeros_like(qkv).cuda(), freqs.cuda()
    q = torch.empty(c.T, 4, 64, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()

    def work():
        torch.mul(real, 1, out=dqkv)
        kva.kva_append_qkv_paged(q, dqkv, keep[3], desc, dfreqs, c.layer, stream=s)
        dqkv.zero_()

    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        work()
    for _ in range(3):
        q.zero_()
        g.replay()
        torch.cuda.synchronize()
        R.check(q, wq, R.HALF_STEP[R.BF16] * wq.abs() * (1 + 2.0 ** -8) + eq, "q")


@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_most_requests(kva, kind):
    """As many requests as a call takes, many without a new token."""
    n = 8192
    new = [(i * 5) % 3 % 2 for i in range(n)]
    prior = [(i * 7) % 5 for i in range(n)]
    kw = dict(page=4, layers=1, layer=0, table_extra=0)
    x = Gqa(kva, 97, new, prior, heads=2, kv_heads=1, head=16, **kw) if kind == "gqa" else \
        Mla(kva, 97, new, prior, heads=1, **kw)
    x.call()
    torch.cuda.synchronize()
    x.check()


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("kind", ["gqa", "mla"])
def test_requests_share_pages(kva, kind, dtype):
    """A common prefix: the same pages in several tables, and twice in one."""
    make = Gqa if kind == "gqa" else Mla
    x = make(kva, 98, [1, 1, 2], [200, 150, 170], dtype=dtype, page=16)
    c = x.c
    c.table[1, :6] = c.table[0, :6]
    c.table[2, 2:5] = c.table[0, 3:6]
    c.table[2, 7] = c.table[2, 1]
    x.keep[1].copy_(c.table)
    x.call()
    torch.cuda.synchronize()
    x.check()


def test_calls_of_one_stream_share_a_workspace(kva):
    a, b, m = MAKE[0](kva, 86, R.BF16), MAKE[0](kva, 87, R.E4M3), MAKE[1](kva, 88, R.E4M3)
    space = space_of(max(x.space.numel() for x in (a, b, m)))
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(4):
        for x in (a, b, m):
            x.call(stream=s, space=space)
    s.synchronize()
    for x in (a, b, m):
        x.check()


@pytest.mark.parametrize("make", MAKE)
def test_on_the_current_stream_of_a_block(kva, make):
    """stream=None is torch's current stream: work queued there comes first."""
    x = make(kva, 89, R.BF16)
    s = torch.cuda.Stream()
    real = x.store.clone()
    x.store.zero_()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(2_000_000)
        x.store.copy_(real)
        x.call()
    s.synchronize()
    x.check()


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_append_then_attention_over_steps(kva, dtype, graph):
    """A prefill and six decode steps of a small model's layer; the cache that
    attention reads is what the append calls wrote."""
    heads, kv_heads, head, rope = 6, 2, 96, 64
    lens, news = [0, 37, 5], [[20, 1, 9]] + [[1, 1, 1]] * 6
    total = [p + sum(n[b] for n in news) for b, p in enumerate(lens)]
    c = R.Paged(92, total, [0, 0, 0], kv_heads=kv_heads, head=head, dtype=dtype, page=12)
    if dtype == R.E4M3:
        c.k_scale, c.v_scale = 1 / 64, 1 / 64
    freqs = R.freqs_table(256, rope)
    gamma = [(1 + 0.1 * torch.randn(head, generator=c.gen)).bfloat16() for _ in range(2)]
    # what is there before the first step
    for b, p in enumerate(lens):
        at = torch.arange(p)
        x = torch.randn(p, kv_heads, head, generator=c.gen)
        for plane, sc in ((0, c.k_scale), (1, c.v_scale)):
            y = x.bfloat16() if dtype == R.BF16 else \
                (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            c.data[c.table[b].long()[at // 12], plane, c.layer, at % 12] = y
    desc, store, keep = c.on()
    dfreqs, dg = freqs.cuda(), [x.cuda() for x in gamma]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = space_of(kva.kva_gqa_decode_workspace(heads, kv_heads, head))
    step_graph = None
    for step, new in enumerate(news):
        T = sum(new)
        s = R.Paged(0, new, lens, kv_heads=kv_heads, head=head, dtype=dtype, page=12)
        s.table, s.pages, s.k_scale, s.v_scale = c.table, c.pages, c.k_scale, c.v_scale
        qkv = (2 * torch.randn(T, (heads + 2 * kv_heads) * head, generator=c.gen)).bfloat16()
        s.store = store.cpu()
        s.data = c.view(s.store)
        (wq, wk, wv), (eq, ek, ev) = R.append(s, qkv, heads, freqs, q_gamma=gamma[0],
                                              k_gamma=gamma[1])
        keep[2].copy_(torch.tensor(lens, dtype=torch.int32))
        if step < 2 or not graph:
            off = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).cuda()
            dqkv = qkv.cuda()
            q = torch.empty(T, heads, head, dtype=torch.bfloat16, device="cuda")
            out = torch.empty_like(q)
        else:
            dqkv.copy_(qkv)

        def both(stream=None):
            kva.kva_append_qkv_paged(q, dqkv, off, desc, dfreqs, c.layer, q_gamma=dg[0],
                                     k_gamma=dg[1], v_scale=c.v_scale, err_flags=flags,
                                     stream=stream)
            kva.kva_gqa_decode_paged(out, q, off, desc, c.layer, 0.1, space, v_scale=c.v_scale,
                                     err_flags=flags, stream=stream)

        if graph and step >= 2:
            if step_graph is None:
                step_graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
                torch.cuda.synchronize()
                with torch.cuda.graph(step_graph, stream=side):
                    both(stream=side)
            step_graph.replay()
        else:
            both()
        torch.cuda.synchronize()
        assert int(flags) == 0
        R.check(q, wq, R.HALF_STEP[R.BF16] * wq.abs() * (1 + 2.0 ** -8) + eq, "q")
        s.data = c.view(store)
        for t, b, pos in s.tokens():
            row = s.data[c.table[b, pos // 12], :, c.layer, pos % 12]
            for plane, (w, e, sc) in enumerate(((wk, ek, c.k_scale), (wv, ev, c.v_scale))):
                have = row[plane].double() if dtype == R.BF16 else \
                    row[plane].view(torch.float8_e4m3fn).double()
                unit = w[t] if dtype == R.BF16 else (w[t] / sc).clamp(-448, 448)
                R.check(have, unit, R.stored_error(w[t], e[t], dtype, sc), "cache")
        # attention: exact over the queries and the cache as they were stored
        want, _, tol, _ = R.gqa(s, q.cpu(), 0.1)
        R.check(out, want, tol, "out")
        lens = [p + n for p, n in zip(lens, new)]


@pytest.mark.parametrize("cache_dtype", [R.BF16, R.E4M3])
def test_mla_write_then_attention(kva, cache_dtype):
    """kvw_mla_rope_rmsnorm_quant writes the new tokens' latent rows and turns
    the queries; attention reads both as they come."""
    from gqa_kv_cache_mla_gb300 import device, workloads as W

    heads = 16
    w = W.mla_workload("st", 1501, [3, 0, 1, 70, 9], [0] * 5, num_heads=heads, page_size=16,
                       max_seq_len=256, num_layers=2, layer_idx=1,
                       cache_dtype=W.DTYPE_BF16 if cache_dtype == R.BF16 else W.DTYPE_FP8_E4M3)
    d = device.DeviceMLA(w, device="cuda:0")
    d.run()
    g = torch.Generator().manual_seed(93)
    c = R.Paged(0, np.diff(w.offsets).tolist(), w.cache.cache_lengths.tolist(), kv_heads=1,
                head=576, planes=1, dtype=cache_dtype, page=16)
    ql = torch.randn(c.T, heads, 512, generator=g).bfloat16()
    out = torch.empty(c.T, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(c.T, heads, device="cuda")
    dql, space = ql.cuda(), space_of(kva.kva_mla_decode_workspace(heads))
    kva.kva_mla_decode_paged(out, dql, d.q_out.tensor, d.offsets.tensor, d.desc, w.layer_idx, 0.07,
                             space, lse=lse, err_flags=d.err.tensor, num_batches=c.B,
                             tot_seq_len=c.T, num_heads=heads, q_rope_row_stride=heads * 64)
    torch.cuda.synchronize()
    assert d.flags() == 0 and d.guards_intact()
    # the evaluation reads what the write call left
    host = torch.from_numpy(d.cache.host().copy())
    item = torch.bfloat16 if cache_dtype == R.BF16 else torch.uint8
    pages = w.cache.num_pages
    host = host.view(torch.uint8).view(item).reshape(pages, 1, 2, 16, 1, 576)
    c.data, c.layer, c.pages, c.k_scale = host, w.layer_idx, pages, float(w.cache.scale)
    c.table = torch.from_numpy(w.cache.page_table.astype(np.int32))
    if cache_dtype == R.BF16:
        c.k_scale = 1.0
    qr = torch.from_numpy(d.q_out.host().copy()).view(torch.uint8).view(torch.bfloat16)
    qr = qr.reshape(-1)[:c.T * heads * 64].reshape(c.T, heads, 64)
    want, want_lse, tol, tol_lse = R.mla(c, ql, qr, 0.07)
    assert bool(torch.isfinite(want).all())
    R.check(out, want, tol, "out")
    R.check(lse, want_lse, tol_lse, "lse")


@pytest.mark.parametrize("kind,dtype", [("gqa", R.BF16), ("gqa", R.E4M3), ("mla", R.BF16),
                                        ("mla", R.E4M3)])
@pytest.mark.parametrize("page", [16, 64])
def test_pages_past_32_bit_offsets(kva, kind, dtype, page):
    """The same pages at the far end of a cache of more than 2^32 elements
    give the same bits; appending to them writes the same rows."""
    from gqa_kv_cache_mla_gb300 import kvw

    kw = dict(dtype=dtype, page=page, layers=1, layer=0)
    x = Gqa(kva, 99, [1, 2], [150, 700], head=128, **kw) if kind == "gqa" else \
        Mla(kva, 99, [1, 2], [150, 700], **kw)
    c = x.c
    one = c.store[0].numel()
    pages = (1 << 32) // one + 8 + c.pages
    big = torch.empty((pages, one), dtype=c.store.dtype, device="cuda")
    far = pages - c.pages
    big[far:] = x.store.reshape(c.pages, one)
    table = torch.where(x.keep[1] >= 0, x.keep[1] + far, x.keep[1])
    st = c.data.stride()
    desc = kvw.paged_cache(big, dtype, table, x.keep[2], pages, 1, page, c.kv_heads, c.head, st[:5],
                           scale=c.k_scale)
    if kind == "gqa":
        qkv, freqs = c.normal(c.T, 12 * 128).cuda(), R.freqs_table(1024, 128).cuda()
        q = [torch.empty(c.T, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for y, d in zip(q, (x.desc, desc)):
            kva.kva_append_qkv_paged(y, qkv, x.keep[3], d, freqs, 0, v_scale=c.v_scale,
                                     err_flags=x.flags)
        assert torch.equal(*q)
        assert torch.equal(big[far:].view(torch.uint8),
                           x.store.reshape(c.pages, one).view(torch.uint8))
    x.call()
    near = x.out.clone()
    x.out.fill_(7.0)
    x.desc = desc
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0 and torch.equal(x.out, near)


@pytest.mark.parametrize("length", [0x7FFFFFFF, 0x80000000, 0xFFFFFFFF])
@pytest.mark.parametrize("kind", ["gqa", "mla"])
@pytest.mark.parametrize("page", [16, 64])
def test_the_longest_lengths(kva, kind, length, page):
    """Positions past the page table have no page: what the table reaches is
    seen, and the flag set."""
    make = Gqa if kind == "gqa" else Mla
    x = make(kva, 100, [1, 1], [191, 30], page=page, table_extra=0)
    x.call()
    torch.cuda.synchronize()
    x.check()
    all_seen = x.out.clone()
    x.keep[2][0] = length - (1 << 32) if length >> 31 else length
    x.out.fill_(7.0)
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 1
    assert torch.equal(x.out, all_seen)
