"""The loops that large calls on a cache held in 4 bits run in (GPU): attention
whose pieces take many tiles, of many segments, over rings that come round again
and again; appends of several passes an item and several items a warp; reads of
several (plane, head) pairs an item; page tables on many CTAs."""
import math

import pytest
import torch

import kva_int4_reference as Q
import kva_reference as R
from test_gpu_kva_int4 import Call, kva, lengths  # noqa: F401 (fixture)
from test_gpu_kva_int4_weights import repeated, run_repeated
from test_gpu_kva_tables import Batch

pytestmark = pytest.mark.gpu

# tiles of the ring, CTAs of an SM
RING = {64: (12, 3), 96: (8, 3), 128: (6, 3), 256: (5, 2)}


def tiles_wanted(head, rings=3):
    """Tiles that are at least `rings` rings for every CTA."""
    ring, ctas = RING[head]
    return rings * ring * ctas * torch.cuda.get_device_properties(0).multi_processor_count


def enough(c, head):
    """Repetitions of c's requests that are."""
    return -(-tiles_wanted(head) // (c.kv_heads * sum(-(-(p + n) // 64) for n, p in
                                                      zip(c.new, c.prior))))


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("head,q_heads", [(64, 8), (96, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("page", [16, 48, 64])
@pytest.mark.parametrize("mods", [
    {}, {"softcap": 5.0}, {"alibi": True}, {"softcap": 20.0, "alibi": True}, {"window": 100},
    {"window": 700, "softcap": 30.0}], ids=lambda m: "-".join(m) or "plain")
def test_many_tiles_and_segments_a_piece(kva, head, q_heads, page, mods):
    c = Q.Int4(220, [1, 2, 1, 1, 3], [1500, 62, 700, 0, 333], kv_heads=2, head=head, page=page,
               layers=1, layer=0).fill()
    run_repeated(kva, c, c.normal(c.T, q_heads, head, std=2.0), enough(c, head), least=0.0, **mods)


@pytest.mark.parametrize("head,q_heads", [(64, 4), (96, 4), (128, 8), (256, 4)])
@pytest.mark.parametrize("page", [16, 48, 64])
@pytest.mark.parametrize("softcap", [0.0, 10.0])
def test_many_tiles_of_one_segment(kva, head, q_heads, page, softcap):
    """One context, whose table goes through the same 13 pages (of 16: 52) over and
    over: the same mean of the values, and a sum as many times as large.

    A piece adds up at most 37 products of 17 cuts, then four warps and 456 pieces
    are joined: fewer terms than two periods have, so twice a period's tolerance."""
    period = 13 * (64 if page == 16 else page)
    c = Q.Int4(221, *lengths(period), kv_heads=1, head=head, page=page, layers=1, layer=0,
               table_extra=0).fill()
    q = c.normal(1, q_heads, head, std=2.0)
    times = -(-tiles_wanted(head) * 64 // period)
    want, lse, to, tl = Q.gqa(c, q, 1 / math.sqrt(head), softcap)
    c.table = c.table.repeat(1, times)
    c.prior, c.lens = [period * times - 1], torch.tensor([period * times - 1], dtype=torch.int32)
    x = Call(kva, c, q_heads, q=q, softcap=softcap)
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0
    R.check(x.out, want, 2 * to, "out")
    R.check(x.lse, lse + math.log(times), tl + 2.0 ** -22 * math.log(times), "lse")


@pytest.mark.parametrize("head,q_heads", [(64, 2), (96, 8), (128, 12), (256, 4)])
@pytest.mark.parametrize("nats", [40, 120, 300])
@pytest.mark.parametrize("early", [True, False])
@pytest.mark.parametrize("mods", [{}, {"softcap": 500.0}, {"alibi": True}],
                         ids=lambda m: "-".join(m) or "plain")
def test_scores_that_rise_along_the_context(kva, head, q_heads, nats, early, mods):
    """Up to `nats` between a context's ends: sums are held, and the reference moves
    as the tiles are taken (from the last to the first) or stays."""
    n = 1000
    c = Q.Int4(222, *lengths(n), kv_heads=1, head=head, page=64, layers=1, layer=0).fill()
    along = torch.arange(n).float() / n
    k = (1 - along if early else along)[:, None, None].expand(n, 1, head)
    c.put(0, 0, 0, *Q.held(k))
    q = torch.full((1, q_heads, head), nats / head).bfloat16()
    run_repeated(kva, c, q, enough(c, head), sm_scale=1.0, least=0.0, **mods)


@pytest.mark.parametrize("head,q_heads", [(64, 2), (96, 8), (128, 12), (256, 4)])
@pytest.mark.parametrize("powers", [(-30, 40), (40, -30), (0, 60), (20, 20)])
def test_value_scales_along_the_context(kva, head, q_heads, powers):
    n = 1000
    c = Q.Int4(223, *lengths(n, 330), kv_heads=1, head=head, page=64, layers=1, layer=0).fill()
    for b in range(2):
        n = c.prior[b] + 1
        ids, row = c.place(b, 0, n)
        e = torch.linspace(powers[0], powers[1], n).round()
        x = c.scales[ids, 1, c.layer, :, :, row].double() * 2.0 ** e.double()[:, None, None]
        c.scales[ids, 1, c.layer, :, :, row] = x.bfloat16()
    run_repeated(kva, c, c.normal(2, q_heads, head, std=2.0), enough(c, head), least=0.0)


@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
def test_bad_pages_among_many_tiles(kva, head, page):
    """Tiles that are only partly there between whole ones."""
    c = Q.Int4(224, *lengths(900, 330), kv_heads=1, head=head, page=page, layers=1, layer=0).fill()
    c.table[0, 200 // page] = R.UNMAPPED
    c.table[0, 700 // page] = c.pages
    c.table[1, 0] = R.UNMAPPED
    q = c.normal(2, 4, head, std=2.0)
    x = Call(kva, repeated(c, enough(c, head)), 4, q=q.repeat(enough(c, head), 1, 1))
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 1
    out, _, to, _ = Q.gqa(c, q, x.scale)
    R.check(x.out.cpu(), out.repeat(enough(c, head), 1, 1), to.repeat(enough(c, head), 1, 1))


@pytest.mark.parametrize("head", [64, 96, 128])
@pytest.mark.parametrize("extra", [0, 40, 4000])
def test_tables_that_reach_further(kva, head, extra):
    """What the page table could hold, not what it holds, decides on the CTAs."""
    c = Q.Int4(225, *lengths(901), kv_heads=2, head=head, page=64, table_extra=extra).fill()
    x = Call(kva, c, 8)
    x.call()
    x.check()


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("tokens,q_heads", [(10500, 17), (5003, 16), (2501, 17)])
@pytest.mark.parametrize("norm,interleaved", [(False, False), (False, True), (True, False)])
def test_large_appends_equal_small_ones(kva, head, tokens, q_heads, norm, interleaved):
    """A token's values do not depend on the call: one of so many tokens that an
    item has several passes and a warp several items, against calls of at most 100
    tokens, which have one pass an item."""
    new, prior, kv_heads, rope = [tokens - 904, 0, 904], [70, 3, 5], 8, 64
    c = Q.Int4(230, new, prior, kv_heads=kv_heads, head=head, page=64, layers=1, layer=0,
               table_extra=0)
    gen = torch.Generator(device="cuda").manual_seed(231)
    qkv = torch.randn(tokens, (q_heads + 2 * kv_heads) * head, generator=gen,
                      device="cuda").bfloat16()
    freqs = R.freqs_table(tokens + 100, rope).cuda()
    g = torch.randn(head, generator=gen, device="cuda").bfloat16() if norm else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    stores, queries = [], []
    for small in (False, True):
        cache, scales, keep = c.on()
        q = torch.full((tokens, q_heads, head), 7.0, dtype=torch.bfloat16, device="cuda")
        kw = dict(q_gamma=g, k_gamma=g, interleaved=interleaved, err_flags=flags)
        if not small:
            kva.kva_append_qkv_int4(q, qkv, keep[4], cache, scales, freqs, 0, **kw)
        else:
            t0 = 0
            for b, n in enumerate(new):
                for at in range(0, n, 100):
                    m = min(100, n - at)
                    lens = torch.tensor([prior[b] + at], dtype=torch.int32, device="cuda")
                    one = torch.tensor([0, m], dtype=torch.int32, device="cuda")
                    part = kva.int4_cache(
                        torch.as_strided(keep[0], c.code_shape, c.code_stride),
                        torch.as_strided(keep[1], c.scale_shape, c.scale_stride),
                        keep[2][b:b + 1], lens)
                    rows = slice(t0 + at, t0 + at + m)
                    kva.kva_append_qkv_int4(q[rows], qkv[rows], one, *part, freqs, 0, **kw)
                    torch.cuda.synchronize()  # the descriptors' tensors live until here
                t0 += n
        stores.append(keep[:2])
        queries.append(q)
    assert int(flags) == 0 and torch.equal(*queries)
    for x, y in zip(*stores):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("head", [64, 96, 128, 256])
def test_bits_of_a_large_append(kva, head):
    """Codes and scales of the header, bit for bit, with several passes an item."""
    tokens, kv_heads = 10100, 16
    c = Q.Int4(232, [tokens], [9], kv_heads=kv_heads, head=head, page=64, layers=1, layer=0)
    qkv = c.normal(tokens, 2 * kv_heads * head)
    cache, scales, keep = c.on()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    kva.kva_append_qkv_int4(None, qkv.cuda(), keep[4], cache, scales, None, 0, err_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    c.see(keep[0], keep[1])
    x = qkv.float().view(tokens, 2, kv_heads, head)
    ids, row = c.place(0, 9, 9 + tokens)
    for plane in range(2):
        u, s = Q.held(x[:, plane])
        assert torch.equal(c.scales[ids, plane, 0, :, :, row].view(torch.int16), s.view(torch.int16))
        assert torch.equal(c.codes[ids, plane, 0, :, row], Q.pack(u))


# ------------------------------------------------------------------ gather

@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("kv_heads,planes", [(1, 2), (3, 1), (3, 2), (5, 1)])
@pytest.mark.parametrize("count", [70, 18])
@pytest.mark.parametrize("page", [16, 64])
def test_large_reads(kva, head, kv_heads, planes, count, page):
    """Items of several (plane, head) pairs, odd numbers of them and a shorter last
    item of a row too."""
    n = 4100
    c = Q.Int4(240, [0], [n], kv_heads=kv_heads, head=head, page=page, layers=1, layer=0).fill()
    first = [(37 * b) % 1500 for b in range(count)]
    rows = [2500 - (53 * b) % 300 for b in range(count)]
    keep = c.on()[2]
    table, lens = keep[2].repeat(count, 1), keep[3].repeat(count)
    cache, scales = kva.int4_cache(torch.as_strided(keep[0], c.code_shape, c.code_stride),
                                   torch.as_strided(keep[1], c.scale_shape, c.scale_stride),
                                   table, lens)
    off = torch.tensor([0] + torch.tensor(rows).cumsum(0).tolist(), dtype=torch.int32).cuda()
    start = torch.tensor(first, dtype=torch.int32).cuda()
    out = [torch.full((sum(rows), kv_heads, head), 7.0, dtype=torch.bfloat16, device="cuda")
           for _ in range(planes)]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    # one plane: the values
    kva.kva_gather_kv_int4(out[0] if planes == 2 else None, out[-1], off, cache, scales, 0,
                           first_positions=start, err_flags=flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    u, s = c.rows(*c.place(0, 0, n))
    for plane, got in zip(range(2 - planes, 2), out):
        want = ((u[:, plane] - 8) * s[:, plane]).bfloat16().cuda()
        want = torch.cat([want[f:f + m] for f, m in zip(first, rows)])
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))


# ------------------------------------------------------------------ page tables

@pytest.mark.parametrize("new,lens", [
    ([5000, 1, 0, 9000, 3000], [100, 200, 300, 0, 17]),
    ([120000, 0, 60000, 1, 20003], [3, 9, 1000, 15, 16])])
@pytest.mark.parametrize("in_place", [False, True])
def test_page_tables_of_many_tokens(kva, new, lens, in_place):
    """More tokens than one CTA takes, and than one token for each thread."""
    Batch(250, new, lens, 16).run(kva, in_place)


def test_page_tables_of_many_requests_and_tokens(kva):
    n = 8192
    Batch(251, [(i * 7) % 5 for i in range(n)], [(i * 13) % 40 for i in range(n)], 8).run(kva)
