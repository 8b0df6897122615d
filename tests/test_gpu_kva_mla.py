"""kva_mla_decode_paged against its 64-bit evaluation (GPU)."""
import math

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


def batch(seed, new, prior, **kw):
    kw.setdefault("page", 16)
    return R.Paged(seed, new, prior, kv_heads=1, head=576, planes=1, **kw).fill()


def run(kva, c, heads, *, sm_scale=1 / math.sqrt(192), q_std=1.2, pad=(0, 0), q=None, launch=None,
        bad_flags=0):
    if q is None:
        q = c.normal(c.T, heads, 512, std=q_std), c.normal(c.T, heads, 64, std=q_std)
    out, lse, to, tl = R.mla(c, *q, sm_scale)
    desc, store, keep = c.on()
    dq = []
    for x, extra in zip(q, pad):
        wide = torch.full((c.T, x[0].numel() + extra), float("nan"), dtype=torch.bfloat16)
        wide[:, :x[0].numel()] = x.reshape(c.T, -1)
        dq.append(wide.cuda())
    got = torch.full((c.T, heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    got_lse = torch.full((c.T, heads), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_mla_decode_workspace(heads),), 0xFF, dtype=torch.uint8,
                       device="cuda")  # NaN patterns

    def call(stream=None):
        kva.kva_mla_decode_paged(got, dq[0], dq[1], keep[3], desc, c.layer, sm_scale, space,
                                 lse=got_lse, err_flags=flags, stream=stream, num_heads=heads)

    (launch or (lambda f: f()))(call)
    torch.cuda.synchronize()
    assert int(flags) == bad_flags
    R.check(got, out, to, "out")
    R.check(got_lse, lse, tl, "lse")
    assert torch.equal(store.cpu().view(torch.uint8), c.store.view(torch.uint8))
    return got, out


def lengths(*total):
    """One new token per request, contexts of `total` positions."""
    return [1] * len(total), [n - 1 for n in total]


SHORT = lengths(1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [64, 16, 128])
def test_short_contexts(kva, dtype, heads):
    run(kva, batch(60, *SHORT, dtype=dtype), heads)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [1, 3, 17, 40, 63, 65, 130, 200])
def test_head_counts(kva, dtype, heads):
    run(kva, batch(61, *lengths(3, 70, 130), dtype=dtype), heads)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [1, 3, 48, 100, 256])
def test_page_sizes_and_strides(kva, dtype, page):
    run(kva, batch(62, *SHORT, dtype=dtype, page=page, head_pad=16, token_pad=32), 16,
        pad=(8, 16))


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_several_new_tokens(kva, dtype):
    run(kva, batch(63, [3, 0, 7, 1, 2, 0, 66], [0, 4, 60, 0, 126, 3, 31], dtype=dtype), 16)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [16, 128])
def test_one_long_context_over_many_pieces(kva, dtype, heads):
    got, want = run(kva, batch(64, [1], [14000], dtype=dtype, layers=1, layer=0, page=64), heads)
    # two independent roundings (weights, result) of at most 2^-8 each
    R.check_norm(got, want, math.sqrt(2) * 2.0 ** -8)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_mixed_lengths_norm(kva, dtype):
    got, want = run(kva, batch(65, *lengths(5000, 3, 900, 1, 64, 2222), dtype=dtype, layers=1,
                               layer=0), 128)
    R.check_norm(got, want, math.sqrt(2) * 2.0 ** -8)


def test_many_requests(kva):
    n = 700
    new = [(i * 7) % 3 for i in range(n)]
    run(kva, batch(66, new, [(i * 13) % 40 for i in range(n)], page=8), 8)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_rising_scores_move_the_maximum(kva, dtype):
    """Rows that grow along the context make every tile raise the maximum by
    more than the slack; falling ones leave it at the first."""
    for sign in (1.0, -1.0):
        c = batch(67, [1], [999], dtype=dtype, layers=1, layer=0)
        at = torch.arange(1000)
        k = c.rows(0, 0, 0, 1000)[:, 0]
        k[:, 0] = sign * at.double() / 8
        k = k.float().bfloat16() if dtype == R.BF16 else \
            (k / c.k_scale).float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        c.data[c.table[0].long()[at // c.page], 0, 0, at % c.page, 0] = k
        q = torch.zeros(1, 20, 512), torch.zeros(1, 20, 64)
        q[0][:, :, 0] = torch.linspace(0.0, 4.0, 20)
        run(kva, c, 20, q=(q[0].bfloat16(), q[1].bfloat16()), sm_scale=1.0)


def test_wide_range_queries_in_fp16(kva):
    """An E4M3 cache multiplies in fp16: rows far outside its range, by row."""
    c = batch(68, *lengths(40, 70), dtype=R.E4M3)
    q = c.normal(2, 4, 512), c.normal(2, 4, 64)
    for x in q:
        x[:, 0] *= 2.0 ** 40
        x[:, 1] *= 2.0 ** -40
        x[:, 2] = 0
    run(kva, c, 4, q=q, sm_scale=2.0 ** -42)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_invalid_pages_are_masked(kva, dtype):
    c = batch(69, *lengths(100, 33, 200, 20), dtype=dtype)
    c.table[0, 2] = R.UNMAPPED
    c.table[2, 0] = c.pages + 5
    c.table[2, 12] = R.UNMAPPED  # the last page: the token's own row
    c.table[3, :] = R.UNMAPPED   # nothing left
    got, _ = run(kva, c, 16, bad_flags=1)
    assert bool((got[3] == 0).all())


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_contexts_past_the_page_table(kva, dtype):
    c = batch(70, [2, 1], [90, 10], dtype=dtype)
    c.table = c.table[:, :3].contiguous()
    run(kva, c, 16, bad_flags=1)


@pytest.mark.parametrize("offsets", [[1, 2, 3], [0, 1, 2], [0, 4, 3], [0, 1, 9]])
def test_malformed_offsets_write_nothing(kva, offsets):
    c = batch(71, [1, 2], [50, 60])
    desc, store, keep = c.on()
    ql, qr = c.normal(3, 4, 512).cuda(), c.normal(3, 4, 64).cuda()
    out, lse = torch.full_like(ql, 7.0), torch.full((3, 4), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_mla_decode_workspace(4),), 0xFF, dtype=torch.uint8, device="cuda")
    bad = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    kva.kva_mla_decode_paged(out, ql, qr, bad, desc, c.layer, 0.1, space, lse=lse, err_flags=flags)
    assert int(flags) == 4
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_nan_propagates_and_stays_in_its_request(kva):
    c = batch(72, *lengths(40, 40, 40))
    at = 20
    page, row = int(c.table[1, at // c.page]), at % c.page
    c.data[page, 0, c.layer, row, 0, 3] = float("nan")
    desc, store, keep = c.on()
    ql, qr = c.normal(3, 4, 512).cuda(), c.normal(3, 4, 64).cuda()
    ql[2, 1, 5] = float("inf")
    out = torch.zeros_like(ql)
    space = torch.empty(kva.kva_mla_decode_workspace(4), dtype=torch.uint8, device="cuda")
    kva.kva_mla_decode_paged(out, ql, qr, keep[3], desc, c.layer, 0.1, space)
    assert bool(torch.isfinite(out[0]).all())
    assert bool(torch.isnan(out[1]).all())
    assert bool(torch.isnan(out[2, 1]).all())
    assert bool(torch.isfinite(out[2, [0, 2, 3]]).all())


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_equal_calls_give_equal_bits(kva, dtype):
    c = batch(73, *lengths(3000, 70, 999), dtype=dtype, layers=1, layer=0)
    q = c.normal(3, 128, 512), c.normal(3, 128, 64)
    first, _ = run(kva, c, 128, q=q)
    for _ in range(3):
        again, _ = run(kva, c, 128, q=q)
        assert torch.equal(first, again)


# tiles within a page are copied in a way of their own
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("page", [64, 128, 192])
def test_whole_pages(kva, dtype, heads, page):
    run(kva, batch(74, [1, 2, 1, 0, 1, 3], [0, 62, 63, 7, 130, 500], dtype=dtype, page=page,
                   head_pad=16, token_pad=32), heads, pad=(8, 16))


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [64, 128])
def test_whole_pages_that_are_not_valid(kva, dtype, page):
    c = batch(75, *lengths(3 * page, 33, 2 * page + 7, 20), dtype=dtype, page=page)
    c.table[0, 1] = R.UNMAPPED
    c.table[2, 0] = c.pages + 5
    c.table[2, 2] = R.UNMAPPED  # the last page: the token's own row
    c.table[3, :] = R.UNMAPPED  # nothing left
    got, _ = run(kva, c, 16, bad_flags=1)
    assert bool((got[3] == 0).all())


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_contexts_past_a_table_of_whole_pages(kva, dtype):
    c = batch(76, [2, 1], [290, 10], dtype=dtype, page=64)
    c.table = c.table[:, :3].contiguous()  # 192 positions
    run(kva, c, 16, bad_flags=1)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("heads", [16, 64])
@pytest.mark.parametrize("page", [16, 64])
def test_last_tile_raises_the_maximum(kva, dtype, heads, page):
    """The token's own row, in the last tile of its segment, lifts the scores of
    most heads far above those before: O^T is rescaled there, and right after it
    the segment's results are taken."""
    n = 400
    total = [65 + (i * 37) % 190 for i in range(n)]
    c = batch(77, *lengths(*total), dtype=dtype, page=page, layers=1, layer=0)
    for b in range(n):
        p = total[b] - 1
        row = c.data[int(c.table[b, p // page]), 0, 0, p % page, 0]
        row[0] = 60.0 if dtype == R.BF16 else \
            torch.tensor(60.0 / c.k_scale).to(torch.float8_e4m3fn).view(torch.uint8)
    q = c.normal(n, heads, 512, std=0.5), c.normal(n, heads, 64, std=0.5)
    q[0][:, :, 0] = torch.linspace(-1.0, 6.0, heads)
    run(kva, c, heads, q=q, sm_scale=0.2)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("low", [-110, -113, -116, -119])
def test_tiny_queries_and_a_large_scale(kva, dtype, low):
    c = batch(78, *lengths(3, 70, 130), dtype=dtype)
    q = c.normal(3, 16, 512, std=2.0 ** low), c.normal(3, 16, 64, std=2.0 ** low)
    run(kva, c, 16, q=q, sm_scale=2.0 ** (-4 - low))
