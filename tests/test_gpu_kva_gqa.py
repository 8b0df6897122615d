"""kva_gqa_decode_paged against its 64-bit evaluation (GPU)."""
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


def run(kva, c, q_heads, *, softcap=0.0, window=0, alibi=False, q_std=2.0, q_pad=0, sm_scale=None,
        launch=None, bad_flags=0, q=None):
    if sm_scale is None:
        sm_scale = 1 / math.sqrt(c.head)
    if q is None:
        q = c.normal(c.T, q_heads, c.head, std=q_std)
    slopes = None
    if alibi:
        slopes = 2.0 ** (-8.0 * torch.arange(1, q_heads + 1).float() / q_heads)
    out, lse, to, tl = R.gqa(c, q, sm_scale, softcap, window, slopes)
    desc, store, keep = c.on()
    wide = torch.full((c.T, q_heads * c.head + q_pad), float("nan"), dtype=torch.bfloat16)
    wide[:, :q_heads * c.head] = q.reshape(c.T, -1)
    dq = wide.cuda()
    got = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    got_lse = torch.full(q.shape[:2], 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = kva.kva_gqa_decode_workspace(q_heads, c.kv_heads, c.head)
    space = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
    ds = None if slopes is None else slopes.cuda()

    def call(stream=None):
        kva.kva_gqa_decode_paged(got, dq, keep[3], desc, c.layer, sm_scale, space, lse=got_lse,
                                 v_scale=c.v_scale, softcap=softcap, window=window,
                                 alibi_slopes=ds, err_flags=flags, stream=stream,
                                 num_q_heads=q_heads)

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
@pytest.mark.parametrize("head", [64, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(2, 2), (8, 2), (15, 3)])
def test_short_contexts(kva, dtype, head, q_heads, kv_heads):
    run(kva, R.Paged(30, *SHORT, kv_heads=kv_heads, head=head, dtype=dtype).fill(), q_heads)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("head", [16, 48, 80, 96, 112, 144, 192, 240])
def test_odd_head_sizes(kva, dtype, head):
    run(kva, R.Paged(31, *SHORT, kv_heads=2, head=head, dtype=dtype, page=12).fill(), 6)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (16, 1), (17, 1), (40, 1), (71, 1), (24, 8)])
def test_group_sizes(kva, dtype, q_heads, kv_heads):
    run(kva, R.Paged(32, *lengths(3, 70, 130), kv_heads=kv_heads, head=64, dtype=dtype).fill(),
        q_heads)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("page", [1, 3, 16, 48, 100, 256])
def test_page_sizes_and_strides(kva, dtype, page):
    run(kva, R.Paged(33, *SHORT, kv_heads=2, head=64, dtype=dtype, page=page, head_pad=16,
                     token_pad=32).fill(), 4, q_pad=8)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_several_new_tokens(kva, dtype):
    c = R.Paged(34, [3, 0, 7, 1, 2, 0, 66], [0, 4, 60, 0, 126, 3, 31], kv_heads=2, head=64,
                dtype=dtype).fill()
    run(kva, c, 4)
    run(kva, c, 4, window=20)


@pytest.mark.parametrize("softcap,window,alibi", [
    (5.0, 0, False), (50.0, 0, False), (0.0, 1, False), (0.0, 2, False), (0.0, 64, False),
    (0.0, 65, False), (0.0, 100, False), (0.0, 1 << 30, False), (0.0, 0, True), (3.0, 40, True)])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_modifiers(kva, dtype, softcap, window, alibi):
    c = R.Paged(35, [1, 2, 1, 1, 1, 3], [0, 62, 63, 64, 130, 300], kv_heads=2, head=64,
                dtype=dtype).fill()
    run(kva, c, 8, softcap=softcap, window=window, alibi=alibi, q_std=4.0)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_one_long_context_over_many_pieces(kva, dtype, head):
    got, want = run(kva, R.Paged(36, [1], [20000], kv_heads=1, head=head, dtype=dtype, layers=1,
                                 layer=0, page=64).fill(), 5)
    # two independent roundings (weights, result) of at most 2^-8 each
    R.check_norm(got, want, math.sqrt(2) * 2.0 ** -8)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_mixed_lengths_norm(kva, dtype):
    got, want = run(kva, R.Paged(37, *lengths(5000, 3, 900, 1, 64, 2222), kv_heads=2, head=128,
                                 dtype=dtype, layers=1, layer=0).fill(), 8)
    R.check_norm(got, want, math.sqrt(2) * 2.0 ** -8)


def test_many_requests(kva):
    n = 1500
    new = [(i * 7) % 3 for i in range(n)]
    run(kva, R.Paged(38, new, [(i * 13) % 40 for i in range(n)], kv_heads=1, head=16,
                     page=8).fill(), 1)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_rising_scores_move_the_maximum(kva, dtype):
    """Keys that grow along the context make every slice raise the maximum;
    falling ones leave it at the first."""
    for sign in (1.0, -1.0):
        c = R.Paged(39, [1], [999], kv_heads=1, head=64, dtype=dtype, layers=1, layer=0).fill()
        at = torch.arange(1000)
        k = torch.zeros(1000, 1, 64)
        k[:, 0, 0] = sign * at.float() / 16
        k = k.bfloat16() if dtype == R.BF16 else \
            (k / c.k_scale).to(torch.float8_e4m3fn).view(torch.uint8)
        c.data[c.table[0].long()[at // c.page], 0, 0, at % c.page] = k
        q = torch.full((1, 2, 64), 4.0).bfloat16()
        run(kva, c, 2, q=q, sm_scale=1.0)


def test_wide_range_queries_in_fp16(kva):
    """An E4M3 cache multiplies in fp16: rows far outside its range, by row."""
    c = R.Paged(40, *lengths(40, 70), kv_heads=1, head=64, dtype=R.E4M3).fill()
    q = c.normal(2, 4, 64)
    q[:, 0] *= 2.0 ** 40
    q[:, 1] *= 2.0 ** -40
    q[:, 2] = 0
    run(kva, c, 4, q=q, sm_scale=2.0 ** -41)


def test_invalid_pages_are_masked(kva):
    c = R.Paged(41, *lengths(100, 33, 200), kv_heads=2, head=64, page=16).fill()
    c.table[0, 2] = R.UNMAPPED
    c.table[2, 0] = c.pages + 5
    c.table[2, 12] = R.UNMAPPED  # the last page: the token's own row
    run(kva, c, 4, bad_flags=1)


@pytest.mark.parametrize("window", [0, 8])
def test_rows_left_without_positions(kva, window):
    c = R.Paged(42, *lengths(30, 20, 300), kv_heads=2, head=64, page=16).fill()
    c.table[1, :] = R.UNMAPPED
    if window:
        c.table[2, 18] = R.UNMAPPED  # positions 288.. : all that the window of 300 sees
    got, _ = run(kva, c, 4, bad_flags=1, window=window)
    assert bool((got[1] == 0).all())


@pytest.mark.parametrize("window", [0, 5, 40])
def test_contexts_past_the_page_table(kva, window):
    c = R.Paged(43, [2, 1], [90, 10], kv_heads=1, head=64, page=16).fill()
    c.table = c.table[:, :3].contiguous()  # 48 positions; window 5 and 40 of 91: 51.. and 52..
    run(kva, c, 2, bad_flags=1, window=window)


@pytest.mark.parametrize("offsets", [[1, 2, 3], [0, 1, 2], [0, 4, 3], [0, 1, 9]])
def test_malformed_offsets_write_nothing(kva, offsets):
    c = R.Paged(44, [1, 2], [50, 60], kv_heads=1, head=64).fill()
    desc, store, keep = c.on()
    q = c.normal(3, 2, 64).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((3, 2), 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.full((kva.kva_gqa_decode_workspace(2, 1, 64),), 0xFF, dtype=torch.uint8,
                       device="cuda")
    bad = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    kva.kva_gqa_decode_paged(out, q, bad, desc, c.layer, 0.1, space, lse=lse, err_flags=flags)
    assert int(flags) == 4
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_nan_and_infinity_propagate(kva):
    c = R.Paged(45, *lengths(40, 40, 40), kv_heads=1, head=64).fill()
    at = 20
    page, row = int(c.table[1, at // c.page]), at % c.page
    c.data[page, 1, c.layer, row, 0, 3] = float("inf")  # a value: column 3 of request 1
    page = int(c.table[2, at // c.page])
    c.data[page, 0, c.layer, row, 0, 3] = float("nan")  # a key: all of request 2
    desc, store, keep = c.on()
    q = c.normal(3, 2, 64).cuda()
    out = torch.zeros_like(q)
    space = torch.empty(kva.kva_gqa_decode_workspace(2, 1, 64), dtype=torch.uint8, device="cuda")
    kva.kva_gqa_decode_paged(out, q, keep[3], desc, c.layer, 0.1, space)
    assert bool(torch.isfinite(out[0]).all())
    assert bool(torch.isinf(out[1, :, 3]).all())
    assert bool(torch.isfinite(out[1, :, [0, 1, 2, 4, 63]]).all())
    assert bool(torch.isnan(out[2]).all())


def test_equal_calls_give_equal_bits(kva):
    c = R.Paged(46, *lengths(3000, 70, 999), kv_heads=2, head=128, layers=1, layer=0).fill()
    q = c.normal(3, 8, 128)
    first, _ = run(kva, c, 8, q=q)
    for _ in range(3):
        again, _ = run(kva, c, 8, q=q)
        assert torch.equal(first, again)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("window", [0, 3])
def test_a_later_tokens_row_does_not_reach_an_earlier_one(kva, dtype, window):
    """Tokens of a request share a pass over the cache: the row of the last one
    is NaN, and with a window so is the first position that only the first
    token sees."""
    c = R.Paged(47, [4, 1], [61, 5], kv_heads=1, head=64, dtype=dtype, page=8).fill()
    nan = float("nan") if dtype == R.BF16 else 0x7F
    at = [64] + ([61 + 1 - window] if window else [])
    for p in at:
        c.data[int(c.table[0, p // 8]), 1, c.layer, p % 8, 0] = nan
    desc, store, keep = c.on()
    q = c.normal(5, 4, 64).cuda()
    out = torch.zeros_like(q)
    space = torch.empty(kva.kva_gqa_decode_workspace(4, 1, 64), dtype=torch.uint8, device="cuda")
    kva.kva_gqa_decode_paged(out, q, keep[3], desc, c.layer, 0.1, space, window=window,
                             v_scale=c.v_scale)
    bad = torch.isnan(out).all(-1).all(-1).tolist()
    some = torch.isnan(out).any(-1).any(-1).tolist()
    assert bad == some == [bool(window), False, False, True, False]


# tiles within a page are fed in a way of their own
WHOLE = [64, 128, 192]


@pytest.mark.parametrize("softcap,window,alibi", [
    (0.0, 0, False), (5.0, 0, False), (0.0, 1, False), (0.0, 65, False), (0.0, 100, True),
    (3.0, 200, True)])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("q_heads", [8, 24])
def test_whole_pages_with_modifiers(kva, dtype, q_heads, softcap, window, alibi):
    for page in WHOLE:
        c = R.Paged(50, [1, 2, 1, 0, 1, 9], [0, 62, 63, 7, 130, 500], kv_heads=2, head=64,
                    dtype=dtype, page=page).fill()
        run(kva, c, q_heads, softcap=softcap, window=window, alibi=alibi, q_std=4.0)


@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_whole_pages_that_are_not_valid(kva, dtype, window):
    for page in WHOLE:
        c = R.Paged(51, *lengths(3 * page, 33, 2 * page + 7, 20), kv_heads=2, head=64, dtype=dtype,
                    page=page).fill()
        c.table[0, 2 if window else 1] = R.UNMAPPED
        c.table[2, 0] = c.pages + 5
        c.table[2, 2] = R.UNMAPPED  # the last page: the token's own row
        c.table[3, :] = R.UNMAPPED  # nothing left
        got, _ = run(kva, c, 4, bad_flags=1, window=window)
        assert bool((got[3] == 0).all())


@pytest.mark.parametrize("window", [0, 70])
def test_contexts_past_a_table_of_whole_pages(kva, window):
    c = R.Paged(52, [2, 1], [290, 10], kv_heads=1, head=64, page=64).fill()
    c.table = c.table[:, :3].contiguous()  # 192 positions
    run(kva, c, 2, bad_flags=1, window=window)


@pytest.mark.parametrize("q_heads,kv_heads", [(5, 5), (28, 7), (16, 16), (34, 2), (51, 3)])
@pytest.mark.parametrize("page", [16, 64])
def test_heads_side_by_side(kva, q_heads, kv_heads, page):
    c = R.Paged(53, [1, 3, 1, 1], [2000, 70, 64, 700], kv_heads=kv_heads, head=64, page=page,
                layers=1, layer=0).fill()
    run(kva, c, q_heads)


@pytest.mark.parametrize("softcap", [1e-38, 1e-3, 1000.0])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_extreme_caps(kva, dtype, softcap):
    """A tiny cap makes every weight nearly the same, a huge one changes little."""
    c = R.Paged(54, *lengths(3, 130), kv_heads=1, head=64, dtype=dtype).fill()
    q = c.normal(2, 4, 64)
    q[:, 0] = 0  # scores of 0
    run(kva, c, 4, q=q, softcap=softcap)


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("low", [-110, -113, -116, -119])
def test_tiny_queries_and_a_large_scale(kva, dtype, low):
    c = R.Paged(55, *lengths(3, 70, 130), kv_heads=1, head=64, dtype=dtype).fill()
    run(kva, c, 4, q=c.normal(3, 4, 64, std=2.0 ** low), sm_scale=2.0 ** (-2 - low))
