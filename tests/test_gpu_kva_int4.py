"""The calls on a cache held in 4 bits against their 64-bit evaluations (GPU)."""
import math

import pytest
import torch

import kva_int4_reference as Q
import kva_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def lengths(*total):
    """One new token per request, contexts of `total` positions."""
    return [1] * len(total), [n - 1 for n in total]


SHORT = lengths(1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 200)


# ------------------------------------------------------------------ attention

class Call:
    """A batch with everything a call needs on the device."""

    def __init__(self, kva, c, q_heads, *, softcap=0.0, window=0, alibi=False, q_std=2.0, q_pad=0,
                 sm_scale=None, q=None):
        self.kva, self.c, self.heads = kva, c, q_heads
        self.scale = 1 / math.sqrt(c.head) if sm_scale is None else sm_scale
        self.q = c.normal(c.T, q_heads, c.head, std=q_std) if q is None else q
        self.softcap, self.window, self.slopes = softcap, window, None
        if alibi:
            self.slopes = 2.0 ** (-8.0 * torch.arange(1, q_heads + 1).float() / q_heads)
        self.cache, self.scales, self.keep = c.on()
        wide = torch.full((c.T, q_heads * c.head + q_pad), float("nan"), dtype=torch.bfloat16)
        wide[:, :q_heads * c.head] = self.q.reshape(c.T, -1)
        self.dq = wide.cuda()
        self.out = torch.full(self.q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full(self.q.shape[:2], 7.0, device="cuda")
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        n = kva.kva_gqa_decode_workspace(q_heads, c.kv_heads, c.head)
        self.space = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN patterns
        self.ds = None if self.slopes is None else self.slopes.cuda()

    def call(self, stream=None, space=None):
        self.kva.kva_gqa_decode_int4(
            self.out, self.dq, self.keep[4], self.cache, self.scales, self.c.layer, self.scale,
            self.space if space is None else space, lse=self.lse, softcap=self.softcap,
            window=self.window, alibi_slopes=self.ds, err_flags=self.flags, stream=stream,
            num_q_heads=self.heads)

    def check(self, flags=0):
        torch.cuda.synchronize()
        c = self.c
        out, lse, to, tl = Q.gqa(c, self.q, self.scale, self.softcap, self.window, self.slopes)
        assert int(self.flags) == flags
        R.check(self.out, out, to, "out")
        R.check(self.lse, lse, tl, "lse")
        # The cuts of the products bound an element loosely.  Of the whole, the
        # result's rounding is 2^-8 at most, a weight's 2^-11, and 17 cuts of 2^-13
        # of a code in one direction, on values of a code and more, 2^-9.
        if float(out.norm()):
            R.check_norm(self.out, out, 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -9, "out")
        assert torch.equal(self.keep[0].cpu(), c.code_store)
        assert torch.equal(self.keep[1].cpu().view(torch.int16), c.scale_store.view(torch.int16))
        return out


def run(kva, c, q_heads, *, flags=0, **kw):
    x = Call(kva, c, q_heads, **kw)
    x.call()
    out = x.check(flags)
    return x, out


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(2, 2), (8, 2), (15, 3), (24, 2)])
def test_short_contexts(kva, head, q_heads, kv_heads):
    run(kva, Q.Int4(130, *SHORT, kv_heads=kv_heads, head=head).fill(), q_heads)


@pytest.mark.parametrize("head", [64, 128])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (16, 1), (17, 1), (40, 1), (71, 1)])
def test_group_sizes(kva, head, q_heads, kv_heads):
    run(kva, Q.Int4(131, *lengths(3, 70, 130), kv_heads=kv_heads, head=head).fill(), q_heads)


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 192])
def test_page_sizes_and_strides(kva, head, page):
    run(kva, Q.Int4(132, *SHORT, kv_heads=2, head=head, page=page, head_pad=2, page_pad=3).fill(),
        4, q_pad=8)


@pytest.mark.parametrize("head", [64, 96, 128, 256])
def test_several_new_tokens(kva, head):
    c = Q.Int4(133, [3, 0, 7, 1, 2, 0, 66], [0, 4, 60, 0, 126, 3, 31], kv_heads=2, head=head).fill()
    run(kva, c, 4)
    run(kva, c, 4, window=20)


@pytest.mark.parametrize("softcap,window,alibi", [
    (5.0, 0, False), (50.0, 0, False), (0.0, 1, False), (0.0, 2, False), (0.0, 64, False),
    (0.0, 65, False), (0.0, 100, False), (0.0, 1 << 30, False), (0.0, 0, True), (3.0, 40, True)])
@pytest.mark.parametrize("head,q_heads", [(64, 8), (128, 24), (256, 4)])
def test_modifiers(kva, head, q_heads, softcap, window, alibi):
    c = Q.Int4(134, [1, 2, 1, 1, 1, 3], [0, 62, 63, 64, 130, 300], kv_heads=2, head=head).fill()
    run(kva, c, q_heads, softcap=softcap, window=window, alibi=alibi, q_std=4.0)


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads", [5, 12])
def test_one_long_context_over_many_pieces(kva, head, q_heads):
    x, want = run(kva, Q.Int4(135, [1], [20000], kv_heads=1, head=head, layers=1, layer=0,
                              page=64).fill(), q_heads)
    # two independent roundings (weights, result) of at most 2^-8 each
    R.check_norm(x.out, want, math.sqrt(2) * 2.0 ** -8)


def test_mixed_lengths(kva):
    run(kva, Q.Int4(136, *lengths(5000, 3, 900, 1, 64, 2222), head=128, layers=1, layer=0).fill(), 8)


def test_many_requests(kva):
    n = 1500
    new = [(i * 7) % 3 for i in range(n)]
    run(kva, Q.Int4(137, new, [(i * 13) % 40 for i in range(n)], kv_heads=1, head=64).fill(), 1)


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("q_heads", [2, 16])
def test_rising_scores_move_the_reference(kva, sign, q_heads):
    c = Q.Int4(138, [1], [999], kv_heads=1, head=64, layers=1, layer=0).fill()
    k = torch.zeros(1000, 1, 64)
    k[:, 0, 0] = sign * torch.arange(1000.0) / 16
    c.put(0, 0, 0, *Q.held(k))
    q = torch.full((1, q_heads, 64), 4.0).bfloat16()
    run(kva, c, q_heads, q=q, sm_scale=1.0)


@pytest.mark.parametrize("powers", [(-120, 60), (60, -120), (0, 90), (-30, -60), (0, 0)])
@pytest.mark.parametrize("head,q_heads", [(64, 2), (128, 16), (256, 4)])
def test_value_scales_far_apart(kva, powers, head, q_heads):
    """Values whose scales rise or fall by many powers of two along the
    context: the weights' reference follows them."""
    c = Q.Int4(139, *lengths(700, 90, 33), kv_heads=1, head=head).fill()
    for b in range(3):
        n = c.prior[b] + 1
        ids, row = c.place(b, 0, n)
        e = torch.linspace(powers[0], powers[1], n).round()
        x = c.scales[ids, 1, c.layer, :, :, row].double() * 2.0 ** e.double()[:, None, None]
        c.scales[ids, 1, c.layer, :, :, row] = x.bfloat16()
    run(kva, c, q_heads)


def test_zero_scales(kva):
    """Keys, values, or both of some positions are all zero."""
    c = Q.Int4(140, *lengths(100, 70, 64), kv_heads=2, head=128).fill()
    for b, plane, lo, hi in ((0, 1, 0, 40), (0, 0, 20, 60), (1, 1, 0, 70), (2, 0, 0, 64)):
        ids, row = c.place(b, lo, hi)
        c.scales[ids, plane, c.layer, :, :, row] = 0
    run(kva, c, 8)


def test_wide_range_queries(kva):
    c = Q.Int4(141, *lengths(40, 70), kv_heads=1, head=64).fill()
    q = c.normal(2, 4, 64)
    q[:, 0] *= 2.0 ** 40
    q[:, 1] *= 2.0 ** -40
    q[:, 2] = 0
    run(kva, c, 4, q=q, sm_scale=2.0 ** -41)


def test_a_far_larger_weight_leaves_the_others(kva):
    """One position 18 above 8191 others, whose values all differ from its own."""
    c = Q.Int4(142, [1], [8191], kv_heads=1, head=64, layers=1, layer=0).fill()
    k = torch.zeros(8192, 1, 64)
    k[0, 0, 0] = 7.0
    c.put(0, 0, 0, *Q.held(k))
    v = torch.ones(8192, 1, 64)
    v[0] = 2.0 ** -10
    c.put(0, 1, 0, *Q.held(v))
    q = torch.zeros(1, 2, 64)
    q[:, :, 0] = 18.0 / 7.0
    run(kva, c, 2, q=q.bfloat16(), sm_scale=1.0)


def test_invalid_pages_are_masked(kva):
    c = Q.Int4(143, *lengths(100, 33, 200), kv_heads=2, head=64, page=16).fill()
    c.table[0, 2] = R.UNMAPPED
    c.table[2, 0] = c.pages + 5
    c.table[2, 12] = R.UNMAPPED  # the last page: the token's own row
    run(kva, c, 4, flags=1)


def test_invalid_whole_tiles_are_masked(kva):
    c = Q.Int4(144, *lengths(300, 64, 200), kv_heads=2, head=128, page=64).fill()
    c.table[0, 1] = R.UNMAPPED
    c.table[2, 3] = c.pages
    run(kva, c, 4, flags=1)


@pytest.mark.parametrize("window", [0, 8])
def test_rows_left_without_positions(kva, window):
    c = Q.Int4(145, *lengths(30, 20, 300), kv_heads=2, head=64, page=16).fill()
    c.table[1, :] = R.UNMAPPED
    if window:
        c.table[2, 18] = R.UNMAPPED  # positions 288.. : all that the window of 300 sees
    x, _ = run(kva, c, 4, flags=1, window=window)
    assert bool((x.out[1] == 0).all())


@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("window", [0, 5, 40])
def test_contexts_past_the_page_table(kva, window, page):
    c = Q.Int4(146, [2, 1], [page * 6 - 6, 10], kv_heads=1, head=64, page=page).fill()
    c.table = c.table[:, :3].contiguous()
    run(kva, c, 2, flags=1, window=window)


@pytest.mark.parametrize("length", [0x7FFFFFFF, 0x80000000, 0xFFFFFFFF])
@pytest.mark.parametrize("page", [16, 64])
def test_the_longest_lengths(kva, length, page):
    """Positions past the page table have no page: what the table reaches is
    seen, and the flag set."""
    x, _ = run(kva, Q.Int4(147, *lengths(192, 31), page=page, table_extra=0).fill(), 4)
    all_seen = x.out.clone()
    x.keep[3][0] = length - (1 << 32) if length >> 31 else length
    x.out.fill_(7.0)
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 1 and torch.equal(x.out, all_seen)


@pytest.mark.parametrize("offsets", [[1, 2, 3], [0, 1, 2], [0, 4, 3], [0, 1, 9]])
def test_malformed_offsets_write_nothing(kva, offsets):
    x = Call(kva, Q.Int4(148, [1, 2], [50, 60], kv_heads=1).fill(), 2)
    x.keep[4].copy_(torch.tensor(offsets, dtype=torch.int32))
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 4
    assert bool((x.out == 7.0).all()) and bool((x.lse == 7.0).all())


@pytest.mark.parametrize("q_heads", [4, 16])
def test_nan_propagates_to_who_sees_it(kva, q_heads):
    """A key scale that is NaN makes the rows that see it NaN, a value scale
    its group's columns; rows before it and other requests stay."""
    c = Q.Int4(149, [3, 1, 1], [40, 80, 33], kv_heads=1, head=128).fill()
    x = Call(kva, c, q_heads)
    x.call()
    torch.cuda.synchronize()
    clean = x.out.clone()
    ids, row = c.place(0, 41, 42)  # seen by the second and third new token
    c.scales[ids, 1, c.layer, 0, 1, row] = float("nan")
    ids, row = c.place(1, 7, 8)
    c.scales[ids, 0, c.layer, 0, 0, row] = float("nan")
    y = Call(kva, c, q_heads, q=x.q)
    y.call()
    torch.cuda.synchronize()
    nan = torch.isnan(y.out)
    assert bool(nan[1:3, :, 64:].all()) and not bool(nan[1:3, :, :64].any())
    assert bool(nan[3].all())
    for t in (0, 4):
        assert torch.equal(y.out[t], clean[t])
    assert torch.equal(y.out[1:3, :, :64], clean[1:3, :, :64])


def test_infinite_queries(kva):
    x = Call(kva, Q.Int4(150, *lengths(40, 40), kv_heads=1).fill(), 2)
    q = x.q.clone()
    q[0, 1, 5] = float("inf")
    y = Call(kva, x.c, 2, q=q)
    x.call()
    y.call()
    torch.cuda.synchronize()
    assert bool(torch.isnan(y.out[0, 1]).all())
    y.out[0, 1] = x.out[0, 1]
    assert torch.equal(x.out, y.out)


def test_equal_calls_give_equal_bits(kva):
    x = Call(kva, Q.Int4(151, *lengths(5000, 3, 900, 1, 64, 2222), head=128, layers=1,
                         layer=0).fill(), 8)
    x.call()
    first = x.out.clone()
    for _ in range(3):
        x.space.random_(0, 256)
        x.call()
        assert torch.equal(x.out, first)


# ------------------------------------------------------------------ append

def append(kva, c, q_heads, *, rope=None, gammas=False, interleaved=False, position_ids=None,
           mrope=None, qkv=None, flags=0, q_std=1.0, in_place=False, weight_offset=0.0):
    rope = c.head if rope is None else rope
    rows = q_heads + 2 * c.kv_heads
    if qkv is None:
        qkv = c.normal(c.T, rows * c.head, std=q_std)
    freqs = R.freqs_table(512, rope) if rope else None
    g = [(1 + 0.1 * torch.randn(c.head, generator=c.gen)).bfloat16() if gammas else None
         for _ in range(2)]
    want, err = R.append(c, qkv, q_heads, freqs, q_gamma=g[0], k_gamma=g[1],
                         position_ids=position_ids, mrope_section=mrope, interleaved=interleaved,
                         weight_offset=weight_offset)
    cache, scales, keep = c.on()
    dev = lambda x: None if x is None else x.cuda()
    dqkv = qkv.cuda()
    q = dqkv if in_place else torch.full((c.T, q_heads, c.head), 7.0, dtype=torch.bfloat16,
                                         device="cuda")
    fl = torch.zeros(1, dtype=torch.int32, device="cuda")
    kva.kva_append_qkv_int4(q if q_heads else None, dqkv, keep[4], cache, scales, dev(freqs),
                            c.layer, q_gamma=dev(g[0]), k_gamma=dev(g[1]),
                            weight_offset=weight_offset, position_ids=dev(position_ids),
                            mrope_section=mrope, interleaved=interleaved, err_flags=fl,
                            num_q_heads=q_heads)
    torch.cuda.synchronize()
    assert int(fl) == flags
    if in_place:
        q = q[:, :q_heads * c.head].reshape(c.T, q_heads, c.head)
    before = c.code_store.clone(), c.scale_store.clone()
    c.see(keep[0], keep[1])
    return q, want, err, before, keep, (cache, scales)


def check_append(c, q, want, err, before):
    if q.shape[1]:
        R.check(q, want[0], R.HALF_STEP[R.BF16] * want[0].abs() * (1 + 2.0 ** -8) + err[0], "q")
    written = [torch.zeros_like(x, dtype=torch.bool) for x in before]
    views = [torch.as_strided(w, *sh) for w, sh in zip(
        written, ((c.code_shape, c.code_stride), (c.scale_shape, c.scale_stride)))]
    for t, b, pos in c.tokens():
        page, row = int(c.table[b, pos // c.page]), pos % c.page
        if not 0 <= page < c.pages:
            continue
        for plane in range(2):
            Q.check_held(Q.unpack(c.codes[page, plane, c.layer, :, row]),
                         c.scales[page, plane, c.layer, :, :, row], want[1 + plane][t],
                         err[1 + plane][t], "kv"[plane])
            views[0][page, plane, c.layer, :, row] = True
            views[1][page, plane, c.layer, :, :, row] = True
    # nothing else is touched
    assert torch.equal(c.code_store[~written[0]], before[0][~written[0]])
    assert torch.equal(c.scale_store.view(torch.int16)[~written[1]],
                       before[1].view(torch.int16)[~written[1]])


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("q_heads,kv_heads", [(4, 2), (3, 1), (0, 5)])
@pytest.mark.parametrize("gammas", [False, True])
def test_append(kva, head, q_heads, kv_heads, gammas):
    c = Q.Int4(160, [3, 0, 1, 40], [0, 5, 47, 16], kv_heads=kv_heads, head=head, head_pad=1,
               page_pad=1)
    check_append(c, *append(kva, c, q_heads, gammas=gammas)[:4])


@pytest.mark.parametrize("head,rope", [(64, 32), (96, 64), (96, 96), (96, 16), (128, 96), (128, 0),
                                       (256, 64), (256, 208)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_partial_rotation(kva, head, rope, interleaved):
    c = Q.Int4(161, [5, 1], [0, 30], kv_heads=2, head=head, page=48)
    check_append(c, *append(kva, c, 4, rope=rope, interleaved=interleaved, gammas=True,
                            weight_offset=1.0)[:4])


def test_append_positions(kva):
    c = Q.Int4(162, [5, 1, 9], [0, 30, 2], head=128)
    ids = torch.randint(0, 500, (c.T,), generator=c.gen, dtype=torch.int32)
    check_append(c, *append(kva, c, 4, position_ids=ids)[:4])
    c = Q.Int4(162, [5, 1, 9], [0, 30, 2], head=128)
    ids = torch.randint(0, 500, (3, c.T), generator=c.gen, dtype=torch.int32)
    check_append(c, *append(kva, c, 4, position_ids=ids, mrope=(16, 24, 24))[:4])


def test_append_in_place_and_long(kva):
    c = Q.Int4(163, [300, 1, 150], [0, 9, 100], kv_heads=1, head=128)
    check_append(c, *append(kva, c, 2, in_place=True)[:4])


def test_append_bits(kva):
    """Without norms every step is one IEEE operation: the codes and scales of
    the header, bit for bit, over many magnitudes."""
    c = Q.Int4(164, [200, 100], [0, 7], kv_heads=4, head=128, layers=1, layer=0)
    qkv = c.normal(c.T, 8 * 128)
    qkv *= 2.0 ** torch.randint(-120, 100, (c.T, 1), generator=c.gen)
    qkv[5] = 0
    qkv[6, 64:128] = 2.0 ** -133
    qkv[:, 640:704] *= 0
    _, _, _, _, _, _ = append(kva, c, 0, rope=0, qkv=qkv)
    x = qkv.float().view(c.T, 8, 128)
    for t, b, pos in c.tokens():
        page, row = int(c.table[b, pos // c.page]), pos % c.page
        for plane in range(2):
            u, s = Q.held(x[t, 4 * plane:4 * plane + 4])
            assert torch.equal(c.scales[page, plane, 0, :, :, row].view(torch.int16),
                               s.view(torch.int16))
            assert torch.equal(Q.unpack(c.codes[page, plane, 0, :, row]), u)


def test_append_ties_go_to_even(kva):
    c = Q.Int4(165, [1], [0], kv_heads=1, head=64, layers=1, layer=0)
    x = torch.zeros(2, 64)
    x[:, 0] = 7.0  # scale 1
    x[:, 1:15] = torch.arange(-6.5, 7.0, 1.0)
    x[1] *= -2.0 ** -9
    append(kva, c, 0, rope=0, qkv=x.bfloat16().reshape(1, 128))
    want = torch.tensor([-6, -6, -4, -4, -2, -2, 0, 0, 2, 2, 4, 4, 6, 6])
    for plane in range(2):
        u = Q.unpack(c.codes[int(c.table[0, 0]), plane, 0, 0, 0]) - 8
        assert torch.equal(u[1:15], -want if plane else want)


def test_append_nan_and_infinity(kva):
    """They make their own group NaN, and no other."""
    c = Q.Int4(166, [3], [0], kv_heads=1, head=128, layers=1, layer=0)
    qkv = c.normal(3, 256)
    qkv[0, 10] = float("nan")
    qkv[1, 70] = float("inf")
    qkv[2, 128 + 100] = -float("inf")
    append(kva, c, 0, rope=0, qkv=qkv)
    page = int(c.table[0, 0])
    nan = torch.isnan(c.scales[page, :, 0, 0, :, :3])  # plane, group, row
    want = torch.zeros(2, 2, 3, dtype=torch.bool)
    want[0, 0, 0] = want[0, 1, 1] = want[1, 1, 2] = True
    assert torch.equal(nan, want)


def test_append_bad_pages_and_positions(kva):
    c = Q.Int4(167, [4, 1, 3], [14, 60, 0], kv_heads=2, head=64)
    c.table[0, 1] = R.UNMAPPED
    c.table[2, 0] = c.pages
    check_append(c, *append(kva, c, 3, flags=1)[:4])


def test_append_malformed_offsets(kva):
    c = Q.Int4(168, [1, 2], [5, 6])
    cache, scales, keep = c.on()
    keep[4].copy_(torch.tensor([0, 2, 1], dtype=torch.int32))
    fl = torch.zeros(1, dtype=torch.int32, device="cuda")
    qkv = c.normal(3, 6 * 64).cuda()
    q = torch.full((3, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kva.kva_append_qkv_int4(q, qkv, keep[4], cache, scales, R.freqs_table(64, 64).cuda(), 1,
                            err_flags=fl)
    torch.cuda.synchronize()
    assert int(fl) == 4 and bool((q == 7.0).all())
    assert torch.equal(keep[0].cpu(), c.code_store)


# ------------------------------------------------------------------ gather

def gather(kva, c, counts, first=None, flags=0, k=True, v=True, pad=0):
    """Reads `counts` rows of each request and compares them bit for bit."""
    cache, scales, keep = c.on()
    rows, width = sum(counts), c.kv_heads * c.head
    off = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32).cuda()
    df = None if first is None else torch.tensor(first, dtype=torch.int32).cuda()
    outs = [torch.full((rows, width + pad), 7.0, dtype=torch.bfloat16, device="cuda")
            for _ in range(2)]
    fl = torch.zeros(1, dtype=torch.int32, device="cuda")
    kva.kva_gather_kv_int4(outs[0] if k else None, outs[1] if v else None, off, cache, scales,
                           c.layer, first_positions=df, err_flags=fl)
    torch.cuda.synchronize()
    assert int(fl) == flags
    want = torch.full((2, rows, c.kv_heads, c.head), 7.0, dtype=torch.bfloat16)
    r = 0
    for b, n in enumerate(counts):
        for pos in range(first[b] if first else 0, (first[b] if first else 0) + n):
            page = int(c.table[b, pos // c.page]) if pos // c.page < c.table.shape[1] else -1
            if 0 <= page < c.pages:
                u, s = c.rows(torch.tensor([page]), torch.tensor([pos % c.page]))
                want[:, r] = ((u - 8) * s)[0].bfloat16()
            r += 1
    for i, asked in enumerate((k, v)):
        got = outs[i].cpu()
        assert bool((got[:, width:] == 7.0).all())
        got = got[:, :width].reshape(rows, c.kv_heads, c.head)
        if not asked:
            assert bool((got == 7.0).all())
            continue
        nan = torch.isnan(want[i])
        assert torch.equal(nan, torch.isnan(got))
        assert torch.equal(got[~nan], want[i][~nan])


@pytest.mark.parametrize("head", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 48, 64])
def test_gather(kva, head, page):
    c = Q.Int4(170, [1, 0, 2, 5], [33, 0, 100, 259], kv_heads=3, head=head, page=page, head_pad=1,
               page_pad=2).fill()
    gather(kva, c, [34, 0, 102, 264])
    gather(kva, c, [1, 0, 2, 5], first=[33, 0, 100, 259], pad=8)


@pytest.mark.parametrize("k,v", [(True, False), (False, True)])
def test_gather_one_plane(kva, k, v):
    gather(kva, Q.Int4(171, [1, 1], [20, 70], head=128).fill(), [21, 71], k=k, v=v)


def test_gather_many_requests(kva):
    new = [(i * 7) % 3 for i in range(3000)]
    prior = [(i * 13) % 40 for i in range(3000)]
    gather(kva, Q.Int4(172, new, prior, kv_heads=1).fill(), [n + p for n, p in zip(new, prior)])


def test_gather_bad_pages(kva):
    c = Q.Int4(173, [1, 1], [40, 70]).fill()
    c.table[0, 1] = R.UNMAPPED
    c.table[1, 0] = c.pages + 1
    gather(kva, c, [41, 71], flags=1)
    gather(kva, Q.Int4(173, [1], [40], table_extra=0).fill(), [90], flags=1)  # past the table


def test_gather_positions_past_32_bits(kva):
    c = Q.Int4(174, [1], [40]).fill()
    cache, scales, keep = c.on()
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    first = torch.tensor([-2], dtype=torch.int32, device="cuda")  # 2^32 - 2
    fl = torch.zeros(1, dtype=torch.int32, device="cuda")
    kva.kva_gather_kv_int4(out, None, off, cache, scales, 1, first_positions=first, err_flags=fl)
    torch.cuda.synchronize()
    assert int(fl) == 1 and bool((out == 7.0).all())


def test_gather_malformed_offsets(kva):
    c = Q.Int4(175, [1, 1], [40, 20]).fill()
    cache, scales, keep = c.on()
    for bad in ([0, 30, 61], [1, 30, 60], [0, 70, 60]):
        out = torch.full((60, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        fl = torch.zeros(1, dtype=torch.int32, device="cuda")
        kva.kva_gather_kv_int4(out, None, torch.tensor(bad, dtype=torch.int32, device="cuda"),
                               cache, scales, 1, err_flags=fl)
        torch.cuda.synchronize()
        assert int(fl) == 4 and bool((out == 7.0).all())


@pytest.mark.parametrize("softcap", [2.0 ** -20, 2.0 ** -3, 2.0 ** 20, 2.0 ** 65])
def test_extreme_caps(kva, softcap):
    """A cap far below the scores, far above them, and one that is none."""
    c = Q.Int4(152, *lengths(100, 70, 200), kv_heads=1, head=128).fill()
    x = Call(kva, c, 4, softcap=softcap)
    x.call()
    if softcap > 2.0 ** 64:
        x.softcap = 0.0
    x.check()


def test_slopes_of_either_sign_and_zero(kva):
    c = Q.Int4(153, [1, 3], [150, 64], kv_heads=1, head=64).fill()
    x = Call(kva, c, 4, alibi=True)
    x.slopes = torch.tensor([0.0, -0.125, 0.5, 2.0])
    x.ds.copy_(x.slopes)
    x.call()
    torch.cuda.synchronize()
    out, lse, to, tl = Q.gqa(c, x.q, x.scale, slopes=x.slopes.abs())
    for h in (0, 2, 3):
        R.check(x.out[:, h], out[:, h], to[:, h])
    # the negative one by hand: its tolerance takes the bias's size
    want, _, tol, _ = Q.gqa(c, x.q, x.scale, slopes=x.slopes)
    spread = tol[:, 1] + 2.0 ** -15 * want[:, 1].abs().max()
    R.check(x.out[:, 1], want[:, 1], spread)
