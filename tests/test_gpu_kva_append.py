"""kva_append_qkv_paged against its 64-bit evaluation (GPU)."""
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


def run(kva, c, q_heads, *, rope=None, norm=(False, False), position=None, interleaved=False,
        qkv_pad=0, in_place=False, weight_offset=0.0, eps=1e-6, std=1.0, launch=None,
        bad_flags=0):
    rope = c.head if rope is None else rope
    rows = q_heads + 2 * c.kv_heads
    qkv = c.normal(c.T, rows * c.head + qkv_pad, std=std)
    top = max([p + n for p, n in zip(c.prior, c.new)] + [1])
    freqs = R.freqs_table(max(top, 64), rope) if rope else None
    gq = (c.normal(c.head, std=0.1) + 1).bfloat16() if norm[0] else None
    gk = (c.normal(c.head, std=0.1) + 1).bfloat16() if norm[1] else None
    ids = sec = None
    if position == "ids":
        ids = torch.randint(0, 64, (c.T,), generator=c.gen, dtype=torch.int32)
    elif position == "mrope":
        ids = torch.randint(0, 64, (3, c.T), generator=c.gen, dtype=torch.int32)
        n = rope // 2
        sec = (n // 4, n // 4 + 3, n - 2 * (n // 4) - 3)
    (q, k, v), (eq, ek, ev) = R.append(c, qkv, q_heads, freqs, q_gamma=gq, k_gamma=gk, eps=eps,
                                       weight_offset=weight_offset, position_ids=ids,
                                       mrope_section=sec, interleaved=interleaved)
    desc, store, keep = c.on()
    before = c.view(store).clone()
    dq = qkv.cuda()
    dev = lambda x: None if x is None else x.cuda()  # noqa: E731
    args = dict(q_gamma=dev(gq), k_gamma=dev(gk), epsilon=eps, weight_offset=weight_offset,
                v_scale=c.v_scale, position_ids=dev(ids), interleaved=interleaved,
                mrope_section=sec, num_q_heads=q_heads)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    if in_place:
        out = dq
    else:
        out = torch.full((c.T, max(q_heads, 1), c.head), 7.0, dtype=torch.bfloat16, device="cuda")
    df = dev(freqs)

    def call(stream=None):
        kva.kva_append_qkv_paged(out, dq, keep[3], desc, df, c.layer, err_flags=flags,
                                 stream=stream, **args)

    (launch or (lambda f: f()))(call)
    torch.cuda.synchronize()
    assert int(flags) == bad_flags
    got_q = out[:, :q_heads * c.head].reshape(c.T, q_heads, c.head) if in_place \
        else out[:, :q_heads]
    if q_heads:
        R.check(got_q, q, R.stored_error(q, eq, R.BF16, 1.0), "queries")
    after = c.view(store)
    touched = torch.zeros(before.shape, dtype=torch.bool)
    for t, b, pos in c.tokens():
        page = int(c.table[b, pos // c.page]) if pos // c.page < c.table.shape[1] else -1
        if not 0 <= page < c.pages:
            continue
        for plane, y, e, s in ((0, k, ek, c.k_scale), (1, v, ev, c.v_scale)):
            at = (page, plane, c.layer, pos % c.page)
            touched[at] = True
            x = after[at]
            x = x.view(torch.float8_e4m3fn).double() if c.dtype == R.E4M3 else x.double()
            want = y[t] if c.dtype == R.BF16 else (y[t] / s).clamp(-448, 448)
            R.check(x, want, R.stored_error(y[t], e[t], c.dtype, s), "plane %d" % plane)
    same = after.view(torch.int16) == before.view(torch.int16) if c.dtype == R.BF16 \
        else after == before
    assert bool((same | touched).all()), "bytes outside the new rows changed"
    return c


BATCHES = {
    "one": ([1], [0]),
    "decode": ([1] * 9, [0, 1, 15, 16, 17, 100, 5, 31, 32]),
    "ragged": ([3, 0, 40, 1, 17], [5, 9, 100, 31, 0]),
}


@pytest.mark.parametrize("batch", sorted(BATCHES))
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [(False, False), (True, True)])
def test_batches(kva, batch, dtype, interleaved, norm):
    run(kva, R.Paged(10, *BATCHES[batch], kv_heads=2, head=128, dtype=dtype), 8,
        interleaved=interleaved, norm=norm)


@pytest.mark.parametrize("head,rope", [(16, 16), (32, 0), (64, 32), (80, 80), (96, 64), (112, 16),
                                       (128, 64), (192, 128), (256, 256), (272, 272), (512, 512),
                                       (512, 96)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_head_sizes(kva, head, rope, interleaved):
    run(kva, R.Paged(11, *BATCHES["ragged"], kv_heads=3, head=head, page=12, dtype=R.E4M3), 5,
        rope=rope, interleaved=interleaved, norm=(True, False))


@pytest.mark.parametrize("position", ["ids", "mrope"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_positions(kva, position, interleaved, dtype):
    run(kva, R.Paged(12, *BATCHES["ragged"], kv_heads=2, head=128, page=100, dtype=dtype), 4,
        rope=96, position=position, interleaved=interleaved, norm=(False, True),
        weight_offset=1.0, eps=0.1)


@pytest.mark.parametrize("q_heads,kv_heads", [(0, 1), (1, 1), (7, 1), (3, 3), (33, 2), (128, 8)])
def test_head_counts(kva, q_heads, kv_heads):
    run(kva, R.Paged(13, [2, 1, 5], [7, 0, 63], kv_heads=kv_heads, head=64, page=8), q_heads)


def test_padded_strides_and_single_token_pages(kva):
    run(kva, R.Paged(14, *BATCHES["ragged"], kv_heads=2, head=64, page=1, head_pad=16,
                     token_pad=48), 4, qkv_pad=24)
    run(kva, R.Paged(15, *BATCHES["ragged"], kv_heads=2, head=64, page=3, head_pad=32,
                     token_pad=16, dtype=R.E4M3), 4, qkv_pad=8)


def test_in_place(kva):
    run(kva, R.Paged(16, *BATCHES["ragged"], kv_heads=2, head=128), 6, in_place=True,
        norm=(True, True))


def test_saturation(kva):
    run(kva, R.Paged(17, *BATCHES["decode"], kv_heads=2, head=64, dtype=R.E4M3, k_scale=1 / 64,
                     v_scale=0.001), 4, std=20.0)


def test_many_requests(kva):
    run(kva, R.Paged(18, [1, 0] * 700, [3] * 1400, kv_heads=1, head=64, page=4), 2)


def test_long_batch_takes_every_pass(kva):
    # enough tokens that an item holds several passes and a warp several items
    run(kva, R.Paged(19, [2500, 1], [0, 3], kv_heads=8, head=16, page=64, layers=1, layer=0), 16)


def test_invalid_pages_and_positions(kva):
    c = R.Paged(20, [4, 3], [14, 2], kv_heads=2, head=64, page=16)
    c.table[0, 1] = R.UNMAPPED  # positions 16, 17 of request 0
    run(kva, c, 4, bad_flags=1)
    c = R.Paged(21, [4, 3], [14, 2], kv_heads=2, head=64, page=16)
    c.table[0, 1] = c.pages
    run(kva, c, 4, bad_flags=1)
    # a table of one column: positions 16, 17 lie past its reach
    c = R.Paged(22, [4, 3], [14, 2], kv_heads=2, head=64, page=16)
    c.table = c.table[:, :1].contiguous()
    run(kva, c, 4, bad_flags=1)


def test_position_past_the_table_leaves_the_token(kva):
    c = R.Paged(23, [4], [2], kv_heads=1, head=64)
    desc, store, keep = c.on()
    before = store.clone()
    qkv = c.normal(4, 4 * 64).cuda()
    out = torch.full((4, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    freqs = R.freqs_table(4, 64).cuda()  # rows 0..3: tokens at 2, 3 fit, 4, 5 do not
    kva.kva_append_qkv_paged(out, qkv, keep[3], desc, freqs, c.layer, err_flags=flags)
    assert int(flags) == 2
    assert bool((out[2:] == 7.0).all()) and not bool((out[:2] == 7.0).all(-1).any())
    a, b = c.view(store), c.view(before)
    page = int(c.table[0, 0])
    assert bool((a[page, :, 1, 2:4] == a[page, :, 1, 2:4]).all())  # written: no NaN left
    assert bool(torch.isnan(a[page, :, 1, 4:]).all()) and bool(torch.isnan(b[page]).all())


@pytest.mark.parametrize("offsets", [[1, 4, 7], [0, 4, 6], [0, 8, 7], [0, 4, 9]])
def test_malformed_offsets_write_nothing(kva, offsets):
    c = R.Paged(24, [4, 3], [2, 0], kv_heads=1, head=64)
    desc, store, keep = c.on()
    qkv = c.normal(7, 4 * 64).cuda()
    out = torch.full((7, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    kva.kva_append_qkv_paged(out, qkv, bad, desc, R.freqs_table(64, 64).cuda(), c.layer,
                             err_flags=flags)
    assert int(flags) == 4
    assert bool((out == 7.0).all()) and bool(torch.isnan(c.view(store)).all())
