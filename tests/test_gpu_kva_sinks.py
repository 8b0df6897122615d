"""Attention over an E4M3 cache where one position takes nearly all the weight
(GPU): what the thousands of others hold, each far below the largest, has to be
in the result.

The weights are rounded to fp16 after a power of two that puts the largest of a
row at 2^9 or above, so each is off by 2^-11 of itself, or, below fp16's
smallest normal, by 2^-25 there: 2^-34 of the largest weight.  The rest of the
tolerance counts the steps of the formula in 32 bits: a score is a sum of d
products, the exponent's argument and value are off by a few 2^-24 of theirs
(2^-20 holds them), and the result is rounded to bf16."""
import pytest
import torch

import kva_reference as R

pytestmark = pytest.mark.gpu

POSITIONS = 8192
REQUESTS = 320  # on the same pages: more than there are CTAs, so that one reads a context


@pytest.fixture(scope="module")
def kva():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gqa_kv_cache_mla_gb300 import kva

    return kva


def check(got, got_lse, q, k, v, width):
    """q [heads, width], k [positions, width], v [positions, columns]."""
    x, size = q @ k.T, (q.abs() @ k.abs().T).max(-1, keepdim=True).values
    top = x.max(-1, keepdim=True).values
    e = torch.exp(x - top)
    total = e.sum(-1, keepdim=True)
    want = e @ v / total
    ds = width * 2.0 ** -24 * size + 2.0 ** -20
    tol = (e @ v.abs() / total) * (2.0 ** -11 * (1 + 2 * ds) + 2 * ds)
    tol = tol + e.clamp(max=2.0 ** -34) @ v.abs() / total
    tol = tol + 2.0 ** -8 * (want.abs() + tol)
    R.check(got, want.expand(got.shape), tol.expand(got.shape), "out")
    lse = (top + torch.log(total))[:, 0]
    allowed = 2 * ds[:, 0] + lse.abs() * 2.0 ** -22
    R.check(got_lse, lse.expand(got_lse.shape), allowed.expand(got_lse.shape), "lse")


def alike(c):
    """The request of `c` many times over: descriptor, offsets, and what keeps them."""
    c.table = c.table.repeat(REQUESTS, 1)
    c.lens = c.lens.repeat(REQUESTS)
    c.offsets = torch.arange(REQUESTS + 1, dtype=torch.int32)
    desc, store, keep = c.on()
    return desc, keep[3], keep


def put(c, plane, at, values):
    scale = c.v_scale if plane else c.k_scale
    codes = (values / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    c.data[c.table[0].long()[at // c.page], plane, c.layer, at % c.page, 0] = codes


@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 18.0, 20.0, 24.0])
@pytest.mark.parametrize("sink", [0, 5000, POSITIONS - 1])
@pytest.mark.parametrize("head,page,biased", [(64, 64, False), (128, 16, False), (256, 64, True)])
def test_gqa(kva, gap, sink, head, page, biased):
    c = R.Paged(110, [1], [POSITIONS - 1], kv_heads=1, head=head, dtype=R.E4M3, page=page,
                layers=1, layer=0)
    k = torch.randn(POSITIONS, head, generator=c.gen) * 0.2
    v = 1 + torch.randn(POSITIONS, head, generator=c.gen)
    k[:, 0] = 0
    k[sink] = 0
    k[sink, 0] = 16
    v[sink] = 0
    put(c, 0, torch.arange(POSITIONS), k)
    put(c, 1, torch.arange(POSITIONS), v)
    q = c.normal(1, 4, head, std=0.1)
    q[:, :, 0] = gap / 16  # the sink's score, exactly
    desc, offsets, keep = alike(c)
    out = torch.zeros(REQUESTS, 4, head, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(REQUESTS, 4, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.empty(kva.kva_gqa_decode_workspace(4, 1, head), dtype=torch.uint8, device="cuda")
    slopes = torch.zeros(4, device="cuda") if biased else None  # the way of the biased scores
    kva.kva_gqa_decode_paged(out, q.repeat(REQUESTS, 1, 1).cuda(), offsets, desc, 0, 1.0, space, lse=lse,
                             v_scale=c.v_scale, alibi_slopes=slopes, err_flags=flags)
    assert int(flags) == 0
    check(out, lse, q[0].double(), c.rows(0, 0, 0, POSITIONS)[:, 0],
          c.rows(0, 1, 0, POSITIONS)[:, 0], head)


@pytest.mark.parametrize("gap", [12.0, 16.0, 17.0, 18.0, 20.0, 24.0])
@pytest.mark.parametrize("sink", [0, 5000, POSITIONS - 1])
@pytest.mark.parametrize("heads,page", [(16, 64), (80, 16)])
def test_mla(kva, gap, sink, heads, page):
    c = R.Paged(111, [1], [POSITIONS - 1], kv_heads=1, head=576, planes=1, dtype=R.E4M3, page=page,
                layers=1, layer=0)
    rows = torch.randn(POSITIONS, 576, generator=c.gen) * 0.2
    rows[:, :512] += 1
    rows[:, 512] = 0
    rows[sink] = 0
    rows[sink, 512] = 16
    put(c, 0, torch.arange(POSITIONS), rows)
    q = torch.cat([c.normal(1, heads, 512, std=0.05), c.normal(1, heads, 64, std=0.05)], -1)
    q[:, :, :512] -= q[:, :, :512].float().mean(-1, keepdim=True).bfloat16()
    q[:, :, 512] = gap / 16
    desc, offsets, keep = alike(c)
    many = q.repeat(REQUESTS, 1, 1)
    ql, qr = many[:, :, :512].contiguous().cuda(), many[:, :, 512:].contiguous().cuda()
    out = torch.zeros(REQUESTS, heads, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(REQUESTS, heads, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.empty(kva.kva_mla_decode_workspace(heads), dtype=torch.uint8, device="cuda")
    kva.kva_mla_decode_paged(out, ql, qr, offsets, desc, 0, 1.0, space, lse=lse, err_flags=flags)
    assert int(flags) == 0
    k = c.rows(0, 0, 0, POSITIONS)[:, 0]
    check(out, lse, q[0].double(), k, k[:, :512], 576)
