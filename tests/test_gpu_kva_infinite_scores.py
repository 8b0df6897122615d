"""Scores of -infinity in the attention calls (GPU): such a position weighs
nothing, as if masked, and a token with no other gets zeros."""
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


def mark(c, column):
    """-infinity in the column of every second row of request 0 and of every row
    of request 1."""
    for b, step in ((0, 2), (1, 1)):
        at = torch.arange(0, c.prior[b] + 1, step)
        c.data[c.table[b].long()[at // c.page], 0, c.layer, at % c.page, :, column] = -math.inf


def without(c, b, step):
    at = torch.arange(c.prior[b] + 1)
    return at[at % step != 0] if step > 1 else at[:0]


def check(c, out, lse, x_of, v_of, rel):
    assert bool((out[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())
    for b, keep in ((0, without(c, 0, 2)), (2, torch.arange(c.prior[2] + 1))):
        x, v = x_of(b, keep), v_of(b, keep)
        p = torch.softmax(x, -1)
        want = p @ v
        # two roundings to bf16 and fp32 steps, all on the sum of p |v|
        tol = (p @ v.abs()) * (2 * 2.0 ** -8 + rel)
        R.check(out[b], want, tol)
        R.check(lse[b], torch.logsumexp(x, -1), rel * (1 + x.abs().max(-1).values))


@pytest.mark.parametrize("page", [12, 64])
@pytest.mark.parametrize("slopes", [False, True])
def test_gqa(kva, page, slopes):
    c = R.Paged(130, [1, 1, 1], [300, 200, 90], kv_heads=1, head=64, page=page).fill()
    mark(c, 0)
    q = c.normal(3, 4, 64)
    q[:, :, 0] = 1.0
    desc, store, keep = c.on()
    out, lse = torch.full_like(q, 7.0).cuda(), torch.full((3, 4), 7.0, device="cuda")
    space = torch.empty(kva.kva_gqa_decode_workspace(4, 1, 64), dtype=torch.uint8, device="cuda")
    kva.kva_gqa_decode_paged(out, q.cuda(), keep[3], desc, c.layer, 0.125, space, lse=lse,
                             alibi_slopes=torch.zeros(4, device="cuda") if slopes else None)

    def rows(b, plane, at):
        return c.rows(b, plane, 0, c.prior[b] + 1)[at, 0]

    check(c, out, lse, lambda b, at: q[b].double() @ rows(b, 0, at).T * 0.125,
          lambda b, at: rows(b, 1, at), 64 * 2.0 ** -20)


@pytest.mark.parametrize("page", [12, 64])
def test_mla(kva, page):
    c = R.Paged(131, [1, 1, 1], [300, 200, 90], kv_heads=1, head=576, planes=1, page=page).fill()
    mark(c, 512)  # the first rotated column: no value is infinite
    ql, qr = c.normal(3, 16, 512), c.normal(3, 16, 64)
    qr[:, :, 0] = 1.0
    desc, store, keep = c.on()
    out, lse = torch.full_like(ql, 7.0).cuda(), torch.full((3, 16), 7.0, device="cuda")
    space = torch.empty(kva.kva_mla_decode_workspace(16), dtype=torch.uint8, device="cuda")
    kva.kva_mla_decode_paged(out, ql.cuda(), qr.cuda(), keep[3], desc, c.layer, 0.07, space,
                             lse=lse)

    def rows(b, at):
        return c.rows(b, 0, 0, c.prior[b] + 1)[at, 0]

    q = torch.cat([ql, qr], -1).double()
    check(c, out, lse, lambda b, at: q[b] @ rows(b, at).T * 0.07,
          lambda b, at: rows(b, at)[:, :512], 64 * 2.0 ** -20)
