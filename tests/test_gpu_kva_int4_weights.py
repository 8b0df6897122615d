"""Attention over a cache held in 4 bits where weights and value scales are far
apart: positions of zero values with large scores, and the ends of the ranges
that the header gives (GPU).  Calls are large enough that a piece takes whole
contexts, tile after tile, so that sums are held while the reference moves."""
import copy

import pytest
import torch

import kva_int4_reference as Q
import kva_reference as R
from test_gpu_kva_int4 import Call, kva, lengths  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def repeated(c, reps):
    """A batch of `reps` times c's requests, over the same pages."""
    m = copy.copy(c)
    m.new, m.prior = c.new * reps, c.prior * reps
    m.B, m.T = c.B * reps, c.T * reps
    m.table, m.lens = c.table.repeat(reps, 1), c.lens.repeat(reps)
    m.offsets = torch.tensor([0] + torch.tensor(m.new).cumsum(0).tolist(), dtype=torch.int32)
    return m


LEAST = 2.0 ** -40  # what a value's scale counts as, at least


def run_repeated(kva, c, q, reps, least=LEAST, **kw):
    """Every repetition against one evaluation in 64 bits.

    A weight times a scale is rounded to fp16, by 2^-34 of the row's largest where
    it is small.  A scale below LEAST counts as that in the largest: a position of
    weight p, at most 1, raises the others' error to 2^-34 LEAST p, times codes up
    to 7, for each of n positions."""
    x = Call(kva, repeated(c, reps), q.shape[1], q=q.repeat(reps, 1, 1), **kw)
    x.call()
    torch.cuda.synchronize()
    assert int(x.flags) == 0
    out, lse, to, tl = Q.gqa(c, q, x.scale, x.softcap, x.window, x.slopes)
    to += 2.0 ** -34 * least * 7 * (max(c.prior) + 1)
    for got, want, tol, what in ((x.out, out, to, "out"), (x.lse, lse, tl, "lse")):
        R.check(got.cpu(), want.repeat(reps, *[1] * (want.dim() - 1)),
                tol.repeat(reps, *[1] * (tol.dim() - 1)), what)
    return x


@pytest.mark.parametrize("head,q_heads", [(64, 2), (96, 8), (128, 12), (256, 4)])
@pytest.mark.parametrize("nats", [60, 74, 77, 80, 81, 100])
@pytest.mark.parametrize("mods", [{}, {"softcap": 500.0}, {"alibi": True}])
def test_zero_values_of_large_scores(kva, head, q_heads, nats, mods):
    """Eight tiles, taken from the last to the first: ordinary values with a score
    of 0, zero values with one of `nats`, ordinary values with the same.  The
    second take part in the sum of the weights alone."""
    n = 512
    c = Q.Int4(200, *lengths(n), kv_heads=1, head=head, page=64, layers=1, layer=0)
    k = torch.ones(n, 1, head)
    k[384:] = 0
    c.put(0, 0, 0, *Q.held(k))
    v = torch.randn(n, 1, head, generator=c.gen)
    v[128:384] = 0
    c.put(0, 1, 0, *Q.held(v))
    # (a key of ones is held as 7 codes of a seventh; scores by many small columns)
    q = torch.full((1, q_heads, head), nats / head).bfloat16()
    run_repeated(kva, c, q, 1200, sm_scale=1.0, **mods)


@pytest.mark.parametrize("head,q_heads", [(64, 2), (128, 12), (256, 4)])
@pytest.mark.parametrize("nats", [77, 80])
def test_zero_values_alone(kva, head, q_heads, nats):
    """Nothing but zero values has weight: rows of zeros, and their sum."""
    n = 512
    c = Q.Int4(201, *lengths(n), kv_heads=1, head=head, page=64, layers=1, layer=0)
    k = torch.ones(n, 1, head)
    k[384:] = 0
    c.put(0, 0, 0, *Q.held(k))
    v = torch.randn(n, 1, head, generator=c.gen)
    v[:384] = 0
    c.put(0, 1, 0, *Q.held(v))
    run_repeated(kva, c, torch.full((1, q_heads, head), nats / head).bfloat16(), 1200, sm_scale=1.0)


@pytest.mark.parametrize("head,q_heads", [(64, 2), (96, 8), (128, 12), (256, 4)])
@pytest.mark.parametrize("power", [-60, -45, -30, 60, 80])
def test_values_of_any_size(kva, head, q_heads, power):
    """A cache whose values are all tiny, or all large, is as exact as any other: at
    2^-60 the 2^-34 of what counts as 2^-40 is 2^-14 of the largest, within the
    2^-11 of a weight."""
    c = Q.Int4(202, *lengths(300, 65, 900), kv_heads=1, head=head, page=64, layers=1,
               layer=0).fill()
    c.scales[:, 1] = (c.scales[:, 1].double() * 2.0 ** power).bfloat16()
    run_repeated(kva, c, c.normal(3, q_heads, head, std=2.0), 300, least=0.0)


@pytest.mark.parametrize("head,q_heads", [(64, 2), (128, 12), (256, 4)])
@pytest.mark.parametrize("zeros", [(0, 512), (512, 896), (64, 128)])
def test_zero_values_beside_the_largest(kva, head, q_heads, zeros):
    """Zero values keep their share of the weights beside values of 2^80."""
    c = Q.Int4(204, *lengths(900, 330), kv_heads=1, head=head, page=64, layers=1, layer=0).fill()
    c.scales[:, 1] = (c.scales[:, 1].double() * 2.0 ** 80).bfloat16()
    for b, n in enumerate((900, 330)):
        ids, row = c.place(b, min(zeros[0], n), min(zeros[1], n))
        c.scales[ids, 1, c.layer, :, :, row] = 0
    run_repeated(kva, c, c.normal(2, q_heads, head), 400)


@pytest.mark.parametrize("head,q_heads", [(64, 2), (128, 12), (256, 4)])
@pytest.mark.parametrize("power,softcap", [(100, 0.0), (117, 0.0), (116, 1.0), (118, 4.0)])
def test_largest_queries(kva, head, q_heads, power, softcap):
    """Queries whose product with sm_scale is just below 2^117 (2^116 times a cap),
    over keys as much smaller."""
    c = Q.Int4(203, *lengths(300, 65), kv_heads=1, head=head, page=64, layers=1, layer=0).fill()
    c.scales[:, 0] = (c.scales[:, 0].double() * 2.0 ** -power).bfloat16()
    q = torch.randn(2, q_heads, head, generator=c.gen).clamp(-1.9, 1.9)
    run_repeated(kva, c, (q * 2.0 ** power).bfloat16(), 4, sm_scale=0.5, softcap=softcap)
