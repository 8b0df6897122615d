"""Caps and distance biases of the GQA scores, with what each step may be off by
counted by itself (GPU).

A score is a sum of `head` products in fp32, each off by half a step (2^-24) of
the sum of their sizes; a cap leaves it off by 2^-19 of itself; a distance bias
adds four half steps of slope times distance (slope in units of log2, its
product with the distance, the bias of the position, the sum) and one of the
score; the exponent's argument and value are off by 2^-20.  Weights are rounded
to bf16, or to fp16 (2^-11 of themselves, at least 2^-34 of the largest), the
result to bf16."""
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


def evaluate(c, q, sm_scale, softcap, window, slopes):
    hq, d = q.shape[1], c.head
    g = hq // c.kv_heads
    outs = [torch.zeros(c.T, hq, d, dtype=torch.float64) for _ in range(2)]
    lses = [torch.zeros(c.T, hq, dtype=torch.float64) for _ in range(2)]
    rel = 2.0 ** -8 if c.dtype == R.BF16 else 2.0 ** -11
    for t, b, pos in c.tokens():
        lo = max(0, pos - window + 1) if window else 0
        k, v = (c.rows(b, p, lo, pos + 1) for p in (0, 1))
        away = (pos - torch.arange(lo, pos + 1)).double()
        for h in range(hq):
            kh, vh, qh = k[:, h // g], v[:, h // g], q[t, h].double()
            x = kh @ qh * sm_scale
            off = (kh.abs() @ qh.abs()) * sm_scale * d * 2.0 ** -24
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                off = off + 2.0 ** -19 * x.abs()
            if slopes is not None:
                bias = float(slopes[h]) * away
                x = x - bias
                off = off + 4 * 2.0 ** -24 * bias.abs() + 2.0 ** -24 * x.abs()
            ds = off + 2.0 ** -20
            top = x.max()
            e = torch.exp(x - top)
            p = e / e.sum()
            out = p @ vh
            # p_j (v_j - out) changes by at most 2 ds_j; roundings act on p |v|
            tol = (p * (rel * (1 + 2 * ds) + 2 * ds)) @ vh.abs() + (2 * p * ds).sum() * out.abs()
            if c.dtype == R.E4M3:
                tol = tol + (e.clamp(max=2.0 ** -34) / e.sum()) @ vh.abs()
            outs[0][t, h], outs[1][t, h] = out, tol + 2.0 ** -8 * (out.abs() + tol)
            lse = top + torch.log(e.sum())
            lses[0][t, h], lses[1][t, h] = lse, 2 * (p * ds).sum() + lse.abs() * 2.0 ** -22
    return outs, lses


def run(kva, c, heads, *, q_std=2.0, softcap=0.0, window=0, slopes=None):
    q, sm_scale = c.normal(c.T, heads, c.head, std=q_std), 1 / math.sqrt(c.head)
    outs, lses = evaluate(c, q, sm_scale, softcap, window, slopes)
    desc, store, keep = c.on()
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    space = torch.empty(kva.kva_gqa_decode_workspace(heads, c.kv_heads, c.head),
                        dtype=torch.uint8, device="cuda")
    kva.kva_gqa_decode_paged(out, q.cuda(), keep[3], desc, c.layer, sm_scale, space, lse=lse,
                             v_scale=c.v_scale, softcap=softcap, window=window,
                             alibi_slopes=None if slopes is None else slopes.cuda(),
                             err_flags=flags)
    assert int(flags) == 0
    R.check(out, *outs, "out")
    R.check(lse, *lses, "lse")


@pytest.mark.parametrize("softcap", [0.3, 5.0, 50.0, 1e3, 1e5, 1e7, 1e12, 1.8e19, 1e30, 3.4e38])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("head", [64, 128, 256])
def test_caps(kva, dtype, head, softcap):
    """From caps that the scores pass to caps that they never feel."""
    c = R.Paged(120, [1, 3, 1], [2, 130, 700], kv_heads=2, head=head, dtype=dtype).fill()
    run(kva, c, 8, softcap=softcap, q_std=4.0)


@pytest.mark.parametrize("softcap", [5.0, 1e6])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_cap_with_scores_near_each_other(kva, dtype, softcap):
    c = R.Paged(121, [1, 1], [300, 900], kv_heads=1, head=64, dtype=dtype).fill()
    run(kva, c, 4, softcap=softcap, q_std=0.05)


@pytest.mark.parametrize("softcap,window", [(0.0, 0), (30.0, 0), (0.0, 500)])
@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_distance_bias(kva, dtype, softcap, window, sign):
    """Also rising with the distance, where the far positions have the weight."""
    c = R.Paged(122, [1, 2, 1], [60, 900, 3000], kv_heads=2, head=64, dtype=dtype,
                page=64).fill()
    slopes = sign * 2.0 ** (-8.0 * torch.arange(1, 9).float() / 8)
    run(kva, c, 8, softcap=softcap, window=window, slopes=slopes)
