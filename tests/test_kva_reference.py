"""The 64-bit evaluations the GPU tests compare with, held to torch's own
float64 functions."""
import math

import pytest
import torch

import kva_reference as R


@pytest.mark.parametrize("dtype", [R.BF16, R.E4M3])
def test_gqa_is_scaled_dot_product_attention(dtype):
    c = R.Paged(1, [1, 3, 0, 2], [0, 17, 5, 40], kv_heads=2, head=32, dtype=dtype).fill()
    q = c.normal(c.T, 6, 32)
    out, lse, _, _ = R.gqa(c, q, 0.2)
    for t, b, pos in c.tokens():
        k, v = c.rows(b, 0, 0, pos + 1), c.rows(b, 1, 0, pos + 1)
        want = torch.nn.functional.scaled_dot_product_attention(
            q[t].double().view(2, 3, 32), k.transpose(0, 1), v.transpose(0, 1), scale=0.2)
        assert torch.allclose(out[t], want.reshape(6, 32), rtol=1e-12, atol=1e-14)
        s = torch.einsum("gd,lgd->gl", q[t].double().view(2, 3, 32)[:, 1], k) * 0.2
        assert torch.allclose(lse[t].view(2, 3)[:, 1], torch.logsumexp(s, -1), rtol=1e-12)


def test_gqa_modifiers():
    c = R.Paged(2, [1], [30], kv_heads=1, head=32).fill()
    q = c.normal(1, 2, 32, std=3.0)
    full = R.gqa(c, q, 0.3)[0]
    assert torch.equal(R.gqa(c, q, 0.3, window=31)[0], full)
    assert torch.allclose(R.gqa(c, q, 0.3, window=1)[0][0, 0], c.rows(0, 1, 30, 31)[0, 0])
    assert torch.allclose(R.gqa(c, q, 0.3, softcap=1e9)[0], full, atol=1e-9)
    steep = R.gqa(c, q, 0.3, slopes=torch.tensor([1e4, 1e4]))[0]
    assert torch.allclose(steep[0, 1], c.rows(0, 1, 30, 31)[0, 0])
    capped = R.gqa(c, q * 1000, 0.3, softcap=0.5)[1]
    assert bool((capped <= math.log(31) + 0.5).all())


def test_mla_is_attention_over_the_latent_rows():
    c = R.Paged(3, [2, 1], [20, 0], kv_heads=1, head=576, planes=1, dtype=R.E4M3).fill()
    ql, qr = c.normal(3, 4, 512), c.normal(3, 4, 64)
    out = R.mla(c, ql, qr, 0.07)[0]
    for t, b, pos in c.tokens():
        rows = c.rows(b, 0, 0, pos + 1)[:, 0]
        want = torch.nn.functional.scaled_dot_product_attention(
            torch.cat([ql[t], qr[t]], -1).double(), rows, rows[:, :512], scale=0.07)
        assert torch.allclose(out[t], want, rtol=1e-12, atol=1e-14)


def test_append_norm_and_rotation():
    c = R.Paged(4, [2, 1], [3, 0], kv_heads=1, head=32)
    freqs = R.freqs_table(8, 32)
    qkv = c.normal(3, 5 * 32)
    g = c.normal(32)
    (q, k, v), _ = R.append(c, qkv, 3, freqs, q_gamma=g, eps=0.25, weight_offset=1.0)
    x = qkv.double().view(3, 5, 32)
    assert torch.equal(v, x[:, 4:])
    n = torch.nn.functional.rms_norm(x[:, :3], (32,), g.double() + 1.0, 0.25)
    assert torch.allclose(q.pow(2).sum(-1), n.pow(2).sum(-1), rtol=1e-6)  # rotations keep norms
    assert torch.allclose(q[2], n[2])  # position 0
    z = torch.complex(x[0, 3, :16], x[0, 3, 16:])
    a = 3.0 * 10000.0 ** (-torch.arange(16, dtype=torch.float64) / 16)
    w = z * torch.polar(torch.ones(16, dtype=torch.float64), a)
    assert torch.allclose(k[0, 0], torch.cat([w.real, w.imag]), atol=1e-6)  # fp32 table
    (q2, _, _), _ = R.append(c, qkv, 3, freqs, interleaved=True)
    z = torch.complex(x[0, 1, 0::2], x[0, 1, 1::2]) * torch.polar(
        torch.ones(16, dtype=torch.float64), a)
    assert torch.allclose(q2[0, 1, 0::2], z.real, atol=1e-6)
    assert torch.allclose(q2[0, 1, 1::2], z.imag, atol=1e-6)
