"""Plain 64-bit evaluations of the calls of ``include/kva.h`` and small paged
batches to run them on (test infrastructure; nothing here is used by the
library).

Each operator is written from its formula in torch float64, token by token,
from the definition of the paged cache; every function also returns what its
tolerance is made of.  Roundings counted below: half a step of bf16 is 2^-8
relative, of fp16 2^-11, of fp32 2^-24, of E4M3 2^-4 (2^-10 of a unit code
below the smallest normal).
"""
import math

import numpy as np
import torch

BF16, E4M3 = 0, 1
HALF_STEP = {BF16: 2.0 ** -8, E4M3: 2.0 ** -4}
UNMAPPED = -1  # 0xFFFFFFFF as int32


class Paged:
    """A paged cache on the CPU: torch tensor [pages, kv, layers, page_size,
    heads, head_size] (bf16, or uint8 codes), every element NaN until put."""

    def __init__(self, seed, new, prior, *, kv_heads=2, head=64, page=16, dtype=BF16, planes=2,
                 layers=2, layer=1, k_scale=0.5, v_scale=0.25, spare_pages=3, table_extra=2,
                 head_pad=0, token_pad=0):
        g = self.gen = torch.Generator().manual_seed(seed)
        self.new, self.prior = list(new), list(prior)
        self.B, self.T = len(self.new), sum(self.new)
        self.dtype, self.page, self.layer, self.layers = dtype, page, layer, layers
        self.kv_heads, self.head, self.planes = kv_heads, head, planes
        self.k_scale, self.v_scale = (k_scale, v_scale) if dtype == E4M3 else (1.0, 1.0)
        need = [-(-(p + n) // page) for n, p in zip(self.new, self.prior)]
        self.pages = sum(need) + spare_pages
        width = max(need + [1]) + table_extra
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((self.B, width), UNMAPPED, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32)
        self.lens = torch.tensor(self.prior, dtype=torch.int32)
        item = torch.bfloat16 if dtype == BF16 else torch.uint8
        nan = float("nan") if dtype == BF16 else 0x7F
        store = torch.full((self.pages, planes, layers, page, kv_heads * (head + head_pad)
                            + token_pad), nan, dtype=item)
        self.data = torch.as_strided(
            store, (self.pages, planes, layers, page, kv_heads, head),
            (*store.stride()[:4], head + head_pad, 1))
        self.store = store

    def rows(self, b, plane, lo, hi, data=None):
        """Rows lo..hi-1 of request b as the cache holds them, float64 [n, heads, head]."""
        data = self.data if data is None else data
        at = torch.arange(lo, hi)
        x = data[self.table[b].long()[at // self.page], plane, self.layer, at % self.page]
        if self.dtype == E4M3:
            scale = self.v_scale if plane else self.k_scale
            return x.view(torch.float8_e4m3fn).double() * scale
        return x.double()

    def fill(self, std=1.0):
        """Normal values in every slot of every context (prior and new)."""
        for b in range(self.B):
            n = self.prior[b] + self.new[b]
            at = torch.arange(n)
            for plane in range(self.planes):
                x = torch.randn((n, self.kv_heads, self.head), generator=self.gen) * std
                scale = self.v_scale if plane else self.k_scale
                x = x.bfloat16() if self.dtype == BF16 else \
                    (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                self.data[self.table[b].long()[at // self.page], plane, self.layer,
                          at % self.page] = x
        return self

    def tokens(self):
        t = 0
        for b in range(self.B):
            for i in range(self.new[b]):
                yield t, b, self.prior[b] + i
                t += 1

    def normal(self, *shape, std=1.0):
        return (torch.randn(shape, generator=self.gen) * std).bfloat16()

    def on(self, device="cuda"):
        """(descriptor, store tensor, the tensors it points to) on the device."""
        from gqa_kv_cache_mla_gb300 import kvw

        store = self.store.to(device)
        keep = [store, self.table.to(device), self.lens.to(device), self.offsets.to(device)]
        s = self.data.stride()
        desc = kvw.paged_cache(store, self.dtype, keep[1], keep[2], self.pages, self.layers,
                               self.page, self.kv_heads, self.head, s[:5], scale=self.k_scale)
        return desc, store, keep

    def view(self, store):
        """The logical view of a store tensor brought back to the CPU."""
        return torch.as_strided(store.cpu(), self.data.shape, self.data.stride())


# ------------------------------------------------------------------ append

def freqs_table(rows, dim, base=10000.0):
    theta = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    a = torch.arange(rows, dtype=torch.float64)[:, None] * theta
    return torch.stack([a.cos(), a.sin()], -1).reshape(rows, dim).float()


def pair_positions(c, position_ids, mrope_section, pairs, t, pos):
    """Position of each rotary pair of token t."""
    if position_ids is None:
        return [pos] * pairs
    if mrope_section is None:
        return [int(position_ids[t])] * pairs
    s0, s1, _ = mrope_section
    return [int(position_ids[0 if k < s0 else 1 if k < s0 + s1 else 2][t]) for k in range(pairs)]


def append(c, qkv, q_heads, freqs, *, q_gamma=None, k_gamma=None, eps=1e-6, weight_offset=0.0,
           position_ids=None, mrope_section=None, interleaved=False):
    """(q, k, v) float64 [T, heads, head] before rounding and the size of the
    fp32 error of each element before rounding: the sum of squares of `head`
    terms and the handful of operations after it are off by at most
    (head + 16) half steps relative to the terms that make the element up."""
    T, d, hk = c.T, c.head, c.kv_heads
    x = qkv.double()[:, :(q_heads + 2 * hk) * d].reshape(T, q_heads + 2 * hk, d).clone()
    for lo, hi, g in ((0, q_heads, q_gamma), (q_heads, q_heads + hk, k_gamma)):
        if g is not None:
            y = x[:, lo:hi]
            r = 1.0 / torch.sqrt((y * y).mean(-1, keepdim=True) + eps)
            x[:, lo:hi] = y * r * (g.double() + weight_offset)
    size = x.abs()
    dim = 0 if freqs is None else freqs.shape[1]
    half = dim // 2
    for t, b, pos in c.tokens():
        ps = pair_positions(c, position_ids, mrope_section, half, t, pos)
        for k, p in enumerate(ps):
            cs, sn = float(freqs[p, 2 * k]), float(freqs[p, 2 * k + 1])
            i, j = (2 * k, 2 * k + 1) if interleaved else (k, k + half)
            u, w = x[t, :q_heads + hk, i].clone(), x[t, :q_heads + hk, j].clone()
            x[t, :q_heads + hk, i] = u * cs - w * sn
            x[t, :q_heads + hk, j] = u * sn + w * cs
            m = u.abs() + w.abs()
            size[t, :q_heads + hk, i] = m
            size[t, :q_heads + hk, j] = m
    err = size * (d + 16) * 2.0 ** -24
    cut = (q_heads, hk, hk)
    return x.split(cut, 1), err.split(cut, 1)


def stored_error(y, err, dtype, scale):
    """Largest |stored value - y| allowed, stored values in cache units (codes)."""
    if dtype == BF16:
        return HALF_STEP[BF16] * y.abs() * (1 + 2.0 ** -8) + err
    z = (y / scale).abs().clamp(max=448)
    # the quotient is rounded once more in fp32
    return torch.maximum(HALF_STEP[E4M3] * z, torch.tensor(2.0 ** -10, dtype=torch.float64)) \
        * (1 + 2.0 ** -4) + err / scale + z * 2.0 ** -23


# ------------------------------------------------------------------ attention

def _finish(x, v, size, dtype, d):
    """Softmax over x [heads, n] (natural log units, -inf masked) of v [n, w]:
    out, lse and the allowed error of out and of lse.

    A score is a sum of d products in fp32, each of size at most `size` (the
    largest sum of |q_i k_i| times the scale): off by at most d half steps of
    that, and the exponent's own error and the later fp32 steps by 2^-20
    relative.  The weight e^s / max is rounded to the operand type: relative
    2^-8 (bf16) or 2^-11 (fp16, at least 2^-25 of the largest weight seen so
    far, below its smallest normal).  Each acts on sum p |v|; the result is
    rounded to bf16 at the end."""
    if x.shape[1] == 0 or bool(torch.isinf(x).all()):
        w = v.shape[-1]
        z = torch.zeros(x.shape[0], w, dtype=torch.float64)
        return z, torch.full((x.shape[0],), -math.inf, dtype=torch.float64), z, z[:, 0]
    top = x.max(-1, keepdim=True).values
    e = torch.exp(x - top)
    l = e.sum(-1, keepdim=True)
    out = (e / l) @ v
    spread = (e / l) @ v.abs()
    rel = HALF_STEP[BF16] if dtype == BF16 else 2.0 ** -11
    ds = d * 2.0 ** -24 * size[:, None] + 2.0 ** -20
    tol = spread * (rel * (1 + 2 * ds) + 2 * ds)
    if dtype == E4M3:
        tol = tol + (torch.minimum(e, torch.tensor(2.0 ** -25, dtype=torch.float64)) / l) @ v.abs()
    tol = tol + HALF_STEP[BF16] * (out.abs() + tol)
    lse = (top + torch.log(l))[:, 0]
    return out, lse, tol, 2 * ds[:, 0] + lse.abs() * 2.0 ** -22


def page_mask(c, b, n):
    """Positions 0..n-1 of request b with a valid page."""
    at = torch.arange(n) // c.page
    ids = torch.where(at < c.table.shape[1], c.table[b].long()[at.clamp(max=c.table.shape[1] - 1)],
                      torch.tensor(-1))
    return (ids >= 0) & (ids < c.pages)


def gqa(c, q, sm_scale, softcap=0.0, window=0, slopes=None):
    """float64 out [T, Hq, D], lse [T, Hq], and the error allowed for each."""
    hq, d, hk = q.shape[1], c.head, c.kv_heads
    g = hq // hk
    outs = [torch.zeros(c.T, hq, d, dtype=torch.float64), torch.zeros(c.T, hq, dtype=torch.float64),
            torch.zeros(c.T, hq, d, dtype=torch.float64), torch.zeros(c.T, hq, dtype=torch.float64)]
    for t, b, pos in c.tokens():
        n = pos + 1
        at = torch.arange(n)
        seen = page_mask(c, b, n)
        if window:
            seen &= at > pos - window
        idx = at[seen]
        ids = c.table[b].long()[idx // c.page]
        kv = c.data[ids, :, c.layer, idx % c.page]
        kv = kv.view(torch.float8_e4m3fn).double() if c.dtype == E4M3 else kv.double()
        for h in range(hq):
            k, v = kv[:, 0, h // g] * c.k_scale, kv[:, 1, h // g] * c.v_scale
            qh = q[t, h].double()
            x = (k @ qh) * sm_scale
            size = float((k.abs() @ qh.abs()).max()) * sm_scale if len(idx) else 0.0
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                size = size + softcap * 2.0  # a few half steps of the cap itself
            if slopes is not None:
                x = x - float(slopes[h]) * (pos - idx).double()
                size = size + float(slopes[h]) * n
            o, lse, to, tl = _finish(x[None], v, torch.tensor([size], dtype=torch.float64),
                                     c.dtype, d)
            outs[0][t, h], outs[1][t, h], outs[2][t, h], outs[3][t, h] = o[0], lse[0], to[0], tl[0]
    return outs


def mla(c, q_latent, q_rope, sm_scale):
    """float64 out [T, H, 512], lse [T, H], and the error allowed for each."""
    h = q_latent.shape[1]
    outs = [torch.zeros(c.T, h, 512, dtype=torch.float64), torch.zeros(c.T, h, dtype=torch.float64),
            torch.zeros(c.T, h, 512, dtype=torch.float64), torch.zeros(c.T, h, dtype=torch.float64)]
    for t, b, pos in c.tokens():
        at = torch.arange(pos + 1)
        idx = at[page_mask(c, b, pos + 1)]
        rows = c.data[c.table[b].long()[idx // c.page], 0, c.layer, idx % c.page, 0]
        rows = (rows.view(torch.float8_e4m3fn).double() if c.dtype == E4M3 else rows.double()) \
            * c.k_scale
        q = torch.cat([q_latent[t], q_rope[t]], -1).double()
        x = q @ rows.T * sm_scale
        size = (q.abs() @ rows.abs().T).max(-1).values * sm_scale if len(idx) else \
            torch.zeros(h, dtype=torch.float64)
        o, lse, to, tl = _finish(x, rows[:, :512], size, c.dtype, 576)
        for dst, src in zip(outs, (o, lse, to, tl)):
            dst[t] = src
    return outs


def check(got, want, tol, what=""):
    """|got - want| <= tol elementwise, and nothing is NaN that should not be."""
    got = got.double().cpu()
    assert bool(torch.isfinite(got).eq(torch.isfinite(want)).all()), what
    fine = torch.isfinite(want)
    over = (got - want).abs()[fine] - tol[fine]
    assert over.numel() == 0 or float(over.max()) <= 0.0, \
        "%s: off by up to %.3g beyond the tolerance" % (what, float(over.max()))
    assert bool((got[~fine] == want[~fine]).all()), what


def check_norm(got, want, bound, what=""):
    """Relative 2-norm of the whole difference."""
    rel = float((got.double().cpu() - want).norm() / want.norm())
    assert rel <= bound, "%s: relative error %.3g over %.3g" % (what, rel, bound)
