"""A cache held in 4 bits on the CPU and plain 64-bit evaluations of the calls
on it (test infrastructure; nothing here is used by the library).

Roundings counted: half a step of bf16 is 2^-8 relative, of fp16 2^-11 (2^-25
below its smallest normal), of fp32 2^-24; half a step of a code is half the
group's scale.
"""
import math

import numpy as np
import torch

import kva_reference as R

GROUP = 64


def groups_of(d):
    return -(-d // GROUP)


def unpack(codes):
    """uint8 [..., D / 2] -> codes 0..15 as int64 [..., D]."""
    c = codes.long()
    return torch.stack([c & 15, c >> 4], -1).flatten(-2)


def pack(u):
    u = u.to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def by_column(scales, d):
    """[..., groups] -> [..., D]."""
    return scales.repeat_interleave(GROUP, -1)[..., :d]


def held(x):
    """(codes 1..15, bf16 scales) of fp32 rows [..., D], as the header defines them."""
    d = x.shape[-1]
    pad = torch.nn.functional.pad(x, (0, -d % GROUP)).unflatten(-1, (-1, GROUP))
    top = pad.abs().amax(-1)
    scales = torch.where(torch.isfinite(pad).all(-1), top * torch.tensor(1 / 7),
                         torch.tensor(float("nan"))).bfloat16()
    s = by_column(scales.float(), d)
    q = torch.where(s > 0, x / s, torch.zeros_like(x)).clamp(-7, 7).round()
    return (q + 8).long(), scales


class Int4:
    """Codes uint8 [pages, 2, layers, heads, page, D/2] and scales bf16 [pages,
    2, layers, heads, groups, page] as views of padded stores; codes 15 and NaN
    scales until put."""

    def __init__(self, seed, new, prior, *, kv_heads=2, head=64, page=16, layers=2, layer=1,
                 spare_pages=3, table_extra=2, head_pad=0, page_pad=0):
        g = self.gen = torch.Generator().manual_seed(seed)
        self.new, self.prior = list(new), list(prior)
        self.B, self.T = len(self.new), sum(self.new)
        self.page, self.layer, self.layers, self.kv_heads, self.head = page, layer, layers, kv_heads, head
        ng = self.groups = groups_of(head)
        need = [-(-(p + n) // page) for n, p in zip(self.new, self.prior)]
        self.pages = sum(need) + spare_pages
        ids = torch.randperm(self.pages, generator=g).to(torch.int32)
        self.table = torch.full((self.B, max(need + [1]) + table_extra), R.UNMAPPED,
                                dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.offsets = torch.tensor(np.concatenate([[0], np.cumsum(self.new)]), dtype=torch.int32)
        self.lens = torch.tensor(self.prior, dtype=torch.int32)

        def make(inner, fill, dtype):
            n = inner[0] * inner[1]
            sh = (kv_heads * (n + 16 * head_pad))
            store = torch.full((self.pages, 2 * layers * sh + 16 * page_pad), fill, dtype=dtype)
            st = (store.stride(0), layers * sh, sh, n + 16 * head_pad, inner[1], 1)
            return store, (self.pages, 2, layers, kv_heads, *inner), st

        self.code_store, self.code_shape, self.code_stride = make((page, head // 2), 0xFF,
                                                                  torch.uint8)
        self.scale_store, self.scale_shape, self.scale_stride = make((ng, page), float("nan"),
                                                                     torch.bfloat16)
        self.see(self.code_store, self.scale_store)

    def see(self, code_store, scale_store):
        """Reads from these stores (brought back from a device) from now on."""
        self.code_store, self.scale_store = code_store.cpu(), scale_store.cpu()
        self.codes = torch.as_strided(self.code_store, self.code_shape, self.code_stride)
        self.scales = torch.as_strided(self.scale_store, self.scale_shape, self.scale_stride)

    def place(self, b, lo, hi):
        at = torch.arange(lo, hi)
        return self.table[b].long()[at // self.page], at % self.page

    def put(self, b, plane, lo, codes, scales):
        """codes [n, heads, D] 0..15, scales [n, heads, groups] bf16 of positions lo ..."""
        ids, row = self.place(b, lo, lo + len(codes))
        self.codes[ids, plane, self.layer, :, row] = pack(codes)
        self.scales[ids, plane, self.layer, :, :, row] = scales

    def fill(self, std=1.0):
        for b in range(self.B):
            n = self.prior[b] + self.new[b]
            for plane in range(2):
                x = torch.randn((n, self.kv_heads, self.head), generator=self.gen) * std
                self.put(b, plane, 0, *held(x))
        return self

    def rows(self, ids, row):
        """(codes 0..15, scales by column) [n, 2, heads, D] float64."""
        u = unpack(self.codes[ids, :, self.layer, :, row]).double()
        s = by_column(self.scales[ids, :, self.layer, :, :, row].double(), self.head)
        return u, s

    tokens = R.Paged.tokens
    normal = R.Paged.normal

    def on(self, device="cuda"):
        """(cache, scales descriptors, what they point to: codes, scales, table, lengths, offsets)."""
        from gqa_kv_cache_mla_gb300 import kva

        keep = [x.to(device) for x in (self.code_store, self.scale_store, self.table, self.lens,
                                       self.offsets)]
        cache, scales = kva.int4_cache(
            torch.as_strided(keep[0], self.code_shape, self.code_stride),
            torch.as_strided(keep[1], self.scale_shape, self.scale_stride), keep[2], keep[3])
        return cache, scales, keep


def gqa(c, q, sm_scale, softcap=0.0, window=0, slopes=None):
    """float64 out [T, Hq, D], lse [T, Hq], and the error allowed for each.

    A score adds up d products whose sizes count codes from 0 and the offset of
    8 a code, in fp32: off by at most d half steps of the sum of those sizes,
    its exponent and the later steps by 2^-20 relative.  A weight times a scale
    is rounded to fp16: 2^-11 of itself or, below fp16's smallest normal, 2^-34
    of the row's largest.  The sums of these times codes 0 to 15, and times the
    offset, are fp32 sums of n terms that may be cut off at 2^-23.  The result
    is rounded to bf16.

    A matrix instruction lines 16 products and the sum before them up at the
    largest exponent and may cut each of the 17 at 2^-23 of that.  A code u is
    the fp16 number u 2^-24 there (16 u 2^-24 for every other one), below the
    smallest normal number 2^-14, whose exponent it is taken with: the cut is at
    2^-23 2^-14 2^24 = 2^-13 of a code, times the other operand's power of two
    (its largest value).
    A score is d / 16 instructions, and d / 16 for its offset; an output
    n / 16 full ones and one for each of the eight warps and its offset."""
    hq, d, hk = q.shape[1], c.head, c.kv_heads
    g = hq // hk
    outs = [torch.zeros(c.T, hq, d, dtype=torch.float64), torch.zeros(c.T, hq, dtype=torch.float64),
            torch.zeros(c.T, hq, d, dtype=torch.float64), torch.zeros(c.T, hq, dtype=torch.float64)]
    outs[1].fill_(-math.inf)
    for t, b, pos in c.tokens():
        at = torch.arange(pos + 1)
        seen = R.page_mask(c, b, pos + 1)
        if window:
            seen &= at > pos - window
        idx = at[seen]
        if len(idx) == 0:
            continue
        ids = c.table[b].long()[idx // c.page]
        u, s = c.rows(ids, idx % c.page)
        for h in range(hq):
            k, v = (u[:, i, h // g] - 8 for i in range(2))
            sk, sv, qh = s[:, 0, h // g], s[:, 1, h // g], q[t, h].double()
            x = (k * sk) @ qh * sm_scale
            size = ((u[:, 0, h // g] + 8) * sk.abs()) @ qh.abs() * sm_scale
            if softcap:
                x = softcap * torch.tanh(x / softcap)
                size = size + softcap * 2.0  # a few half steps of the cap itself
            if slopes is not None:
                x = x - float(slopes[h]) * (pos - idx).double()
                size = size + float(slopes[h]) * (pos + 1)
            cut = 17 * 2.0 ** -13
            ds = d * 2.0 ** -24 * float(size.max()) + 2.0 ** -20 + \
                cut * d / 8 * float(qh.abs().max() * sk.abs().max()) * sm_scale
            top = x.max()
            if top == -math.inf:
                continue
            e = torch.exp(x - top)
            p = e / e.sum()
            out = p @ (sv * v)
            tol = p @ (sv * v).abs() * (2.0 ** -11 * (1 + 2 * ds) + 2 * ds)
            tol = tol + 2.0 ** -34 * 7 * len(idx) * (p[:, None] * sv).abs().max()
            tol = tol + len(idx) * 2.0 ** -23 * (p @ (sv.abs() * (u[:, 1, h // g] + 8)))
            tol = tol + cut * 2 * (len(idx) / 16 + 8) * (p[:, None] * sv).abs().max()
            outs[0][t, h] = out
            outs[2][t, h] = tol + R.HALF_STEP[R.BF16] * (out.abs() + tol)
            outs[1][t, h] = lse = top + torch.log(e.sum())
            outs[3][t, h] = 2 * ds + abs(float(lse)) * 2.0 ** -22
    return outs


def check_held(codes, scales, y, err, what=""):
    """Codes 0..15 [..., D] and scales [..., groups] hold y (float64), each of
    whose values was known to within err when it was quantised."""
    d = y.shape[-1]
    fold = lambda x: torch.nn.functional.pad(x, (0, -d % GROUP)).unflatten(-1, (-1, GROUP))
    top, e = fold(y.abs()).amax(-1), fold(err).amax(-1)
    s = scales.double()
    # the seventh is rounded to fp32 twice, then to bf16 (2^-134: half its last step)
    off = (s - top / 7).abs() - (R.HALF_STEP[R.BF16] * top / 7 * (1 + 2.0 ** -8) + e / 7 + 2.0 ** -134)
    assert float(off.max()) <= 0, "%s: scales off by %.3g more" % (what, float(off.max()))
    assert bool(((codes >= 1) & (codes <= 15)).all()), what
    by = by_column(s, d)
    # half a step, and the quotient's own rounding of up to 7 half steps of fp32
    off = ((codes - 8).double() * by - y).abs() - (by * (0.5 + 2.0 ** -20) + err + 2.0 ** -131)
    assert float(off.max()) <= 0, "%s: values off by %.3g more" % (what, float(off.max()))
