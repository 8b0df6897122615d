"""Measured cases of the attention side of the paged key-value cache.

Three operators, each as a serving loop calls it:

``append``  the fused projection of a step's new tokens is split into heads,
            queries and keys are RMS-normalised per head (optional) and
            rotated, queries go to their own buffer, keys and values into
            their cache slots (bf16, or E4M3 with a static scale)
``gqa``     each new token's query heads attend over the token's whole paged
            context, one key-value head per group of query heads; optional
            tanh cap, sliding window and distance bias
``mla``     the same over the latent cache: every head reads the same
            576-wide row, its first 512 columns are the value

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

GOLDEN = 0.6180339887498949


def listed():
    return [
        # one chat stream's next token: nothing but latency
        dict(name="append_one", op="append", batch=1, new=1, prior=700, q_heads=32, kv_heads=8,
             head=128, rope=128, page=128, dtype="bf16", norm=False, interleaved=False),
        # a decode step of a large batch, keys and queries normalised, E4M3 cache
        dict(name="append_decode_256", op="append", batch=256, new=1, prior=1024, q_heads=32,
             kv_heads=8, head=128, rope=128, page=64, dtype="e4m3", norm=True,
             interleaved=False),
        # the Llama-3-8B prefill batch of the benchmark: 32 ragged requests
        dict(name="append_prefill", op="append", batch=32, new=2048, prior=4096, q_heads=32,
             kv_heads=8, head=128, rope=128, page=128, dtype="bf16", norm=False,
             interleaved=True),
        # odd sizes: 96-wide heads of which 64 columns turn, pages of 48 tokens
        dict(name="append_odd", op="append", batch=13, new=301, prior=77, q_heads=10, kv_heads=5,
             head=96, rope=64, page=48, dtype="bf16", norm=True, interleaved=False),
        # one chat stream's next token over a short context
        dict(name="gqa_one", op="gqa", batch=1, new=1, prior=900, q_heads=32, kv_heads=8,
             head=128, page=128, dtype="bf16", cap=0.0, window=0, alibi=False),
        # a decode step of the benchmark's 32 requests
        dict(name="gqa_decode_32", op="gqa", batch=32, new=1, prior=4096, q_heads=32, kv_heads=8,
             head=128, page=128, dtype="bf16", cap=0.0, window=0, alibi=False),
        # the benchmark's decode batch of 256, E4M3 cache
        dict(name="gqa_decode_256_e4m3", op="gqa", batch=256, new=1, prior=8192, q_heads=32,
             kv_heads=8, head=128, page=64, dtype="e4m3", cap=0.0, window=0, alibi=False),
        # few requests with very long contexts
        dict(name="gqa_long", op="gqa", batch=8, new=1, prior=131072, q_heads=64, kv_heads=8,
             head=128, page=128, dtype="bf16", cap=0.0, window=0, alibi=False),
        # wide heads, capped scores, a sliding window, pages of 100, two tokens per request
        dict(name="gqa_cap_window", op="gqa", batch=48, new=2, prior=9001, q_heads=16,
             kv_heads=8, head=256, page=100, dtype="bf16", cap=50.0, window=4096, alibi=False),
        # one request on a slice of 16 heads
        dict(name="mla_one", op="mla", batch=1, new=1, prior=1500, heads=16, page=64,
             dtype="bf16"),
        # the benchmark's DeepSeek-V3 decode batch: 128 heads, E4M3 latent cache
        dict(name="mla_decode_256_e4m3", op="mla", batch=256, new=1, prior=8192, heads=128,
             page=128, dtype="e4m3"),
        # a smaller batch with a bf16 latent cache
        dict(name="mla_decode_64", op="mla", batch=64, new=1, prior=8192, heads=128, page=128,
             dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "gqa", "gqa", "mla", "mla"])
    dtype = rng.choice(["bf16", "e4m3"])
    page = rng.choice([16, 48, 64, 100, 128, 256])
    if op == "append":
        batch = _log(rng, 1, 256)
        head = rng.choice([64, 96, 128, 256])
        kv = rng.choice([1, 2, 5, 8])
        q = kv * rng.choice([1, 4, 7, 8])
        tokens = 29000 * 48 * 128 // ((q + 2 * kv) * head)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(1, min(2048, 2 * tokens // batch))),
                    prior=_log(rng, 1, min(4096, 98304 // batch)), q_heads=q, kv_heads=kv,
                    head=head, rope=rng.choice([head, 32]), page=page, dtype=dtype,
                    norm=rng.random() < 0.5, interleaved=rng.random() < 0.5)
    if op == "gqa":
        batch = _log(rng, 1, 256)
        new = rng.choice([1, 1, 1, 2, 4])
        head = rng.choice([64, 96, 128, 256])
        kv = rng.choice([1, 2, 4, 8])
        q = kv * rng.choice([1, 4, 5, 8, 16])
        rows = 8 * 131072 * 8 * 128 // (kv * head * batch * new)
        return dict(op=op, batch=batch, new=new, prior=_log(rng, 16, max(17, min(131072, rows))),
                    q_heads=q, kv_heads=kv, head=head, page=page, dtype=dtype,
                    cap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, 0, 129, 2048]),
                    alibi=rng.random() < 0.25)
    batch = _log(rng, 1, 256)
    new = rng.choice([1, 1, 1, 2])
    heads = rng.choice([8, 16, 40, 64, 128])
    return dict(op=op, batch=batch, new=new,
                prior=_log(rng, 16, min(65536, 256 * 8192 // (batch * new))), heads=heads,
                page=page, dtype=dtype)


# ------------------------------------------------------------------ lengths

def _spread(count, top, phase):
    """`count` lengths spread over 1..top, in no order; one alone has the top."""
    if count == 1:
        return np.full(1, top, np.int64)
    i = np.arange(count)
    return 1 + np.floor(top * ((i + 0.5) * GOLDEN + phase) % top).astype(np.int64)


def _lengths(case):
    """(new tokens, tokens cached before) of each request."""
    b = case["batch"]
    if case["op"] == "append" and case["new"] > 1:
        new = _spread(b, case["new"], 0.25)
    else:
        new = np.full(b, case["new"], np.int64)
    return new, _spread(b, case["prior"], 0.5)


def _rows_read(case):
    """(distinct cache rows read, (token, row) products) of an attention pass."""
    new, prior = _lengths(case)
    window = case.get("window") or (1 << 40)
    first = np.maximum(0, prior + 1 - window)
    rows = int((prior + new - first).sum())
    seen = sum(int(np.minimum(prior + 1 + i, window).sum()) for i in range(int(new[0])))
    return rows, seen


def work(case):
    new, prior = _lengths(case)
    t = int(new.sum())
    item = 2 if case["dtype"] == "bf16" else 1
    if case["op"] == "append":
        q, kv, d = case["q_heads"], case["kv_heads"], case["head"]
        moved = t * ((q + 2 * kv) * d * 2 + q * d * 2 + 2 * kv * d * item)
        angles = int((prior + new).max() - prior.min()) if t > len(new) else len(np.unique(prior))
        moved += angles * case["rope"] * 4
        return dict(bytes=moved, flops=t * (q + kv) * (3 * case["rope"] + 4 * d * case["norm"]))
    rows, seen = _rows_read(case)
    if case["op"] == "gqa":
        q, kv, d = case["q_heads"], case["kv_heads"], case["head"]
        return dict(bytes=rows * 2 * kv * d * item + 2 * t * q * d * 2, flops=seen * q * 4 * d)
    h = case["heads"]
    return dict(bytes=rows * 576 * item + t * h * (576 + 512) * 2, flops=seen * h * 2 * (576 + 512))


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _bf16(gen, shape, std=1.0):
    # in pieces: the caches are several GB
    out = torch.empty(shape, device="cuda", dtype=torch.bfloat16)
    flat = out.view(-1)
    for part in flat.split(1 << 28):
        part.copy_(_normal(gen, part.shape, std))
    return out


def _codes(gen, shape, std):
    """E4M3 codes of normal values in units of the cache scale."""
    out = torch.empty(shape, device="cuda", dtype=torch.uint8)
    for part in out.view(-1).split(1 << 28):
        part.copy_(_normal(gen, part.shape, std).clamp_(-448, 448).to(torch.float8_e4m3fn)
                   .view(torch.uint8))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    new, prior = _lengths(case)
    b, t, page = len(new), int(new.sum()), case["page"]
    pages = -(-(prior + new) // page)
    total, width = int(pages.sum()), int(pages.max())
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    used = torch.arange(width, device="cuda")[None, :] < torch.from_numpy(pages).cuda()[:, None]
    table = torch.full((b, width), -1, device="cuda", dtype=torch.int32)
    table[used] = ids
    offsets = np.concatenate([[0], np.cumsum(new)])
    s = dict(case=case, t=t, table=table, pages=total,
             offsets=torch.from_numpy(offsets.astype(np.int32)).cuda(),
             lens=torch.from_numpy(prior.astype(np.int32)).cuda(),
             flags=torch.zeros(1, device="cuda", dtype=torch.int32), longest=int((prior + new).max()))
    if case["op"] == "mla":
        kv, heads, head = 1, 1, 576
    else:
        kv, heads, head = 2, case["kv_heads"], case["head"]
    shape = (total, kv, 1, page, heads, head)
    if case["dtype"] == "bf16":
        s["cache"], s["k_scale"], s["v_scale"] = _bf16(gen, shape), 1.0, 1.0
    else:  # keys and values of about unit size, held in units of a static scale
        s["k_scale"], s["v_scale"] = 1 / 64, 0.02
        s["cache"] = _codes(gen, shape, 60.0)
    if case["op"] == "append":
        q, d, rope = case["q_heads"], case["head"], case["rope"]
        s["qkv"] = _bf16(gen, (t, (q + 2 * heads) * d))
        s["q_out"] = torch.zeros((t, q, d), device="cuda", dtype=torch.bfloat16)
        theta = 500000.0 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)
        angle = torch.arange(s["longest"], device="cuda", dtype=torch.float64)[:, None] * theta
        s["freqs"] = torch.stack([angle.cos(), angle.sin()], -1).reshape(-1, rope).float()
        s["q_gamma"] = s["k_gamma"] = None
        if case["norm"]:
            s["q_gamma"] = _normal(gen, (d,), 0.1).add_(1).bfloat16()
            s["k_gamma"] = _normal(gen, (d,), 0.1).add_(1).bfloat16()
    elif case["op"] == "gqa":
        q, d = case["q_heads"], case["head"]
        s["q"] = _bf16(gen, (t, q, d), 2.0)  # scores of standard deviation 2
        s["out"] = torch.zeros((t, q, d), device="cuda", dtype=torch.bfloat16)
        s["sm_scale"] = 1 / math.sqrt(d)
        s["slopes"] = None
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, q + 1, device="cuda").float() / q)
    else:
        h = case["heads"]
        s["q_latent"] = _bf16(gen, (t, h, 512), 1.2)  # scores of standard deviation 2
        s["q_rope"] = _bf16(gen, (t, h, 64), 1.2)
        s["out"] = torch.zeros((t, h, 512), device="cuda", dtype=torch.bfloat16)
        s["sm_scale"] = 1 / math.sqrt(192)  # 128 + 64 columns before the absorption
    return s


# ------------------------------------------------------------------ plain form

def _owner(s):
    """Request and slot position of each token."""
    n = s["offsets"].diff().long()
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=s["t"])
    pos = s["lens"].long()[b] + torch.arange(s["t"], device="cuda") - s["offsets"].long()[b]
    return b, pos


def _plain_norm(x, gamma):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * gamma.float()


def _plain_rope(x, cs, interleaved):
    rope = cs.shape[-2] * 2
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    if interleaved:
        a, b = x[..., 0:rope:2], x[..., 1:rope:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rope // 2], x[..., rope // 2:rope]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., rope:]], -1)


def _held(x, dtype, scale):
    """Values as the cache holds them."""
    if dtype == "bf16":
        return x.bfloat16()
    return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    c = s["case"]
    q, kv, d, page = c["q_heads"], c["kv_heads"], c["head"], c["page"]
    b, pos = _owner(s)
    x = s["qkv"].float().view(s["t"], q + 2 * kv, d)
    xq, xk, xv = x.split([q, kv, kv], 1)
    if c["norm"]:
        xq, xk = _plain_norm(xq, s["q_gamma"]), _plain_norm(xk, s["k_gamma"])
    cs = s["freqs"][pos].view(s["t"], -1, 2)
    s["q_out"].copy_(_plain_rope(xq, cs, c["interleaved"]))
    slot_page, row = s["table"][b, pos // page].long(), pos % page
    s["cache"][slot_page, 0, 0, row] = _held(_plain_rope(xk, cs, c["interleaved"]), c["dtype"],
                                             s["k_scale"])
    s["cache"][slot_page, 1, 0, row] = _held(xv, c["dtype"], s["v_scale"])


def _context(s, b, plane, scale):
    """[tokens, positions, heads, head] rows of the owners' contexts in 32 bits."""
    page = s["case"]["page"]
    at = torch.arange(s["longest"], device="cuda")
    ids = s["table"].long().clamp(min=0)[b][:, at // page]
    rows = s["cache"][ids, plane, 0, at % page]
    if rows.dtype == torch.uint8:
        return rows.view(torch.float8_e4m3fn).float().mul_(scale)
    return rows.float()


def _softmax(x):
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def _plain_gqa(s):
    c = s["case"]
    q, kv, d, t = c["q_heads"], c["kv_heads"], c["head"], s["t"]
    b, pos = _owner(s)
    k = _context(s, b, 0, s["k_scale"]).permute(0, 2, 3, 1)
    x = torch.matmul(s["q"].float().view(t, kv, q // kv, d), k).mul_(s["sm_scale"])
    del k
    if c["cap"]:
        x = c["cap"] * torch.tanh(x / c["cap"])
    away = pos[:, None] - torch.arange(s["longest"], device="cuda")
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, kv, q // kv, 1) * away[:, None, None, :].float()
    hidden = away < 0
    if c["window"]:
        hidden = hidden | (away >= c["window"])
    p = _softmax(x.masked_fill(hidden[:, None, None, :], -math.inf))
    v = _context(s, b, 1, s["v_scale"]).permute(0, 2, 1, 3)
    return torch.matmul(p, v).view(t, q, d).bfloat16()


def _plain_mla(s):
    b, pos = _owner(s)
    rows = _context(s, b, 0, s["k_scale"])[:, :, 0]
    q = torch.cat([s["q_latent"], s["q_rope"]], -1).float()
    x = torch.matmul(q, rows.transpose(1, 2)).mul_(s["sm_scale"])
    hidden = torch.arange(s["longest"], device="cuda")[None, :] > pos[:, None]
    p = _softmax(x.masked_fill(hidden[:, None, :], -math.inf))
    return torch.matmul(p, rows[:, :, :512]).bfloat16()


# ------------------------------------------------------------------ one pass

def _handle(s):
    """What a serving loop makes once and keeps for its steps: the cache
    descriptor and the attention workspace."""
    if "handle" not in s:
        from gqa_kv_cache_mla_gb300 import kva, kvw

        c, cache = s["case"], s["cache"]
        kind = kvw.DTYPE_BF16 if c["dtype"] == "bf16" else kvw.DTYPE_FP8_E4M3
        desc = kvw.paged_cache(cache, kind, s["table"], s["lens"], s["pages"], 1, c["page"],
                               cache.shape[4], cache.shape[5], cache.stride()[:5],
                               scale=s["k_scale"])
        need = 0
        if c["op"] == "gqa":
            need = kva.kva_gqa_decode_workspace(c["q_heads"], c["kv_heads"], c["head"])
        elif c["op"] == "mla":
            need = kva.kva_mla_decode_workspace(c["heads"])
        s["handle"] = kva, desc, torch.empty(need, device="cuda", dtype=torch.uint8)
    return s["handle"]


def _stored(s):
    """The cache with E4M3 codes as values of their type."""
    cache = s["cache"]
    return cache if cache.dtype == torch.bfloat16 else cache.view(torch.float8_e4m3fn)


def run(s):
    c = s["case"]
    if own:
        kva, desc, space = _handle(s)
        if c["op"] == "append":
            kva.kva_append_qkv_paged(s["q_out"], s["qkv"], s["offsets"], desc, s["freqs"], 0,
                                     q_gamma=s["q_gamma"], k_gamma=s["k_gamma"], epsilon=1e-6,
                                     v_scale=s["v_scale"], interleaved=c["interleaved"],
                                     err_flags=s["flags"])
            return s["q_out"], _stored(s)
        if c["op"] == "gqa":
            kva.kva_gqa_decode_paged(s["out"], s["q"], s["offsets"], desc, 0, s["sm_scale"],
                                     space, v_scale=s["v_scale"], softcap=c["cap"],
                                     window=c["window"], alibi_slopes=s["slopes"],
                                     err_flags=s["flags"])
            return s["out"]
        kva.kva_mla_decode_paged(s["out"], s["q_latent"], s["q_rope"], s["offsets"], desc, 0,
                                 s["sm_scale"], space, err_flags=s["flags"])
        return s["out"]
    if c["op"] == "append":
        _plain_append(s)
        return s["q_out"], _stored(s)
    return _plain_gqa(s) if c["op"] == "gqa" else _plain_mla(s)


# ------------------------------------------------------------------ 64 bits

def _exact_tokens(s):
    """(token, request, position) of every new token, by walking the requests."""
    off, lens, t = s["offsets"].tolist(), s["lens"].tolist(), 0
    for b, prior in enumerate(lens):
        for i in range(off[b + 1] - off[b]):
            yield t, b, prior + i
            t += 1


def _exact_append(s):
    c = s["case"]
    q, kv, d, rope, page = c["q_heads"], c["kv_heads"], c["head"], c["rope"], c["page"]
    where = list(_exact_tokens(s))
    pos = torch.tensor([p for _, _, p in where], device="cuda")
    req = torch.tensor([b for _, b, _ in where], device="cuda")
    x = s["qkv"].double().view(len(where), q + 2 * kv, d).clone()
    for lo, hi, gamma in ((0, q, s["q_gamma"]), (q, q + kv, s["k_gamma"])):
        if gamma is not None:
            part = x[:, lo:hi]
            x[:, lo:hi] = part / (part.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * gamma.double()
    # rotation as a product of complex numbers, by the table's own cosines and sines
    turn = torch.view_as_complex(s["freqs"].double()[pos].view(len(where), 1, rope // 2, 2))
    qk = x[:, :q + kv, :rope]
    first = torch.arange(0, rope, 2) if c["interleaved"] else torch.arange(rope // 2)
    second = first + (1 if c["interleaved"] else rope // 2)
    z = torch.complex(qk[..., first].contiguous(), qk[..., second].contiguous()) * turn
    x[:, :q + kv, first.cuda()] = z.real
    x[:, :q + kv, second.cuda()] = z.imag
    held = _stored(s).double()
    ids = s["table"].long()[req, torch.div(pos, page, rounding_mode="floor")]
    k, v = x[:, q:q + kv], x[:, q + kv:]
    if c["dtype"] != "bf16":
        k, v = (k / s["k_scale"]).clamp(-448, 448), (v / s["v_scale"]).clamp(-448, 448)
    held[ids, 0, 0, pos % page] = k
    held[ids, 1, 0, pos % page] = v
    return x[:, :q], held


def _exact_rows(s, b, lo, hi):
    page = s["case"]["page"]
    at = torch.arange(lo, hi, device="cuda")
    ids = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
    return _stored(s)[ids, :, 0, at % page].double() if s["cache"].dtype == torch.bfloat16 else \
        s["cache"][ids, :, 0, at % page].view(torch.float8_e4m3fn).double()


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    for t, b, pos in _exact_tokens(s):
        if case["op"] == "gqa":
            lo = max(0, pos + 1 - case["window"]) if case["window"] else 0
            rows = _exact_rows(s, b, lo, pos + 1)
            k, v = rows[:, 0] * s["k_scale"], rows[:, 1] * s["v_scale"]
            group = case["q_heads"] // case["kv_heads"]
            qh = s["q"][t].double().view(case["kv_heads"], group, case["head"])
            x = torch.einsum("grd,lgd->grl", qh, k) * s["sm_scale"]
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                far = pos - torch.arange(lo, pos + 1, device="cuda").double()
                x = x - s["slopes"].double().view(case["kv_heads"], group, 1) * far
            out[t] = torch.einsum("grl,lgd->grd", torch.softmax(x, -1), v).reshape(out[t].shape)
        else:
            rows = _exact_rows(s, b, 0, pos + 1)[:, 0, 0] * s["k_scale"]
            x = (s["q_latent"][t].double() @ rows[:, :512].T
                 + s["q_rope"][t].double() @ rows[:, 512:].T) * s["sm_scale"]
            out[t] = torch.softmax(x, -1) @ rows[:, :512]
    return out
