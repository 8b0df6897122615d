"""Measured cases of the cache held in 4 bits and of its page tables.

Four operators, each as a serving loop calls it:

``tables``  before a step: the pages that the new tokens need are taken from
            the list of free ones and written to the page tables, and each
            new token's slot (page * page size + row) is worked out
``append``  the fused projection of a step's new tokens is split into heads,
            queries and keys are rotated, queries go to their own buffer, keys
            and values are quantised (groups of 64 columns of a row share a
            bf16 scale, codes -7 to 7) and written to their slots; what the
            cache then holds of them is read back in bf16, as the attention
            within a prompt's chunk needs it
``gather``  the cached prefix of each request, as contiguous bf16 rows
``gqa``     each new token's query heads attend over the token's whole paged
            context, one key-value head per group of query heads; optional
            tanh cap, sliding window and distance bias

``own`` chooses between the plain form (elementary torch operations in 32
bits) and the framework's entry points.
"""
import math

import numpy as np
import torch

own = False

GOLDEN = 0.6180339887498949
GROUP = 64  # columns that share a scale


def listed():
    return [
        # a decode step of the benchmark's batch of 256: one new token each
        dict(name="tables_decode_256", op="tables", batch=256, new=1, prior=8192, page=64),
        # chunks of 64 prompts at once
        dict(name="tables_prefill", op="tables", batch=64, new=4096, prior=2048, page=16),
        # one chat stream's next token: nothing but latency
        dict(name="append_one", op="append", batch=1, new=1, prior=700, q_heads=32, kv_heads=8,
             head=128, rope=128, page=64, interleaved=False),
        # the Llama-3-8B prefill batch of the benchmark: 32 ragged requests
        dict(name="append_prefill", op="append", batch=32, new=2048, prior=4096, q_heads=32,
             kv_heads=8, head=128, rope=128, page=64, interleaved=True),
        # odd sizes: 96-wide heads of which 64 columns turn, pages of 48 tokens
        dict(name="append_odd", op="append", batch=13, new=301, prior=77, q_heads=10, kv_heads=5,
             head=96, rope=64, page=48, interleaved=False),
        # prefixes of a few long documents, for the next chunks of their prompts
        dict(name="gather_long", op="gather", batch=24, prior=32768, kv_heads=8, head=128, page=64),
        # odd sizes, a few short prefixes
        dict(name="gather_odd", op="gather", batch=5, prior=701, kv_heads=3, head=96, page=48),
        # one chat stream's next token over a short context
        dict(name="gqa_one", op="gqa", batch=1, new=1, prior=900, q_heads=32, kv_heads=8,
             head=128, page=128, cap=0.0, window=0, alibi=False),
        # a decode step of the benchmark's 32 requests
        dict(name="gqa_decode_32", op="gqa", batch=32, new=1, prior=4096, q_heads=32, kv_heads=8,
             head=128, page=128, cap=0.0, window=0, alibi=False),
        # the benchmark's decode batch of 256
        dict(name="gqa_decode_256", op="gqa", batch=256, new=1, prior=8192, q_heads=32,
             kv_heads=8, head=128, page=64, cap=0.0, window=0, alibi=False),
        # few requests with very long contexts
        dict(name="gqa_long", op="gqa", batch=8, new=1, prior=131072, q_heads=64, kv_heads=8,
             head=128, page=128, cap=0.0, window=0, alibi=False),
        # wide heads, capped scores, a sliding window, pages of 48, two tokens per request
        dict(name="gqa_cap_window", op="gqa", batch=48, new=2, prior=9001, q_heads=16,
             kv_heads=8, head=256, page=48, cap=50.0, window=4096, alibi=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "gather", "gqa", "gqa", "gqa"])
    page = rng.choice([16, 32, 48, 64, 80, 128, 256])
    if op == "tables":
        batch = _log(rng, 1, 2048)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(1, min(8192, 200000 // batch))),
                    prior=_log(rng, 1, 16384), page=page)
    head = rng.choice([64, 96, 128, 128, 256])
    if op == "append":
        batch = _log(rng, 1, 256)
        kv = rng.choice([1, 2, 5, 8])
        q = kv * rng.choice([1, 4, 7, 8])
        tokens = 29000 * 48 * 128 // ((q + 4 * kv) * head)
        return dict(op=op, batch=batch, new=_log(rng, 1, max(1, min(2048, 2 * tokens // batch))),
                    prior=_log(rng, 1, min(4096, 98304 // batch)), q_heads=q, kv_heads=kv,
                    head=head, rope=rng.choice([head, 32]), page=page,
                    interleaved=rng.random() < 0.5)
    if op == "gather":
        batch = _log(rng, 1, 256)
        kv = rng.choice([1, 2, 3, 8])
        rows = 24 * 32768 * 8 * 128 // (kv * head * batch)
        return dict(op=op, batch=batch, prior=_log(rng, 16, max(17, min(65536, rows))), kv_heads=kv,
                    head=head, page=page)
    batch = _log(rng, 1, 256)
    new = rng.choice([1, 1, 1, 2, 4])
    kv = rng.choice([1, 2, 4, 8])
    q = kv * rng.choice([1, 4, 5, 8, 16])
    rows = 8 * 131072 * 8 * 128 // (kv * head * batch * new)
    return dict(op=op, batch=batch, new=new, prior=_log(rng, 16, max(17, min(131072, rows))),
                q_heads=q, kv_heads=kv, head=head, page=page, cap=rng.choice([0.0, 0.0, 30.0]),
                window=rng.choice([0, 0, 0, 129, 2048]), alibi=rng.random() < 0.25)


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
    if case["op"] == "gather":
        new = np.zeros(b, np.int64)
    elif case["op"] != "gqa" and case["new"] > 1:
        new = _spread(b, case["new"], 0.25)
    else:
        new = np.full(b, case["new"], np.int64)
    return new, _spread(b, case["prior"], 0.5)


def _groups(case):
    return -(-case["head"] // GROUP)


def work(case):
    new, prior = _lengths(case)
    t, b = int(new.sum()), len(new)
    if case["op"] == "tables":
        page = case["page"]
        have, need = -(-prior // page), -(-(prior + new) // page)
        fresh = int((need - have).sum())
        # offsets, lengths; taken ids read and written; the open pages' ids; slots
        return dict(bytes=8 * b + 8 * fresh + 4 * int((prior % page != 0).sum()) + 8 * t, flops=t)
    kv, d = case["kv_heads"], case["head"]
    row = 2 * kv * (d // 2 + 2 * _groups(case))  # of keys and values as held
    if case["op"] == "append":
        q = case["q_heads"]
        moved = t * ((q + 2 * kv) * d * 2 + q * d * 2 + 2 * row + 2 * kv * d * 2)
        angles = int((prior + new).max() - prior.min()) if t > b else len(np.unique(prior))
        return dict(bytes=moved + angles * case["rope"] * 4,
                    flops=t * ((q + kv) * 3 * case["rope"] + 2 * kv * d * 4))
    if case["op"] == "gather":
        rows = int(prior.sum())
        return dict(bytes=rows * (row + 2 * kv * d * 2), flops=rows * 2 * kv * d)
    window = case["window"] or (1 << 40)
    first = np.maximum(0, prior + 1 - window)
    rows = int((prior + new - first).sum())
    seen = sum(int(np.minimum(prior + 1 + i, window).sum()) for i in range(int(new[0])))
    q = case["q_heads"]
    return dict(bytes=rows * row + 2 * t * q * d * 2, flops=seen * q * 4 * d)


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, std=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std)


def _held_codes(gen, shape):
    """Bytes of two codes, normal values as a group's scale leaves them."""
    out = torch.empty(shape, device="cuda", dtype=torch.uint8)
    for part in out.view(-1).split(1 << 28):  # in pieces: the caches are a few GB
        for i in range(2):
            u = _normal(gen, part.shape, 2.8).round_().clamp_(-7, 7).add_(8).to(torch.uint8)
            part.copy_(u) if i == 0 else part.add_(u.mul_(16))
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    new, prior = _lengths(case)
    b, t, page, op = len(new), int(new.sum()), case["page"], case["op"]
    have, need = -(-prior // page), -(-(prior + new) // page)
    mapped = have if op == "tables" else need
    total, width = int(need.sum()), int(need.max())
    ids = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    used = torch.arange(width, device="cuda")[None, :] < torch.from_numpy(mapped).cuda()[:, None]
    table = torch.full((b, width), -1, device="cuda", dtype=torch.int32)
    table[used] = ids[:int(mapped.sum())]
    offsets = np.concatenate([[0], np.cumsum(new)])
    s = dict(case=case, t=t, table=table, pages=total,
             offsets=torch.from_numpy(offsets.astype(np.int32)).cuda(),
             lens=torch.from_numpy(prior.astype(np.int32)).cuda(),
             flags=torch.zeros(1, device="cuda", dtype=torch.int32), longest=int((prior + new).max()))
    if op == "tables":
        # seven pages of the list are in use already
        s["free"] = torch.cat([ids.new_zeros(7), ids[int(mapped.sum()):]])
        s["taken"] = torch.full((1,), 7, device="cuda", dtype=torch.int32)
        s["taken_out"] = torch.zeros_like(s["taken"])
        s["slots"] = torch.zeros(t, device="cuda", dtype=torch.int64)
        return s
    heads, d, ng = case["kv_heads"], case["head"], _groups(case)
    s["codes"] = _held_codes(gen, (total, 2, 1, heads, page, d // 2))
    s["scales"] = torch.rand((total, 2, 1, heads, ng, page), generator=gen, device="cuda") \
        .mul_(0.3).add_(0.2).bfloat16()  # values of about unit size
    if op == "gather":
        s["ctx"] = torch.from_numpy(np.concatenate([[0], np.cumsum(prior)]).astype(np.int32)).cuda()
        s["rows"] = int(prior.sum())
    elif op == "append":
        q, rope = case["q_heads"], case["rope"]
        s["qkv"] = _normal(gen, (t, (q + 2 * heads) * d)).bfloat16()
        s["q_out"] = torch.zeros((t, q, d), device="cuda", dtype=torch.bfloat16)
        theta = 500000.0 ** (-torch.arange(0, rope, 2, device="cuda", dtype=torch.float64) / rope)
        angle = torch.arange(s["longest"], device="cuda", dtype=torch.float64)[:, None] * theta
        s["freqs"] = torch.stack([angle.cos(), angle.sin()], -1).reshape(-1, rope).float()
        s["rows"] = t
    else:
        q = case["q_heads"]
        s["q"] = _normal(gen, (t, q, d), 2.0).bfloat16()  # scores of standard deviation 2
        s["out"] = torch.zeros((t, q, d), device="cuda", dtype=torch.bfloat16)
        s["sm_scale"] = 1 / math.sqrt(d)
        s["slopes"] = None
        if case["alibi"]:
            s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, q + 1, device="cuda").float() / q)
    if op != "gqa":
        s["k_rows"] = torch.zeros((s["rows"], heads, d), device="cuda", dtype=torch.bfloat16)
        s["v_rows"] = torch.zeros_like(s["k_rows"])
    return s


# ------------------------------------------------------------------ plain form

def _owner(offsets, count, first):
    """Request and position of each of `count` rows."""
    n = offsets.diff().long()
    b = torch.repeat_interleave(torch.arange(len(n), device="cuda"), n, output_size=count)
    at = torch.arange(count, device="cuda") - offsets.long()[b]
    return b, at if first is None else at + first.long()[b]


def _plain_tables(s):
    page = s["case"]["page"]
    lens, n = s["lens"].long(), s["offsets"].diff().long()
    have, need = (lens + page - 1) // page, (lens + n + page - 1) // page
    fresh = need - have
    base = s["taken"].long() + fresh.cumsum(0) - fresh
    b, pos = _owner(s["offsets"], s["t"], s["lens"])
    idx, row = pos // page, pos % page
    new = idx - have[b]
    at = (base[b] + new).clamp(max=len(s["free"]) - 1)
    ids = torch.where(new >= 0, s["free"][at], s["table"][b, idx])
    s["table"][b, idx] = ids
    s["slots"].copy_(ids.long() * page + row)
    s["taken_out"].copy_(s["taken"] + fresh.sum().int())
    return s["table"], s["slots"], s["taken_out"]


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


def _by_group(x):
    """[..., D] as [..., groups, GROUP], a short last group filled with zeros."""
    d = x.shape[-1]
    pad = -d % GROUP
    if pad:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], pad)], -1)
    return x.view(*x.shape[:-1], -1, GROUP)


def _plain_held(x):
    """(bytes of two codes, scales) of rows x [T, heads, D]."""
    g = _by_group(x)
    scale = (g.abs().amax(-1) / 7).bfloat16()
    by = scale.float()[..., None]
    u = torch.where(by > 0, g / by, torch.zeros_like(g)).round().clamp(-7, 7) + 8
    u = u.flatten(-2)[..., :x.shape[-1]].to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4), scale


def _plain_values(codes, scales):
    """fp32 values of codes [..., D / 2] and scales [..., groups]."""
    u = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().sub_(8)
    return u * scales.float().repeat_interleave(GROUP, -1)[..., :u.shape[-1]]


def _plain_rows(s, b, pos, plane):
    page = s["case"]["page"]
    ids, row = s["table"][b, pos // page].long(), pos % page
    return _plain_values(s["codes"][ids, plane, 0, :, row], s["scales"][ids, plane, 0, :, :, row])


def _plain_append(s):
    c = s["case"]
    q, kv, d, page = c["q_heads"], c["kv_heads"], c["head"], c["page"]
    b, pos = _owner(s["offsets"], s["t"], s["lens"])
    x = s["qkv"].float().view(s["t"], q + 2 * kv, d)
    cs = s["freqs"][pos].view(s["t"], -1, 2)
    turned = _plain_rope(x[:, :q + kv], cs, c["interleaved"])
    s["q_out"].copy_(turned[:, :q])
    ids, row = s["table"][b, pos // page].long(), pos % page
    for plane, rows in ((0, turned[:, q:]), (1, x[:, q + kv:])):
        codes, scale = _plain_held(rows)
        s["codes"][ids, plane, 0, :, row] = codes
        s["scales"][ids, plane, 0, :, :, row] = scale
    s["k_rows"].copy_(_plain_rows(s, b, pos, 0))
    s["v_rows"].copy_(_plain_rows(s, b, pos, 1))
    return s["q_out"], s["k_rows"], s["v_rows"]


def _plain_gather(s):
    b, pos = _owner(s["ctx"], s["rows"], None)
    s["k_rows"].copy_(_plain_rows(s, b, pos, 0))
    s["v_rows"].copy_(_plain_rows(s, b, pos, 1))
    return s["k_rows"], s["v_rows"]


def _context(s, b, plane):
    """[tokens, positions, heads, head] rows of the owners' contexts in 32 bits."""
    page = s["case"]["page"]
    at = torch.arange(s["longest"], device="cuda")
    ids = s["table"].long().clamp(min=0)[b][:, at // page]
    return _plain_values(s["codes"][ids, plane, 0, :, at % page],
                         s["scales"][ids, plane, 0, :, :, at % page])


def _softmax(x):
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def _plain_gqa(s):
    c = s["case"]
    q, kv, d, t = c["q_heads"], c["kv_heads"], c["head"], s["t"]
    b, pos = _owner(s["offsets"], t, s["lens"])
    k = _context(s, b, 0).permute(0, 2, 3, 1)
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
    v = _context(s, b, 1).permute(0, 2, 1, 3)
    return torch.matmul(p, v).view(t, q, d).bfloat16()


# ------------------------------------------------------------------ one pass

def _handle(s):
    """What a serving loop makes once and keeps for its steps: the cache
    descriptor and the attention workspace."""
    if "handle" not in s:
        from gqa_kv_cache_mla_gb300 import kva

        c = s["case"]
        cache, scales = kva.int4_cache(s["codes"], s["scales"], s["table"], s["lens"])
        space = None
        if c["op"] == "gqa":
            need = kva.kva_gqa_decode_workspace(c["q_heads"], c["kv_heads"], c["head"])
            space = torch.empty(need, device="cuda", dtype=torch.uint8)
        s["handle"] = kva, cache, scales, space
    return s["handle"]


def run(s):
    c = s["case"]
    if own:
        if c["op"] == "tables":
            from gqa_kv_cache_mla_gb300 import kva

            kva.kva_extend_page_tables(s["table"], s["lens"], s["offsets"], s["free"], s["taken"],
                                       s["taken_out"], c["page"], s["pages"], slot_map=s["slots"],
                                       err_flags=s["flags"])
            return s["table"], s["slots"], s["taken_out"]
        kva, cache, scales, space = _handle(s)
        if c["op"] == "append":
            kva.kva_append_qkv_int4(s["q_out"], s["qkv"], s["offsets"], cache, scales, s["freqs"],
                                    0, interleaved=c["interleaved"], err_flags=s["flags"])
            kva.kva_gather_kv_int4(s["k_rows"], s["v_rows"], s["offsets"], cache, scales, 0,
                                   first_positions=s["lens"], err_flags=s["flags"])
            return s["q_out"], s["k_rows"], s["v_rows"]
        if c["op"] == "gather":
            kva.kva_gather_kv_int4(s["k_rows"], s["v_rows"], s["ctx"], cache, scales, 0,
                                   err_flags=s["flags"])
            return s["k_rows"], s["v_rows"]
        kva.kva_gqa_decode_int4(s["out"], s["q"], s["offsets"], cache, scales, 0, s["sm_scale"],
                                space, softcap=c["cap"], window=c["window"],
                                alibi_slopes=s["slopes"], err_flags=s["flags"])
        return s["out"]
    if c["op"] == "tables":
        return _plain_tables(s)
    if c["op"] == "append":
        return _plain_append(s)
    return _plain_gather(s) if c["op"] == "gather" else _plain_gqa(s)


# ------------------------------------------------------------------ 64 bits

def _exact_tables(s):
    page, table = s["case"]["page"], s["table"].cpu().numpy().copy()
    off, lens = s["offsets"].cpu().numpy(), s["lens"].cpu().numpy().astype(np.int64)
    free, at = s["free"].cpu().numpy(), int(s["taken"])
    slots = np.zeros(s["t"], np.int64)
    for b, prior in enumerate(lens):
        pos = np.arange(prior, prior + off[b + 1] - off[b])
        while at < len(free) and len(pos) and table[b].size > pos[-1] // page \
                and table[b, pos[-1] // page] < 0:
            table[b, int((table[b] >= 0).sum())] = free[at]
            at += 1
        slots[off[b]:off[b + 1]] = table[b, pos // page].astype(np.int64) * page + pos % page
    return (torch.from_numpy(table).cuda(), torch.from_numpy(slots).cuda(),
            torch.tensor([at], dtype=torch.int32).cuda())


def _exact_held(x):
    """Values that the cache holds of rows x [T, heads, D]."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[-1], GROUP):
        part = x[..., lo:lo + GROUP]
        scale = (part.abs().max(-1, keepdim=True).values / 7).bfloat16().double()
        safe = torch.where(scale == 0, torch.ones_like(scale), scale)
        out[..., lo:lo + GROUP] = torch.clamp(torch.round(part / safe), -7, 7) * scale
    return out


def _exact_append(s):
    c = s["case"]
    q, kv, d, rope = c["q_heads"], c["kv_heads"], c["head"], c["rope"]
    pos = torch.cat([torch.arange(p, p + n) for p, n in
                     zip(s["lens"].tolist(), s["offsets"].diff().tolist())]).cuda()
    x = s["qkv"].double().view(len(pos), q + 2 * kv, d).clone()
    # rotation as a product of complex numbers, by the table's own cosines and sines
    turn = torch.view_as_complex(s["freqs"].double()[pos].view(len(pos), 1, rope // 2, 2))
    first = torch.arange(0, rope, 2) if c["interleaved"] else torch.arange(rope // 2)
    second = first + (1 if c["interleaved"] else rope // 2)
    first, second = first.cuda(), second.cuda()
    z = torch.complex(x[:, :q + kv, first], x[:, :q + kv, second]) * turn
    x[:, :q + kv, first] = z.real
    x[:, :q + kv, second] = z.imag
    return x[:, :q], _exact_held(x[:, q:q + kv]), _exact_held(x[:, q + kv:])


def _exact_rows(s, b, lo, hi):
    """Rows lo .. hi - 1 of request b, keys and values [rows, 2, heads, D]."""
    page, d = s["case"]["page"], s["case"]["head"]
    at = torch.arange(lo, hi, device="cuda")
    ids = s["table"][b].long()[torch.div(at, page, rounding_mode="floor")]
    codes = s["codes"][ids, :, 0, :, at % page]
    out = torch.empty(*codes.shape[:-1], d, device="cuda", dtype=torch.float64)
    out[..., 0::2] = torch.remainder(codes, 16).double() - 8
    out[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double() - 8
    scales = s["scales"][ids, :, 0, :, :, at % page].double()
    for g in range(scales.shape[-1]):
        out[..., g * GROUP:(g + 1) * GROUP] *= scales[..., g:g + 1]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    if case["op"] == "append":
        return _exact_append(s)
    if case["op"] == "gather":
        rows = torch.cat([_exact_rows(s, b, 0, n) for b, n in enumerate(s["lens"].tolist())])
        return rows[:, 0], rows[:, 1]
    out = torch.zeros(s["out"].shape, device="cuda", dtype=torch.float64)
    off, lens = s["offsets"].tolist(), s["lens"].tolist()
    group = case["q_heads"] // case["kv_heads"]
    for b, prior in enumerate(lens):
        for t in range(off[b], off[b + 1]):
            pos = prior + t - off[b]
            lo = max(0, pos + 1 - case["window"]) if case["window"] else 0
            rows = _exact_rows(s, b, lo, pos + 1)
            qh = s["q"][t].double().view(case["kv_heads"], group, case["head"])
            x = torch.einsum("grd,lgd->grl", qh, rows[:, 0]) * s["sm_scale"]
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if s["slopes"] is not None:
                far = pos - torch.arange(lo, pos + 1, device="cuda").double()
                x = x - s["slopes"].double().view(case["kv_heads"], group, 1) * far
            out[t] = torch.einsum("grl,lgd->grd", torch.softmax(x, -1),
                                  rows[:, 1]).reshape(out[t].shape)
    return out
