"""Operators of a serving step over a paged KV cache, for measurement.

Four operators that follow one another in a server's layer: the page tables
and slot map of a step (built once for all layers), the rotation of the new
tokens with their append to the paged cache, causal attention over packed
prompts, and attention of new tokens (a chunk, or one token) over the pages.

``run`` computes them in plain torch operations, or through
``long_context_blockwise_max_b200.serving`` where ``own`` is true.
"""
import math
import random

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the tables of one generation step: 64 requests, one token each
        dict(name="schedule-decode-64", op="schedule", batch=64, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=32768, page=16, lens=11),
        # a step that mixes prompts and generation, 512 requests
        dict(name="schedule-mixed-512", op="schedule", batch=512, q_lo=1, q_hi=2048, ctx_lo=0, ctx_hi=8192, page=64, lens=12),
        # 16 generated tokens behind 128K contexts (the batch of the 128K decode)
        dict(name="append-decode-16", op="append", dtype="bf16", tokens=16, hq=32, hkv=8, d=128, page=16, base=131072, theta=500000.0),
        # the tokens of a 32K prompt
        dict(name="append-prompt-32k", op="append", dtype="bf16", tokens=32768, hq=32, hkv=8, d=128, page=64, base=0, theta=500000.0),
        # the fp32 configuration's 2048-token sequence
        dict(name="prompt-2k-fp32", op="prompt", dtype="fp32", batch=1, lo=2048, hi=2048, hq=4, hkv=2, d=64, lens=13),
        # a packed batch of prompts of odd lengths, 1 to 4096 tokens
        dict(name="prompt-ragged-24", op="prompt", dtype="bf16", batch=24, lo=1, hi=4096, hq=32, hkv=8, d=128, lens=14),
        # one 32K prompt
        dict(name="prompt-32k", op="prompt", dtype="bf16", batch=1, lo=32768, hi=32768, hq=32, hkv=8, d=128, lens=15),
        # one token of each of 8 short requests: latency
        dict(name="attend-decode-8", op="attend", dtype="bf16", batch=8, q_lo=1, q_hi=1, ctx_lo=0, ctx_hi=2048, hq=32, hkv=8, d=128, page=16, lens=16),
        # one token of each of 16 requests of 128K keys: the cache's bytes count
        dict(name="attend-decode-128k", op="attend", dtype="bf16", batch=16, q_lo=1, q_hi=1, ctx_lo=131071, ctx_hi=131071, hq=32, hkv=8, d=128, page=64, lens=17),
        # a 64-token query over a 128K cache
        dict(name="attend-query-64", op="attend", dtype="bf16", batch=1, q_lo=64, q_hi=64, ctx_lo=131072, ctx_hi=131072, hq=32, hkv=8, d=128, page=16, lens=18),
        # prompt chunks and generated tokens of 32 requests in one call
        dict(name="attend-mixed-32", op="attend", dtype="bf16", batch=32, q_lo=1, q_hi=512, ctx_lo=0, ctx_hi=8192, hq=32, hkv=8, d=128, page=16, lens=19),
        # the fp32 configuration's heads, 32-token queries
        dict(name="attend-query-fp32", op="attend", dtype="fp32", batch=4, q_lo=1, q_hi=32, ctx_lo=512, ctx_hi=2048, hq=4, hkv=2, d=64, page=32, lens=20),
    ]


def _log_int(rng, lo, hi):
    """Spread over the logarithm of [lo, hi], zero among them."""
    return min(hi, max(lo, int(math.exp(rng.uniform(math.log(lo + 1), math.log(hi + 2))) - 1)))


def draw(rng):
    op = rng.choice(["schedule", "append", "prompt", "prompt", "attend", "attend", "attend"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    hq, hkv = rng.choice([(32, 8), (32, 8), (8, 8), (16, 2), (12, 4), (28, 4), (8, 1), (5, 1), (4, 2), (32, 1)])
    d = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    lens = rng.randrange(1 << 30)
    if op == "schedule":
        q_hi = rng.choice([1, _log_int(rng, 2, 2048)])
        return dict(op=op, batch=_log_int(rng, 1, 1024), q_lo=rng.choice([0, 1]) if q_hi > 1 else 1, q_hi=q_hi, ctx_lo=0, ctx_hi=_log_int(rng, 16, 32768), page=page, lens=lens)
    if op == "append":
        return dict(op=op, dtype=dtype, tokens=_log_int(rng, 1, 16384), hq=hq, hkv=hkv, d=d, page=page, base=_log_int(rng, 0, 1 << 20), theta=rng.choice([10000.0, 500000.0]))
    if op == "prompt":
        hi = _log_int(rng, 1, 16384 if dtype == "bf16" else 4096)
        batch = _log_int(rng, 1, max(1, min(64, 32768 // hi)))
        return dict(op=op, dtype=dtype, batch=batch, lo=rng.choice([1, max(1, hi // 2)]), hi=hi, hq=hq, hkv=hkv, d=d, lens=lens)
    q_hi = rng.choice([1, 1, _log_int(rng, 2, 1024)])
    ctx_hi = _log_int(rng, 1, 131072 if dtype == "bf16" else 16384)
    batch = _log_int(rng, 1, max(1, min(128, (1 << 20) // (ctx_hi + 16 * q_hi))))
    return dict(op=op, dtype=dtype, batch=batch, q_lo=1, q_hi=q_hi, ctx_lo=rng.choice([0, ctx_hi // 2]), ctx_hi=ctx_hi, hq=hq, hkv=hkv, d=d, page=page, lens=lens)


def _lengths(case):
    """(new tokens, tokens in the cache before) of each request, as the case has them."""
    rng = random.Random(case["lens"])
    if case["op"] == "prompt":
        return [_log_int(rng, case["lo"], case["hi"]) for _ in range(case["batch"])], [0] * case["batch"]
    q = [_log_int(rng, case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return q, [_log_int(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]


# --------------------------------------------------------------- the inputs
def _i32(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"op": case["op"]}
    if case["op"] == "append":
        dt, n, p = _TYPES[case["dtype"]], case["tokens"], case["page"]
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        pages = -(-n // p) + 8
        # q, k and v as one fused projection leaves them: slices of a row
        fused = torch.randn((n, hq + 2 * hkv, d), generator=gen, device=dev).to(dt)
        s["q"], s["k"], s["v"] = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        s["positions"] = (case["base"] + torch.arange(n, device=dev)).to(torch.int32)
        order = torch.randperm(pages, generator=gen, device=dev)
        tok = torch.arange(n, device=dev)
        s["slots"] = (order[tok // p] * p + tok % p).to(torch.int32)
        s["k_pages"] = torch.zeros((pages, p, hkv, d), dtype=dt, device=dev)
        s["v_pages"] = torch.zeros((pages, p, hkv, d), dtype=dt, device=dev)
        s["theta"] = case["theta"]
        return s
    q_len, ctx = _lengths(case)
    n = sum(q_len)
    if case["op"] == "schedule":
        p = case["page"]
        # the same requests in another order, so that another seed is another step
        order = list(range(len(ctx)))
        random.Random(seed).shuffle(order)
        ctx = [ctx[i] for i in order]
        held = [-(-c // p) for c in ctx]
        need = [-(-(c + m) // p) - h for c, m, h in zip(ctx, q_len, held)]
        width = -(-(case["ctx_hi"] + case["q_hi"]) // p)
        pool = torch.randperm(sum(held) + sum(need) + 8, generator=gen, device=dev).to(torch.int32)
        col = torch.arange(width, device=dev)
        mine = col[None] < _i32(held, dev)[:, None]
        at = torch.cumsum(_i32(held, dev), 0)[:, None] - _i32(held, dev)[:, None] + col[None]
        s["block_table"] = torch.where(mine, pool[at.clamp(max=pool.numel() - 1)], -1).to(torch.int32).contiguous()
        s["free_pages"] = pool[sum(held):].contiguous()
        s["q_len"], s["kv_len"], s["page"], s["tokens"] = _i32(q_len, dev), _i32(ctx, dev), p, n
        return s
    dt, hq, hkv, d = _TYPES[case["dtype"]], case["hq"], case["hkv"], case["d"]
    cu = [0]
    for m in q_len:
        cu.append(cu[-1] + m)
    s["cu_q"], s["max_q"], s["batch"] = _i32(cu, dev), max(q_len), len(q_len)
    s["q"] = torch.randn((n, hq, d), generator=gen, device=dev).to(dt)
    if case["op"] == "prompt":
        s["k"] = torch.randn((n, hkv, d), generator=gen, device=dev).to(dt)
        s["v"] = torch.randn((n, hkv, d), generator=gen, device=dev).to(dt)
        return s
    p = case["page"]
    kv = [c + m for c, m in zip(ctx, q_len)]
    held = [-(-c // p) for c in kv]
    width = max(held) + 1
    pages = sum(held) + 4
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    col = torch.arange(width, device=dev)
    mine = col[None] < _i32(held, dev)[:, None]
    at = torch.cumsum(_i32(held, dev), 0)[:, None] - _i32(held, dev)[:, None] + col[None]
    s["block_table"] = torch.where(mine, order[at.clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    s["kv_len"], s["max_kv"] = _i32(kv, dev), max(kv)
    s["k_pages"] = torch.empty((pages, p, hkv, d), dtype=dt, device=dev).normal_(generator=gen)
    s["v_pages"] = torch.empty((pages, p, hkv, d), dtype=dt, device=dev).normal_(generator=gen)
    return s


# ----------------------------------------------------------------- one pass
def run(s):
    if own:
        from long_context_blockwise_max_b200 import serving
        if s["op"] == "schedule":
            cu, kv, pos, slots, used, _ = serving.pa_paged_schedule(s["q_len"], s["kv_len"], s["block_table"], s["free_pages"], s["page"], s["tokens"])
            return {"cu_q": cu, "kv_len": kv, "positions": pos, "slots": slots, "used": used, "block_table": s["block_table"]}
        if s["op"] == "append":
            q, _, _ = serving.pa_paged_append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pages"], s["v_pages"], rope_theta=s["theta"])
            return {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
        if s["op"] == "prompt":
            o, lse, _ = serving.pa_prompt_attend(s["q"], s["k"], s["v"], s["cu_q"])
            return {"o": o, "lse": lse}
        o, lse, _ = serving.pa_paged_attend(s["q"], s["cu_q"], s["kv_len"], s["block_table"], s["k_pages"], s["v_pages"], s["max_q"])
        return {"o": o, "lse": lse}
    return {"schedule": _schedule, "append": _append, "prompt": _prompt, "attend": _attend}[s["op"]](s)


def _schedule(s):
    p, n, dev = s["page"], s["tokens"], s["q_len"].device
    q, kv, table, free = s["q_len"].long(), s["kv_len"].long(), s["block_table"], s["free_pages"]
    cu = torch.nn.functional.pad(torch.cumsum(q, 0), (1, 0))
    held = (kv + p - 1) // p
    need = (kv + q + p - 1) // p - held
    ends = torch.cumsum(need, 0)
    # the new pages of each request, in its order, behind those that it holds
    col = torch.arange(table.shape[1], device=dev)[None]
    nth = col - held[:, None]
    new = (nth >= 0) & (nth < need[:, None])
    at = (ends - need)[:, None] + nth
    table.copy_(torch.where(new, free[at.clamp(0, free.numel() - 1)], table))
    tok = torch.arange(n, device=dev)
    b = torch.searchsorted(cu[1:], tok, right=True)
    pos = kv[b] + tok - cu[b]
    slots = table[b, pos // p].long() * p + pos % p
    return {"cu_q": cu.int(), "kv_len": (kv + q).int(), "positions": pos.int(), "slots": slots.int(), "used": ends[-1:].int(), "block_table": table}


def _rotated(x, positions, theta):
    """Rotate-half RoPE in 32 bits, angles in 64."""
    half = x.shape[-1] // 2
    omega = theta ** (-torch.arange(half, dtype=torch.float64, device=x.device) / half)
    angle = positions.double()[:, None, None] * omega
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    a, b = x[..., :half].float(), x[..., half:].float()
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1).to(x.dtype)


def _append(s):
    hkv, d = s["k"].shape[1:]
    slots = s["slots"].long()
    s["k_pages"].view(-1, hkv, d)[slots] = _rotated(s["k"], s["positions"], s["theta"])
    s["v_pages"].view(-1, hkv, d)[slots] = s["v"]
    return {"q": _rotated(s["q"], s["positions"], s["theta"]), "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attention(q, k, v, first, cu, max_q, base):
    """Row i of request b sees its keys 0 .. first[b] + i. q packed [n][hq][d]; k and v in 32 bits,
    padded [batch][length][hkv][d]; base: the largest of first. Blocks of rows, so that the scores fit."""
    n, hq, d = q.shape
    batch, length, hkv, _ = k.shape
    g, dev = hq // hkv, q.device
    kt, vt = k.permute(0, 2, 3, 1), v.permute(0, 2, 1, 3)
    tok = torch.arange(n, device=dev)
    b = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[b]
    rows = torch.zeros((batch, max_q, hq, d), device=dev)
    rows[b, i] = q.float()
    o, lse = torch.empty_like(rows), torch.empty((batch, max_q, hq), device=dev)
    step = max(1, min(max_q, (1 << 30) // (batch * hq * length)))
    for r in range(0, max_q, step):
        m = min(step, max_q - r)
        end = min(length, base + r + m)
        x = rows[:, r:r + m].view(batch, m, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(batch, hkv, g * m, d)
        x = (x @ kt[..., :end] / math.sqrt(d)).view(batch, hkv, g, m, end)
        seen = torch.arange(end, device=dev) <= (first[:, None] + torch.arange(r, r + m, device=dev))[..., None]
        x = x.masked_fill_(~seen[:, None, None], -math.inf)
        top = x.amax(-1, keepdim=True)
        x = x.sub_(top).exp_()
        total = x.sum(-1, keepdim=True)
        y = (x.view(batch, hkv, g * m, end) @ vt[:, :, :end]).view(batch, hkv, g, m, d) / total
        o[:, r:r + m] = y.permute(0, 3, 1, 2, 4).reshape(batch, m, hq, d)
        lse[:, r:r + m] = (top + total.log())[..., 0].permute(0, 3, 1, 2).reshape(batch, m, hq)
    return {"o": o[b, i].to(q.dtype), "lse": lse[b, i]}


def _prompt(s):
    cu = s["cu_q"].long()
    tok = torch.arange(s["q"].shape[0], device=cu.device)
    b = torch.searchsorted(cu[1:], tok, right=True)
    i = tok - cu[b]
    k = torch.zeros((s["batch"], s["max_q"], *s["k"].shape[1:]), device=cu.device)
    v = torch.zeros_like(k)
    k[b, i], v[b, i] = s["k"].float(), s["v"].float()
    return _attention(s["q"], k, v, torch.zeros_like(cu[1:]), cu, s["max_q"], 0)


def _attend(s):
    cu = s["cu_q"].long()
    _, p, hkv, d = s["k_pages"].shape
    table = s["block_table"][:, :-(-s["max_kv"] // p)].long()
    k = s["k_pages"][table].view(s["batch"], -1, hkv, d).float()
    v = s["v_pages"][table].view(s["batch"], -1, hkv, d).float()
    first = s["kv_len"].long() - (cu[1:] - cu[:-1])
    return _attention(s["q"], k, v, first, cu, s["max_q"], s["max_kv"])


# ------------------------------------------------------------------ its work
def work(case):
    if case["op"] == "append":
        size, n, d = (2, 4)[case["dtype"] == "fp32"], case["tokens"], case["d"]
        rotated = (case["hq"] + case["hkv"]) * d
        return {"bytes": n * (2 * size * (rotated + case["hkv"] * d) + 8), "flops": 3 * n * rotated}
    q, ctx = _lengths(case)
    n, batch = sum(q), len(q)
    if case["op"] == "schedule":
        p = case["page"]
        new = sum(-(-(c + m) // p) + -c // p for c, m in zip(ctx, q))
        # lengths in and out, the new pages from the free list into the table, a position and a slot each token
        return {"bytes": 16 * batch + 8 * new + 8 * n, "flops": 4 * n}
    size, hq, hkv, d = (2, 4)[case["dtype"] == "fp32"], case["hq"], case["hkv"], case["d"]
    seen = sum(m * c + m * (m + 1) // 2 for c, m in zip(ctx, q))
    keys = sum(c + m for c, m in zip(ctx, q))
    pages = sum(-(-(c + m) // case["page"]) for c, m in zip(ctx, q)) if case["op"] == "attend" else 0
    return {"bytes": 2 * size * d * (n * hq + keys * hkv) + 4 * (n * hq + pages + 2 * batch), "flops": 4 * d * hq * seen}


# ------------------------------------------------- the definition, in 64 bits
def exact(case, seed):
    if case["op"] == "schedule":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        hkv, d = s["k"].shape[1:]
        pair = torch.arange(d // 2, device="cuda", dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * torch.exp(-2 * pair / d * math.log(s["theta"])))

        def spun(x):
            z = torch.complex(x[..., :d // 2].double(), x[..., d // 2:].double()) * turn[:, None]
            return torch.cat([z.real, z.imag], -1)

        out = {"q": spun(s["q"])}
        for name, rows in (("k_pages", spun(s["k"])), ("v_pages", s["v"].double())):
            pages = s[name].double()
            pages.view(-1, hkv, d).index_copy_(0, s["slots"].long(), rows)
            out[name] = pages
        return out
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    new, ctx = _lengths(case)
    o = torch.empty((sum(new), hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((sum(new), hq), dtype=torch.float64, device="cuda")
    begin = 0
    for b, (m, c) in enumerate(zip(new, ctx)):
        if case["op"] == "prompt":
            k, v = s["k"][begin:begin + m], s["v"][begin:begin + m]
        else:
            at = torch.arange(c + m, device="cuda")
            page = s["block_table"][b].long()[at // case["page"]]
            k, v = s["k_pages"][page, at % case["page"]], s["v_pages"][page, at % case["page"]]
        for h in range(hkv):
            kh, vh = k[:, h].double(), v[:, h].double()
            heads = slice(h * (hq // hkv), (h + 1) * (hq // hkv))
            for r in range(0, m, 2048):
                end = min(m, r + 2048)
                sees = c + end
                x = torch.einsum("thd,kd->htk", s["q"][begin + r:begin + end, heads].double(), kh[:sees]) * d ** -0.5
                x += torch.full((end - r, sees), -math.inf, dtype=torch.float64, device="cuda").triu(c + r + 1)
                z = torch.logsumexp(x, -1)
                o[begin + r:begin + end, heads] = torch.einsum("htk,kd->thd", torch.exp(x - z[..., None]), vh[:sees])
                lse[begin + r:begin + end, heads] = z.T
        begin += m
    return {"o": o, "lse": lse}
