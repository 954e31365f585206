"""Cases, inputs and plain forms of the attention layer's operators: the block plan of a paged 8-bit KV
cache, the append that quantizes new keys and values into it, attention over it, and the residual norms
around a block.

    listed()             the named cases;  draw(rng)  one more of the same ranges
    prepare(case, seed)  inputs on the GPU
    run(state)           one pass: the plain forms, or the library's calls where ``own`` is true
    work(case)           compulsory bytes and operations of one pass
    exact(case, seed)    the definitions in 64 bits

The cache holds E4M3 codes in pages of ``page`` tokens, [pages, kv heads, page, 128], and one power-of-two
scale per page and head, as a byte: a value is code * 2^(byte - 127). A slot is page_number * page + offset.
"""

from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

D = 128          # head width
LOW, HIGH = -40, 40   # exponents a page's scale can take


def listed():
    return [
        # one decode step of a full batch: latency is all that counts
        dict(name="plan_step", op="plan", lens=1, batch=64, page=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=32000),
        # a large mixed batch: prompts' chunks of every length next to single tokens
        dict(name="plan_batch", op="plan", lens=2, batch=2048, page=16, q_lo=1, q_hi=256, ctx_lo=0, ctx_hi=8000),
        # the keys and values of one decode step: each token lands in a page of its own
        dict(name="append_step", op="append", lens=3, batch=128, page=64, q_lo=1, q_hi=1, ctx_lo=1, ctx_hi=2000,
             kv_heads=8),
        # ragged prompts, some continued in the middle of a page
        dict(name="append_prompts", op="append", lens=4, batch=16, page=64, q_lo=64, q_hi=4096, ctx_lo=0, ctx_hi=500,
             kv_heads=8),
        # around the blocks of the dense 5120-wide model: a decode step of 16 tokens
        dict(name="norm_step", op="norm", rows=16, width=5120, gate="channel", weights="bf16", out="codes"),
        # the same at prefill
        dict(name="norm_prefill", op="norm", rows=8192, width=5120, gate="channel", weights="bf16", out="codes"),
        # an odd width, a gate per token, and a BF16 result next to the codes
        dict(name="norm_odd", op="norm", rows=949, width=2072, gate="token", weights="f32", out="both"),
        # one user's decode step behind a 949-token prompt, 64 query heads on 8 KV heads
        dict(name="attn_one", op="attn", lens=5, batch=1, page=64, q_lo=1, q_hi=1, ctx_lo=949, ctx_hi=949, heads=64,
             kv_heads=8, window=-1),
        # a serving batch's decode step, lengths from short chats to long documents
        dict(name="attn_ragged", op="attn", lens=6, batch=64, page=64, q_lo=1, q_hi=1, ctx_lo=100, ctx_hi=32000,
             heads=64, kv_heads=8, window=-1),
        # three drafted tokens per request verified at once: few heads per KV head, a window, small pages
        dict(name="attn_draft", op="attn", lens=7, batch=17, page=16, q_lo=3, q_hi=3, ctx_lo=700, ctx_hi=16000,
             heads=32, kv_heads=16, window=4001),
        # a prompt of 4096 tokens, as the attention projections are measured at
        dict(name="attn_prompt", op="attn", lens=8, batch=1, page=128, q_lo=4096, q_hi=4096, ctx_lo=0, ctx_hi=0,
             heads=64, kv_heads=8, window=-1),
        # chunks of prompts behind cached prefixes, next to single tokens
        dict(name="attn_chunks", op="attn", lens=9, batch=6, page=32, q_lo=1, q_hi=949, ctx_lo=20, ctx_hi=6000,
             heads=64, kv_heads=8, window=-1),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]; lo may be 0."""
    lo, hi = lo + 1, hi + 1
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))) - 1


def _span(rng, lo, hi):
    """A range of lengths: its end spread over the logarithm of [lo, hi], its start at a share of that."""
    end = _log(rng, lo, hi)
    return end // rng.choice([1, 3, 10, 100]), end


def draw(rng):
    op = rng.choice(["plan", "append", "norm", "attn", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        width = rng.choice([2048, 5120, _log(rng, 100, 8192)])
        return dict(op=op, rows=_log(rng, 1, 5000), width=width, gate=rng.choice(["none", "channel", "token"]),
                    weights=rng.choice(["bf16", "f32"]), out=rng.choice(["codes", "both", "bf16"]))
    case = dict(op=op, lens=rng.randrange(1 << 30), page=page)
    if op == "plan":
        (ctx_lo, ctx_hi), (q_lo, q_hi) = _span(rng, 10, 8000), _span(rng, 1, 256)
        return dict(case, batch=_log(rng, 1, 2048), q_lo=q_lo, q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi)
    case["kv_heads"] = rng.choice([1, 2, 4, 8])
    if op == "append":
        (ctx_lo, ctx_hi), (q_lo, q_hi) = _span(rng, 1, 2000), _span(rng, 1, 4096)
        return dict(case, batch=_log(rng, 1, 16), q_lo=max(1, q_lo), q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi)
    case |= dict(heads=case["kv_heads"] * rng.choice([1, 2, 4, 5, 8]), window=rng.choice([-1, -1, _log(rng, 16, 4000)]))
    if rng.random() < 0.5:                           # a decode step, a few drafted tokens in some
        q = rng.choice([1, 1, 2, 4])
        ctx_lo, ctx_hi = _span(rng, 100, 30000)
        return dict(case, batch=_log(rng, 1, 64), q_lo=q, q_hi=q, ctx_lo=ctx_lo, ctx_hi=ctx_hi)
    (ctx_lo, ctx_hi), (q_lo, q_hi) = _span(rng, 1, 4000), _span(rng, 20, 2000)
    batch = _log(rng, 1, 4)
    while batch > 1 and batch * q_hi * (ctx_hi + q_hi / 2) > 4096 * 2048:
        batch -= 1
    return dict(case, batch=batch, q_lo=max(1, q_lo), q_hi=q_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi)


def _lengths(case):
    """Tokens in the cache before this step and new ones, of each request: the case's own, whatever the seed."""
    rng = random.Random(case["lens"])
    ctx = [_log(rng, case["ctx_lo"], case["ctx_hi"]) for _ in range(case["batch"])]
    new = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return ctx, new


def _pages(n, page):
    return -(-n // page)


# ---- inputs ----------------------------------------------------------------


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _scatter_pages(counts, width, perm):
    """A block table [requests, width]: row b holds its counts[b] pages, taken from perm in order; -1 behind them."""
    n = torch.tensor(counts, dtype=torch.int64, device="cuda")
    at = (torch.cumsum(n, 0) - n)[:, None] + torch.arange(width, device="cuda")[None]
    have = torch.arange(width, device="cuda")[None] < n[:, None]
    return torch.where(have, perm[at.clamp(max=perm.numel() - 1)], -1).to(torch.int32).contiguous()


def _prepare_plan(case, g):
    ctx, new = _lengths(case)
    page = case["page"]
    before = [_pages(c, page) for c in ctx]
    after = [_pages(c + n, page) for c, n in zip(ctx, new)]
    total = sum(after) + 7
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    width = max(after) + 3
    tokens = max(1, _pages(sum(new), 64) * 64)       # a captured step's fixed token count
    return dict(case, ctx=_i32(ctx), new=_i32(new), free=perm[sum(before):].contiguous(),
                table=_scatter_pages(before, width, perm), tokens=tokens,
                q_offsets=torch.empty(len(ctx) + 1, dtype=torch.int32, device="cuda"),
                kv_len=torch.empty(len(ctx), dtype=torch.int32, device="cuda"),
                slots=torch.empty(tokens, dtype=torch.int64, device="cuda"),
                positions=torch.empty(tokens, dtype=torch.int32, device="cuda"),
                counts=torch.empty(3, dtype=torch.int32, device="cuda"))


def _random_cache(pages, heads, page, g):
    """Codes as pages of N(0, 1)-like values leave them, and their scales' bytes."""
    codes = torch.empty(pages, heads, page, D, dtype=torch.float8_e4m3fn, device="cuda")
    for p in range(0, pages, 1024):
        part = torch.randn(codes[p:p + 1024].shape, generator=g, device="cuda")
        codes[p:p + 1024] = (part * 85).clamp_(-448, 448).to(torch.float8_e4m3fn)
    exps = torch.randint(119, 122, (pages, heads), generator=g, device="cuda", dtype=torch.int32).to(torch.uint8)
    return codes.view(torch.uint8), exps


def _new_kv(tokens, heads, g):
    """Keys (a few channels far larger than the rest) and values, as rows of one projection's output."""
    kv = torch.randn(tokens, 2, heads, D, generator=g, device="cuda")
    loud = torch.randint(0, D, (heads, 2), generator=g, device="cuda")
    kv[:, 0].scatter_(2, loud[None].expand(tokens, -1, -1), 12.0)
    kv = kv.to(torch.bfloat16)
    return kv[:, 0], kv[:, 1]


def _prepare_append(case, g):
    ctx, new = _lengths(case)
    page, heads = case["page"], case["kv_heads"]
    after = [_pages(c + n, page) for c, n in zip(ctx, new)]
    total = sum(after) + 3
    table = _scatter_pages(after, max(after), torch.randperm(total, generator=g, device="cuda")).to(torch.int64)
    req = torch.repeat_interleave(torch.arange(len(new)), torch.tensor(new)).cuda()
    first = torch.tensor([sum(new[:b]) for b in range(len(new))], device="cuda")
    pos = torch.arange(sum(new), device="cuda") - first[req] + torch.tensor(ctx, device="cuda")[req]
    slots = table[req, pos // page] * page + pos % page
    k, v = _new_kv(sum(new), heads, g)
    kc, ke = _random_cache(total, heads, page, g)
    vc, ve = _random_cache(total, heads, page, g)
    return dict(case, k=k, v=v, slots=slots, k_cache=kc, v_cache=vc, k_exp=ke, v_exp=ve)


def _prepare_norm(case, g):
    rows, width = case["rows"], case["width"]
    wt = torch.bfloat16 if case["weights"] == "bf16" else torch.float32

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    loud = torch.randint(0, width, (max(1, width // 200),), generator=g, device="cuda")
    res = randn(rows, width)
    res[:, loud] *= 30.0                             # the residual stream's outlier channels
    s = dict(case, y=(0.3 * randn(rows, width)).to(torch.bfloat16), res=res.to(torch.bfloat16),
             w_post=(1 + 0.2 * randn(width)).to(wt), w_pre=(1 + 0.2 * randn(width)).to(wt), gate_t=None,
             res_scale=0.875, eps=1e-6, res_out=torch.empty(rows, width, dtype=torch.bfloat16, device="cuda"),
             q=None, scales=None, n=None)
    if case["gate"] != "none":
        s["gate_t"] = torch.sigmoid(randn(*((width,) if case["gate"] == "channel" else (rows, width)))).to(torch.bfloat16)
    if case["out"] != "bf16":
        s["q"] = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(rows, _pages(width, 128), dtype=torch.float32, device="cuda")
    if case["out"] != "codes":
        s["n"] = torch.empty(rows, width, dtype=torch.bfloat16, device="cuda")
    return s


def _prepare_attn(case, g):
    ctx, new = _lengths(case)
    page, heads, kv_heads, tokens = case["page"], case["heads"], case["kv_heads"], sum(new)
    kv_len = [c + n for c, n in zip(ctx, new)]
    used = [_pages(n, page) for n in kv_len]
    total = sum(used) + 3
    table = _scatter_pages(used, max(used) + 2, torch.randperm(total, generator=g, device="cuda"))
    kc, ke = _random_cache(total, kv_heads, page, g)
    vc, ve = _random_cache(total, kv_heads, page, g)
    # what is behind a request's last token in its last page was never written: NaN codes here
    last = table[torch.arange(len(used), device="cuda"), torch.tensor([u - 1 for u in used], device="cuda")].long()
    fill = torch.tensor([n - (u - 1) * page for n, u in zip(kv_len, used)], device="cuda")
    unwritten = (torch.arange(page, device="cuda")[None] >= fill[:, None])[:, None, :, None]
    for c in (kc, vc):
        c[last] = torch.where(unwritten, 0x7F, c[last])
    offsets = [sum(new[:b]) for b in range(len(new) + 1)]
    # queries as the leading columns of a fused projection's rows
    qkv = torch.randn(tokens, heads + 2 * kv_heads, D, generator=g, device="cuda").to(torch.bfloat16)
    s = dict(case, q=qkv[:, :heads], k_cache=kc, v_cache=vc, k_exp=ke, v_exp=ve, table=table, q_offsets=_i32(offsets),
             kv_len=_i32(kv_len), new=new, lengths=kv_len, scale=1.0 / math.sqrt(D),
             out=torch.empty(tokens, heads, D, dtype=torch.bfloat16, device="cuda"),
             lse=torch.empty(tokens, heads, dtype=torch.float32, device="cuda"))
    if own:                                          # the scratch that a serving program keeps
        from block_scaled_fp8_token_gb300 import bfp8
        s["ws"] = torch.empty(bfp8.bfp8_kv_attention_workspace(len(new), tokens, max(new), heads, kv_heads),
                              dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"plan": _prepare_plan, "append": _prepare_append, "norm": _prepare_norm, "attn": _prepare_attn}[case["op"]](case, g)


# ---- the library's calls -----------------------------------------------------


def _own_plan(s, lib):
    lib.bfp8_kv_plan(s["ctx"], s["new"], s["free"], s["table"], s["page"], s["q_offsets"], s["kv_len"], s["slots"],
                     s["positions"], s["counts"])
    return {k: s[k] for k in ("table", "q_offsets", "kv_len", "slots", "positions", "counts")}


def _cache_values(s):
    return dict(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn), k_exp=s["k_exp"],
                v_exp=s["v_exp"])


def _own_append(s, lib):
    lib.bfp8_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"])
    return _cache_values(s)


def _norm_values(s):
    r = dict(residual=s["res_out"])
    if s["q"] is not None:
        r |= dict(codes=s["q"].view(torch.float8_e4m3fn), scales=s["scales"])
    if s["n"] is not None:
        r["normed"] = s["n"]
    return r


def _own_norm(s, lib):
    lib.bfp8_residual_norm(s["y"], s["res"], s["res_out"], q=s["q"], scales=s["scales"], norm_out=s["n"],
                           w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate_t"], residual_scale=s["res_scale"],
                           eps=s["eps"])
    return _norm_values(s)


def _own_attn(s, lib):
    lib.bfp8_kv_attention(s["q"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["table"], s["q_offsets"],
                          s["kv_len"], s["out"], max(s["new"]), softmax_scale=s["scale"], window=s["window"],
                          lse=s["lse"], workspace=s["ws"])
    return dict(out=s["out"], lse=s["lse"])


# ---- the plain forms -----------------------------------------------------------


def _plain_plan(s):
    page, ctx, new, tokens, dev = s["page"], s["ctx"].long(), s["new"].long(), s["tokens"], s["ctx"].device
    before, after = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    need = after - before
    page_at = torch.cumsum(need, 0) - need           # this request's first page in the free list
    width = s["table"].shape[1]
    j = torch.arange(width, device=dev)[None]
    fresh = (j >= before[:, None]) & (j < after[:, None])
    which = (page_at[:, None] + j - before[:, None]).clamp(0, s["free"].numel() - 1)
    s["table"].copy_(torch.where(fresh, s["free"][which], s["table"]))
    ends = torch.cumsum(new, 0)
    t = torch.arange(tokens, device=dev)
    req = torch.searchsorted(ends, t, right=True)
    real, req = req < ends.numel(), req.clamp(max=ends.numel() - 1)
    pos = ctx[req] + t - (ends - new)[req]
    slot = s["table"][req, (pos // page).clamp(0, width - 1)].long() * page + pos % page
    s["slots"].copy_(torch.where(real, slot, -1))
    s["positions"].copy_(torch.where(real, pos, -1))
    s["q_offsets"].copy_(torch.cat([torch.zeros_like(ends[:1]), ends]))
    s["kv_len"].copy_(ctx + new)
    s["counts"].copy_(torch.stack([need.sum(), torch.zeros_like(ends[0]), torch.zeros_like(ends[0])]))
    return {k: s[k] for k in ("table", "q_offsets", "kv_len", "slots", "positions", "counts")}


def _plain_append_one(x, slots, codes, exps):
    pages, heads, page, _ = codes.shape
    p, off = slots // page, slots % page
    big = x.float().abs().amax(2)                    # [tokens, heads]
    amax = torch.zeros(pages, heads, device=x.device).index_reduce_(0, p, big, "amax")
    first = torch.full((pages,), page, device=x.device).index_reduce_(0, p, off, "amin")
    m, e = torch.frexp(amax)                         # amax = m 2^e: the least e' with amax <= 448 2^e'
    fit = (e - 9 + (m > 0.875)).clamp(LOW, HIGH)
    fit = torch.where(amax > 0, fit, LOW)
    held = exps.int() - 127
    touched = (first < page)[:, None]
    fresh = (first == 0)[:, None]
    now = torch.where(touched, torch.where(fresh, fit, torch.maximum(fit, held)), held)
    older = torch.arange(page, device=x.device)[None, None, :, None] < torch.where(first < page, first, 0)[:, None, None, None]
    value = codes.view(torch.float8_e4m3fn).float()
    moved = (value * torch.exp2((held - now).float())[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes.copy_(torch.where(older, moved, codes))
    exps.copy_((now + 127).to(torch.uint8))
    codes[p, :, off] = (x.float() * torch.exp2(-now[p].float())[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_append(s):
    _plain_append_one(s["k"], s["slots"], s["k_cache"], s["k_exp"])
    _plain_append_one(s["v"], s["slots"], s["v_cache"], s["v_exp"])
    return _cache_values(s)


def _plain_norm(s):
    def normed(x, w):
        return x * torch.rsqrt((x * x).mean(1, keepdim=True) + s["eps"]) * w.float()

    y = normed(s["y"].float(), s["w_post"])
    if s["gate_t"] is not None:
        y = y * s["gate_t"].float()
    h = s["res_scale"] * s["res"].float() + y
    s["res_out"].copy_(h)
    n = normed(h, s["w_pre"])
    if s["n"] is not None:
        s["n"].copy_(n)
    if s["q"] is not None:
        rows, width = n.shape
        groups = s["scales"].shape[1]
        full = torch.nn.functional.pad(n, (0, groups * 128 - width)).view(rows, groups, 128)
        scale = full.abs().amax(2).clamp(min=1e-10) / 448.0
        s["scales"].copy_(scale)
        codes = (full / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["q"].copy_(codes.view(torch.uint8).view(rows, groups * 128)[:, :width])
    return _norm_values(s)


def _plain_attn(s):
    page, heads, kv_heads, new = s["page"], s["heads"], s["kv_heads"], s["new"]
    group, q_max, nb, dev = heads // kv_heads, max(new), _pages(max(s["lengths"]), page), s["q"].device
    batch, length = len(new), nb * page
    pages = s["table"][:, :nb].long().clamp(0, s["k_cache"].shape[0] - 1)
    kv_len, q_off = s["kv_len"].long(), s["q_offsets"].long()
    q_len = q_off[1:] - q_off[:-1]
    at = torch.arange(length, device=dev)
    held = (at[None] < kv_len[:, None])[:, None, :, None]

    def values(codes, exps):                         # [batch, kv heads, length, D], zero where nothing was written
        x = codes[pages].view(torch.float8_e4m3fn).float() * torch.exp2(exps[pages].float() - 127.0)[..., None, None]
        x = x.transpose(1, 2).reshape(batch, kv_heads, length, D)
        return torch.where(held, x, 0.0)

    i = torch.arange(q_max, device=dev)
    real = i[None] < q_len[:, None]
    rows = (q_off[:-1, None] + i[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][rows].float().view(batch, q_max, kv_heads, group, D).permute(0, 2, 1, 3, 4)
    z = torch.matmul(q.reshape(batch, kv_heads, q_max * group, D), values(s["k_cache"], s["k_exp"]).transpose(2, 3))
    z = z.view(batch, kv_heads, q_max, group, length).mul_(s["scale"])
    pos = (kv_len - q_len)[:, None] + i[None]        # a query's place in its request
    seen = (at[None, None] <= pos[..., None]) & (at[None, None] < kv_len[:, None, None])
    if s["window"] >= 0:
        seen &= at[None, None] >= pos[..., None] - s["window"]
    z.masked_fill_(~seen[:, None, :, None], float("-inf"))
    top = z.amax(4, keepdim=True)
    top = torch.where(top == float("-inf"), 0.0, top)
    z.sub_(top).exp_()
    total = z.sum(4, keepdim=True)
    o = torch.matmul(z.view(batch, kv_heads, q_max * group, length), values(s["v_cache"], s["v_exp"]))
    o = o.view(batch, kv_heads, q_max, group, D) / torch.where(total > 0, total, 1.0)
    lse = (torch.log(total) + top)[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(batch, q_max, heads, D)
    lse = lse.permute(0, 2, 1, 3).reshape(batch, q_max, heads)
    # a padded row goes nowhere: each output row is fetched from its place
    t = torch.arange(s["q"].shape[0], device=dev)
    b = torch.searchsorted(q_off[1:].contiguous(), t, right=True)
    s["out"].copy_(o[b, t - q_off[b]])
    s["lse"].copy_(lse[b, t - q_off[b]])
    return dict(out=s["out"], lse=s["lse"])


def run(state):
    op = state["op"]
    if own:
        from block_scaled_fp8_token_gb300 import bfp8
        return {"plan": _own_plan, "append": _own_append, "norm": _own_norm, "attn": _own_attn}[op](state, bfp8)
    return {"plan": _plain_plan, "append": _plain_append, "norm": _plain_norm, "attn": _plain_attn}[op](state)


# ---- what a pass cannot do without -----------------------------------------------


def work(case):
    op = case["op"]
    if op == "norm":
        rows, width = case["rows"], case["width"]
        n = rows * width
        weights = 2 * width * (2 if case["weights"] == "bf16" else 4)
        gate = {"none": 0, "channel": 2 * width, "token": 2 * n}[case["gate"]]
        codes = n + 4 * rows * _pages(width, 128) if case["out"] != "bf16" else 0
        return {"bytes": 6 * n + weights + gate + codes + (2 * n if case["out"] != "codes" else 0), "flops": 12 * n}
    ctx, new = _lengths(case)
    page, batch, tokens = case["page"], case["batch"], sum(new)
    if op == "plan":
        fresh = sum(_pages(c + n, page) - _pages(c, page) for c, n in zip(ctx, new))
        padded = max(1, _pages(tokens, 64) * 64)
        held = sum(n > 0 and c % page > 0 for c, n in zip(ctx, new))     # tables entries read: pages continued
        return {"bytes": 8 * batch + 8 * fresh + 4 * held + 12 * padded + 8 * batch + 16, "flops": 0}
    heads = case["kv_heads"]
    if op == "append":
        touched = sum(_pages(c + n, page) - c // page for c, n in zip(ctx, new) if n)
        return {"bytes": 2 * tokens * heads * D * 3 + 8 * tokens + 4 * touched * heads, "flops": 6 * tokens * heads * D}
    pairs = kept = 0
    for c, n in zip(ctx, new):
        w = case["window"]
        pairs += sum(min(c + i, w if w >= 0 else c + i) + 1 for i in range(n))
        kept += min(c + n, n + w) if w >= 0 else c + n
    group_rows = tokens * case["heads"]
    return {"bytes": 2 * kept * heads * D + 2 * _pages(kept, page) * heads + group_rows * (4 * D + 4)
            + 4 * _pages(kept, page) + 8 * batch, "flops": 4 * D * case["heads"] * pairs}


# ---- the definitions in 64 bits ---------------------------------------------------


def _e4m3_table():
    """The value of each E4M3 code."""
    t = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        t[c] = (-v if c & 128 else v) if (c & 127) != 127 else np.nan
    return t


def _encode(x):
    """Values to the nearest E4M3 values, ties to the even code, saturating: as float64 values."""
    a = np.minimum(np.abs(x), 448.0)
    _, e = np.frexp(a)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)      # eight steps to a power of two, the last ones below 2^-6
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def _exact_norm(s):
    wide = {k: s[k].double().cpu().numpy() for k in ("y", "res", "w_post", "w_pre")}
    y = wide["y"] / np.sqrt(np.mean(wide["y"] ** 2, axis=1, keepdims=True) + s["eps"]) * wide["w_post"]
    if s["gate_t"] is not None:
        y = y * s["gate_t"].double().cpu().numpy()
    h = s["res_scale"] * wide["res"] + y
    n = h / np.sqrt(np.mean(h ** 2, axis=1, keepdims=True) + s["eps"]) * wide["w_pre"]
    r = dict(residual=h)
    if s["q"] is not None:
        edges = np.arange(0, n.shape[1], 128)
        scale = np.maximum(np.maximum.reduceat(np.abs(n), edges, axis=1), 1e-10) / 448.0
        r |= dict(codes=_encode(n / np.repeat(scale, 128, axis=1)[:, :n.shape[1]]), scales=scale)
    if s["n"] is not None:
        r["normed"] = n
    return r


def _exact_append_one(x, slots, codes, exps):
    table, page = _e4m3_table(), codes.shape[2]
    value, exps = table[codes.cpu().numpy()], exps.cpu().numpy().astype(np.int64) - 127
    x, slots = x.double().cpu().numpy(), slots.cpu().numpy()
    by_page = {}
    for t, slot in enumerate(slots.tolist()):
        by_page.setdefault(slot // page, []).append((slot % page, t))
    for p, rows in by_page.items():
        off, t = (np.array(c) for c in zip(*rows))
        amax = np.abs(x[t]).max(axis=(0, 2))
        fit = np.full(amax.shape, LOW)
        some = amax > 0
        fit[some] = np.clip(np.ceil(np.log2(amax[some] / 448.0)), LOW, HIGH)
        if off.min() > 0:
            fit = np.maximum(fit, exps[p])
            value[p, :, :off.min()] = _encode(value[p, :, :off.min()] * np.exp2(1.0 * exps[p] - fit)[:, None, None])
        exps[p] = fit
        value[p][:, off] = _encode(x[t] * np.exp2(-1.0 * fit)[None, :, None]).transpose(1, 0, 2)
    return value, exps + 127


def _exact_append(s):
    k, ke = _exact_append_one(s["k"], s["slots"], s["k_cache"], s["k_exp"])
    v, ve = _exact_append_one(s["v"], s["slots"], s["v_cache"], s["v_exp"])
    return dict(k=k, v=v, k_exp=ke, v_exp=ve)


def _exact_attn(s):
    table = torch.tensor(_e4m3_table(), device="cuda")
    heads, kv_heads = s["heads"], s["kv_heads"]
    group = heads // kv_heads
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device="cuda")
    t0 = 0
    for b, (n, length) in enumerate(zip(s["new"], s["lengths"])):
        pages = s["table"][b, :_pages(length, s["page"])].long()
        scale = {x: torch.pow(2.0, s[x][pages].double() - 127.0) for x in ("k_exp", "v_exp")}
        for h in range(kv_heads):
            k = (table[s["k_cache"][pages, h].long()] * scale["k_exp"][:, h, None, None]).reshape(-1, D)[:length]
            v = (table[s["v_cache"][pages, h].long()] * scale["v_exp"][:, h, None, None]).reshape(-1, D)[:length]
            for r0 in range(0, n, 512):
                r1 = min(n, r0 + 512)
                rows, mine = slice(t0 + r0, t0 + r1), slice(h * group, (h + 1) * group)
                pos = length - n + torch.arange(r0, r1, device="cuda")
                hi = length - n + r1
                lo = max(0, length - n + r0 - s["window"]) if s["window"] >= 0 else 0
                z = torch.einsum("tgd,ld->tgl", s["q"][rows, mine].double(), k[lo:hi]) * s["scale"]
                at = torch.arange(lo, hi, device="cuda")
                hidden = at[None] > pos[:, None]
                if s["window"] >= 0:
                    hidden |= at[None] < pos[:, None] - s["window"]
                z = z.masked_fill(hidden[:, None], -math.inf)
                lse[rows, mine] = torch.logsumexp(z, 2)
                out[rows, mine] = torch.einsum("tgl,ld->tgd", torch.softmax(z, 2), v[lo:hi])
        t0 += n
    return dict(out=out, lse=lse)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    state = prepare(case, seed)
    return {"append": _exact_append, "norm": _exact_norm, "attn": _exact_attn}[case["op"]](state)
