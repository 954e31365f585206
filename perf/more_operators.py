"""Cases, inputs and plain forms of a hybrid decoder's operators: the gated delta rule with the short causal
convolution ahead of it and the gated norm behind it (linear-attention layers), and rotary positions of one or
several axes with the heads' norms (full-attention layers).

    listed()             the named cases;  draw(rng)  one more of the same ranges
    prepare(case, seed)  inputs on the GPU
    run(state)           one pass: the plain forms, or the library's calls where ``own`` is true
    work(case)           compulsory bytes and operations of one pass
    exact(case, seed)    the definitions in 64 bits

Tokens of a step's requests lie one behind another, ``offsets`` apart. What a request keeps between steps is in a
slot of a pool: the last inputs of the convolution, and for each value head the state [128 values, 128 keys]. Every
pass reads the states from the slots of ``slots_in`` and leaves the new ones in those of ``slots_out``, as a
program does that keeps a step's states until its drafted tokens are accepted; -1 begins from nothing.
"""

from __future__ import annotations

import math
import random

import torch

own = False

D = 128          # width of a head of the delta rule
CHUNK = 64       # tokens that the plain delta rule takes at a time


def listed():
    return [
        # the convolution of a full batch's decode step, queries, keys and values of 16 + 16 + 32 heads: latency
        dict(name="conv_step", op="conv", lens=1, batch=64, q_lo=1, q_hi=1, fresh=0.0, channels=8192, width=4, bias=False),
        # ragged prompts, some of them continued
        dict(name="conv_prompts", op="conv", lens=2, batch=8, q_lo=64, q_hi=4096, fresh=0.5, channels=8192, width=4,
             bias=False),
        # one user's next token: the smallest call
        dict(name="delta_one", op="delta", lens=3, batch=1, q_lo=1, q_hi=1, fresh=0.0, qk_heads=16, v_heads=32),
        # a serving batch's decode step: the states' traffic
        dict(name="delta_step", op="delta", lens=4, batch=64, q_lo=1, q_hi=1, fresh=0.0, qk_heads=16, v_heads=48),
        # three drafted tokens of each request verified at once
        dict(name="delta_draft", op="delta", lens=5, batch=17, q_lo=3, q_hi=3, fresh=0.0, qk_heads=16, v_heads=32),
        # one long prompt: a chain of chunks with little beside it
        dict(name="delta_prompt", op="delta", lens=6, batch=1, q_lo=8192, q_hi=8192, fresh=1.0, qk_heads=16, v_heads=32),
        # prompts, continued chunks and single tokens in one step
        dict(name="delta_mixed", op="delta", lens=7, batch=12, q_lo=1, q_hi=2000, fresh=0.4, qk_heads=16, v_heads=48),
        # behind the delta rule of a decode step, codes for the FP8 output projection
        dict(name="gated_step", op="gated", rows=64, heads=48, dim=128, out="codes"),
        # the same for a long prompt
        dict(name="gated_prompt", op="gated", rows=8192, heads=48, dim=128, out="codes"),
        # the queries and keys of a decode step of text, 64 heads on 8
        dict(name="rotary_step", op="rotary", tokens=64, heads=64, kv_heads=8, dim=128, rotary=128, axes=1, inter=False,
             adjacent=False, norm=False, far=131072),
        # a prompt of text and images: three axes taking turns over a quarter of each head, heads normed first
        dict(name="rotary_images", op="rotary", tokens=8192, heads=16, kv_heads=2, dim=256, rotary=64, axes=3, inter=True,
             adjacent=False, norm=True, far=32768),
        # an odd number of tokens, three axes in sections of the whole head, as image towers and older models have them
        dict(name="rotary_odd", op="rotary", tokens=949, heads=64, kv_heads=8, dim=128, rotary=128, axes=3, inter=False,
             adjacent=True, norm=False, far=1000000),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["conv", "delta", "delta", "delta", "gated", "rotary"])
    if op == "gated":
        return dict(op=op, rows=_log(rng, 1, 6000), heads=rng.choice([1, 2, 5, 16, 32, 40]), dim=rng.choice([64, 128, 128, 256]),
                    out=rng.choice(["codes", "both", "bf16"]))
    if op == "rotary":
        dim = rng.choice([64, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 8000), heads=rng.choice([1, 2, 5, 16, 32]), kv_heads=rng.choice([1, 2, 5]), dim=dim,
                    rotary=rng.choice([dim, dim // 2, 16 * rng.randint(2, dim // 16)]), axes=rng.choice([1, 2, 3, 4]),
                    inter=rng.random() < 0.5, adjacent=rng.random() < 0.5, norm=rng.random() < 0.5, far=_log(rng, 10, 4000000))
    case = dict(op=op, lens=rng.randrange(1 << 30), fresh=rng.choice([0.0, 0.3, 1.0]))
    if rng.random() < 0.4:                           # a decode step, a few drafted tokens in some
        q = rng.choice([1, 1, 2, 4, 7])
        case |= dict(batch=_log(rng, 1, 64), q_lo=q, q_hi=q)
    else:
        batch = _log(rng, 1, 10)
        hi = _log(rng, 8, 8192 // batch)
        case |= dict(batch=batch, q_lo=max(1, hi // rng.choice([1, 3, 10, 100])), q_hi=hi)
    if op == "conv":
        return dict(case, channels=8 * _log(rng, 8, 1000), width=rng.choice([2, 3, 4, 4]), bias=rng.random() < 0.5)
    qk = rng.choice([1, 2, 5, 16])
    return dict(case, qk_heads=qk, v_heads=qk * rng.choice([1, 2, 2, 3 if qk > 2 else 4]))


def _lengths(case):
    """New tokens of each request, and which requests begin: the case's own, whatever the seed."""
    rng = random.Random(case["lens"])
    new = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    return new, [rng.random() < case["fresh"] for _ in range(case["batch"])]


# ---- inputs ----------------------------------------------------------------


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _requests(case, g):
    """Offsets and slots of the step's requests; the pool has two slots a request and one to spare, in no order."""
    new, begins = _lengths(case)
    n = len(new)
    slots = torch.randperm(2 * n + 1, generator=g, device="cuda").to(torch.int32)
    held = torch.tensor([not b for b in begins], device="cuda")
    return dict(new=new, n_slots=2 * n + 1, offsets=_i32([sum(new[:b]) for b in range(n + 1)]),
                slots_in=torch.where(held, slots[:n], -1), slots_out=slots[n:2 * n].contiguous())


def _prepare_conv(case, g):
    s = dict(case, **_requests(case, g))
    C, W, T = case["channels"], case["width"], sum(s["new"])

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    return dict(s, x=randn(T, C), weight=(randn(C, W).float() / math.sqrt(W)).to(torch.bfloat16),
                bias_t=randn(C) if case["bias"] else None, state=randn(s["n_slots"], W - 1, C),
                out=torch.empty(T, C, dtype=torch.bfloat16, device="cuda"))


def _prepare_delta(case, g):
    s = dict(case, **_requests(case, g))
    hk, hv, T = case["qk_heads"], case["v_heads"], sum(s["new"])

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # queries, keys and values as the convolution's SiLU leaves them, the columns of one matrix
    qkv = torch.nn.functional.silu(1.5 * randn(T, 2 * hk + hv, D)).to(torch.bfloat16)
    ab = randn(T, 2, hv).to(torch.bfloat16)
    # heads that forget within a few tokens next to heads that keep thousands
    rate = torch.exp(math.log(1e-3) + math.log(1e2) * torch.rand(hv, generator=g, device="cuda"))
    s |= dict(q=qkv[:, :hk], k=qkv[:, hk:2 * hk], v=qkv[:, 2 * hk:], a=ab[:, 0], b=ab[:, 1],
              a_log=torch.log(1 + 15 * torch.rand(hv, generator=g, device="cuda")), dt_bias=rate + torch.log(-torch.expm1(-rate)),
              state=0.3 * randn(s["n_slots"], hv, D, D), scale=D ** -0.5, eps=1e-6,
              out=torch.empty(T, hv, D, dtype=torch.bfloat16, device="cuda"))
    if own:                                          # the scratch that a serving program keeps
        from block_scaled_fp8_token_gb300 import bfp8
        s["ws"] = torch.empty(bfp8.bfp8_delta_rule_workspace(len(s["new"]), T, max(s["new"]), hk, hv), dtype=torch.uint8,
                              device="cuda")
    return s


def _prepare_gated(case, g):
    rows, heads, dim = case["rows"], case["heads"], case["dim"]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = dict(case, x=(0.2 * randn(rows, heads, dim)).to(torch.bfloat16), gate=(1.5 * randn(rows, heads, dim)).to(torch.bfloat16),
             weight=1 + 0.2 * randn(dim), eps=1e-6, y=None, codes=None, scales=None)
    if case["out"] != "codes":
        s["y"] = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda")
    if case["out"] != "bf16":
        s["codes"] = torch.empty(rows, heads * dim, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(rows, -(-heads * dim // 128), dtype=torch.float32, device="cuda")
    return s


def _sections(case):
    """How many pairs turn with each axis."""
    pairs, axes = case["rotary"] // 2, case["axes"]
    return [pairs - (axes - 1) * (pairs // (axes + 1))] + (axes - 1) * [pairs // (axes + 1)]


def _prepare_rotary(case, g):
    T, heads, kv, dim, r = (case[k] for k in ("tokens", "heads", "kv_heads", "dim", "rotary"))

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # runs of text, where all axes count on together, and pictures, where the last two run over rows and columns
    t = torch.arange(T, device="cuda")
    start = int(torch.randint(0, case["far"], (1,), generator=g, device="cuda"))
    axes = [start + t]
    if case["axes"] > 1:
        side = 24
        block, at = t // (2 * side * side), t % (2 * side * side)
        base, pic = start + block * (side * side + side), at >= side * side
        at = torch.where(pic, at - side * side, at)
        text = base + at
        rows, cols = base + side * side + at // side, base + side * side + at % side
        turns = [torch.where(pic, base + side * side, text), torch.where(pic, rows, text), torch.where(pic, cols, text)]
        axes = (turns + [text])[:case["axes"]]
    qkv = randn(T, heads + 2 * kv, dim).to(torch.bfloat16)
    inv_freq = (5e5 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()
    weights = [(1 + 0.2 * randn(dim)).to(torch.bfloat16) for _ in range(2)]
    return dict(case, q=qkv[:, :heads], k=qkv[:, heads:heads + kv], positions=torch.stack(axes).to(torch.int32).contiguous(),
                inv_freq=inv_freq, q_weight=weights[0] if case["norm"] else None, k_weight=weights[1] if case["norm"] else None,
                eps=1e-6, sections=_sections(case), q_out=torch.empty(T, heads, dim, dtype=torch.bfloat16, device="cuda"),
                k_out=torch.empty(T, kv, dim, dtype=torch.bfloat16, device="cuda"))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return {"conv": _prepare_conv, "delta": _prepare_delta, "gated": _prepare_gated, "rotary": _prepare_rotary}[case["op"]](case, g)


# ---- the library's calls -----------------------------------------------------


def _own_conv(s, lib):
    lib.bfp8_causal_conv(s["x"], s["weight"], s["out"], s["offsets"], s["state"], s["slots_in"], s["slots_out"],
                         bias=s["bias_t"], silu=True)
    return dict(out=s["out"], state=s["state"])


def _own_delta(s, lib):
    lib.bfp8_delta_rule(s["q"], s["k"], s["v"], s["a"], s["b"], s["a_log"], s["dt_bias"], s["state"], s["slots_in"],
                        s["slots_out"], s["offsets"], s["out"], max(s["new"]), scale=s["scale"], eps=s["eps"],
                        workspace=s["ws"])
    return dict(out=s["out"], state=s["state"])


def _gated_values(s):
    r = {} if s["y"] is None else dict(y=s["y"])
    return r if s["codes"] is None else dict(r, codes=s["codes"].view(torch.float8_e4m3fn), scales=s["scales"])


def _own_gated(s, lib):
    lib.bfp8_gated_norm(s["x"], s["gate"], s["weight"], s["y"], q=s["codes"], scales=s["scales"], eps=s["eps"])
    return _gated_values(s)


def _own_rotary(s, lib):
    lib.bfp8_rotary(s["q"], s["k"], s["positions"], s["inv_freq"], s["q_out"], s["k_out"], sections=s["sections"],
                    interleaved=s["inter"], adjacent=s["adjacent"], q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"])
    return dict(q=s["q_out"], k=s["k_out"])


# ---- the plain forms -----------------------------------------------------------


def _padded_rows(s, chunk):
    """Each request's tokens as rows of one length, a multiple of `chunk`: [batch, length] indices, and which are real."""
    length = -(-max(s["new"]) // chunk) * chunk
    at = torch.arange(length, device="cuda")
    off = s["offsets"].long()
    real = at[None] < (off[1:] - off[:-1])[:, None]
    return (off[:-1, None] + at[None]).clamp(max=int(sum(s["new"])) - 1), real


def _unpadded(s):
    """For each token its request and its place in it."""
    off = s["offsets"].long()
    t = torch.arange(sum(s["new"]), device="cuda")
    b = torch.searchsorted(off[1:].contiguous(), t, right=True)
    return b, t - off[b]


def _state_in(s):
    at = s["slots_in"].long()
    held = (at >= 0).view(-1, *(1,) * (s["state"].dim() - 1))
    return torch.where(held, s["state"][at.clamp(min=0)], torch.zeros((), dtype=s["state"].dtype, device="cuda"))


def _silu(x):
    return x / (1 + torch.exp(-x))


def _plain_conv(s):
    W, x, first = s["width"], s["x"].float(), _state_in(s).float()
    b, i = _unpadded(s)
    off, w = s["offsets"].long(), s["weight"].float()

    def before(n, b, i):                             # the input n places ahead of place i of request b
        return torch.where((i >= n)[:, None], x[(off[b] + i - n).clamp(0, x.shape[0] - 1)], first[b, (W - 1 + i - n).clamp(0, W - 2)])

    y = sum(w[:, W - 1 - n] * before(n, b, i) for n in range(W))
    if s["bias_t"] is not None:
        y = y + s["bias_t"].float()
    s["out"].copy_(_silu(y))
    every, ends = torch.arange(len(s["new"]), device="cuda"), off[1:] - off[:-1]
    last = torch.stack([before(n, every, ends - 1) for n in range(W - 2, -1, -1)], 1)
    s["state"][s["slots_out"].long()] = last.to(torch.bfloat16)
    return dict(out=s["out"], state=s["state"])


def _plain_delta(s):
    hk, hv, chunk = s["qk_heads"], s["v_heads"], min(CHUNK, max(s["new"]))
    rows, real = _padded_rows(s, chunk)
    B, L = rows.shape
    n = L // chunk

    def heads(x):                                    # [batch, value heads, chunks, chunk, ...] of [tokens, heads, ...]
        y = torch.where(real.view(B, L, *(1,) * (x.dim() - 1)), x[rows].float(), 0.0).movedim(2, 1)
        return y.reshape(B, x.shape[1], n, chunk, *x.shape[2:]).repeat_interleave(hv // x.shape[1], 1)

    def unit(x):
        return x * torch.rsqrt((x * x).sum(-1, keepdim=True) + s["eps"])

    q, k, v = unit(heads(s["q"])) * s["scale"], unit(heads(s["k"])), heads(s["v"])
    z = s["a"].float() + s["dt_bias"]
    g = heads(-torch.exp(s["a_log"]) * torch.where(z > 20, z, torch.log1p(torch.exp(z.clamp(max=20)))))
    beta = heads(1 / (1 + torch.exp(-s["b"].float())))
    total = torch.cumsum(g, -1)
    i = torch.arange(chunk, device="cuda")
    within = (total[..., :, None] - total[..., None, :]).masked_fill(i[:, None] < i[None], -math.inf).exp()
    lower = (beta[..., None] * within * (k @ k.transpose(-1, -2))).masked_fill(i[:, None] <= i[None], 0.0)
    inverse = torch.eye(chunk, device="cuda").expand_as(lower).clone()
    for r in range(1, chunk):                        # the rows of (1 + lower)^-1, one from those above it
        inverse[..., r, :r] = -(lower[..., r, None, :r] @ inverse[..., :r, :r])[..., 0, :]
    u0, w = inverse @ (beta[..., None] * v), inverse @ ((beta * total.exp())[..., None] * k)
    mix, q = within * (q @ k.transpose(-1, -2)), total.exp()[..., None] * q
    k = k * (total[..., -1:] - total).exp()[..., None]
    state = _state_in(s).transpose(-1, -2)
    out = torch.empty_like(v)
    for c in range(n):                               # each chunk needs the state that the one before it leaves
        u = u0[:, :, c] - w[:, :, c] @ state
        out[:, :, c] = q[:, :, c] @ state + mix[:, :, c] @ u
        state = total[:, :, c, -1, None, None].exp() * state + k[:, :, c].transpose(-1, -2) @ u
    s["state"][s["slots_out"].long()] = state.transpose(-1, -2)
    b, at = _unpadded(s)
    s["out"].copy_(out.view(B, hv, L, D)[b, :, at])
    return dict(out=s["out"], state=s["state"])


def _plain_gated(s):
    x, rows = s["x"].float(), s["rows"]
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["weight"] * _silu(s["gate"].float())
    if s["y"] is not None:
        s["y"].copy_(y)
    if s["codes"] is not None:
        width, groups = s["codes"].shape[1], s["scales"].shape[1]
        full = torch.nn.functional.pad(y.view(rows, width), (0, groups * 128 - width)).view(rows, groups, 128)
        scale = full.abs().amax(2).clamp(min=1e-10) / 448.0
        s["scales"].copy_(scale)
        codes = (full / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        s["codes"].copy_(codes.view(torch.uint8).view(rows, groups * 128)[:, :width])
    return _gated_values(s)


def _axis_of_pair(s):
    """The axis that each pair turns with: sections one behind another, or the axes in turn while their sections last
    and the first axis for the rest."""
    pairs, axes, sections = s["rotary"] // 2, s["axes"], torch.tensor(s["sections"], device="cuda")
    i = torch.arange(pairs, device="cuda")
    if s["inter"]:
        return torch.where(i // axes < sections[i % axes], i % axes, 0)
    return torch.searchsorted(torch.cumsum(sections, 0), i, right=True)


def _plain_rotary(s):
    r = s["rotary"]
    angle = s["positions"].double()[_axis_of_pair(s)].T * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight, out):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * weight.float()
        a, b = (x[..., 0:r:2], x[..., 1:r:2]) if s["adjacent"] else (x[..., :r // 2], x[..., r // 2:r])
        pair = a * cos - b * sin, b * cos + a * sin
        y = torch.stack(pair, -1).flatten(-2) if s["adjacent"] else torch.cat(pair, -1)
        out.copy_(torch.cat([y, x[..., r:]], -1))

    turned(s["q"], s["q_weight"], s["q_out"])
    turned(s["k"], s["k_weight"], s["k_out"])
    return dict(q=s["q_out"], k=s["k_out"])


def run(state):
    op = state["op"]
    if own:
        from block_scaled_fp8_token_gb300 import bfp8
        return {"conv": _own_conv, "delta": _own_delta, "gated": _own_gated, "rotary": _own_rotary}[op](state, bfp8)
    return {"conv": _plain_conv, "delta": _plain_delta, "gated": _plain_gated, "rotary": _plain_rotary}[op](state)


# ---- what a pass cannot do without -----------------------------------------------


def work(case):
    op = case["op"]
    if op == "gated":
        n = case["rows"] * case["heads"] * case["dim"]
        codes = n + 4 * case["rows"] * -(-case["heads"] * case["dim"] // 128) if case["out"] != "bf16" else 0
        return {"bytes": 4 * n + 4 * case["dim"] + codes + (2 * n if case["out"] != "codes" else 0), "flops": 10 * n}
    if op == "rotary":
        n = case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * n + 4 * case["axes"] * case["tokens"] + 2 * case["rotary"] + (4 * case["dim"] if case["norm"] else 0),
                "flops": 3 * n * case["rotary"] // case["dim"] + (4 * n if case["norm"] else 0)}
    new, begins = _lengths(case)
    tokens, held, batch = sum(new), begins.count(False), len(new)
    if op == "conv":
        C, W = case["channels"], case["width"]
        return {"bytes": 4 * tokens * C + 2 * C * (W + case["bias"]) + 2 * (W - 1) * C * (held + batch) + 12 * batch,
                "flops": (2 * W + 4) * tokens * C}
    hk, hv = case["qk_heads"], case["v_heads"]
    # of a chain of single tokens the recurrence's operations; of longer requests a chunk's products, a head and token:
    # the state met by key and query and its update, the chunk's keys and queries among themselves, and their use
    flops = sum(hv * n * (7 * D * D if n < 32 else 6 * D * D + 4 * CHUNK * D + 4 * D * min(n, CHUNK)) for n in new)
    return {"bytes": tokens * (4 * hk * D + 4 * hv * D + 4 * hv) + 4 * hv * D * D * (held + batch) + 8 * hv + 12 * batch,
            "flops": flops}


# ---- the definitions in 64 bits ---------------------------------------------------


def _exact_conv(s):
    W, C = s["width"], s["channels"]
    state, out, t0 = s["state"].double(), [], 0
    for n, src, dst in zip(s["new"], s["slots_in"].tolist(), s["slots_out"].tolist()):
        past = s["state"][src].double() if src >= 0 else torch.zeros(W - 1, C, dtype=torch.float64, device="cuda")
        x = torch.cat([past, s["x"][t0:t0 + n].double()])
        y = (x.unfold(0, W, 1) * s["weight"].double()).sum(-1)
        if s["bias_t"] is not None:
            y += s["bias_t"].double()
        out.append(y * torch.sigmoid(y))
        state[dst] = x[n:]
        t0 += n
    return dict(out=torch.cat(out), state=state)


def _exact_delta(s):
    hv, group = s["v_heads"], s["v_heads"] // s["qk_heads"]

    def wide(x, normed):
        x = x.double()
        if normed:
            x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) + s["eps"])
        return torch.repeat_interleave(x, hv // x.shape[1], 1)

    q, k, v = wide(s["q"], True) * s["scale"], wide(s["k"], True), wide(s["v"], False)
    keep = torch.exp(-torch.exp(s["a_log"].double()) * torch.nn.functional.softplus(s["a"].double() + s["dt_bias"].double(), threshold=50))
    beta = torch.sigmoid(s["b"].double())
    off, pool = s["offsets"].long(), s["state"].double()
    every = _state_in(s).double()
    out = torch.empty_like(v)
    order = sorted(range(len(s["new"])), key=lambda b: -s["new"][b])   # the longest first: those left at t are a prefix
    S, first = every[order], off[torch.tensor(order, device="cuda")]
    for t in range(max(s["new"])):
        live = sum(n > t for n in s["new"])
        at = first[:live] + t
        S[:live] *= keep[at][..., None, None]
        kt = k[at]
        u = beta[at][..., None] * (v[at] - torch.einsum("bhvk,bhk->bhv", S[:live], kt))
        S[:live] += u[..., None] * kt[..., None, :]
        out[at] = torch.einsum("bhvk,bhk->bhv", S[:live], q[at])
    pool[s["slots_out"].long()[order]] = S
    return dict(out=out, state=pool)


def _nearest_e4m3(x):
    """The nearest E4M3 values, ties to even, saturating."""
    a = x.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    return torch.copysign((torch.round(a / step) * step).clamp(max=448.0), x)


def _exact_gated(s):
    x, z, rows = s["x"].double(), s["gate"].double(), s["rows"]
    y = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + s["eps"]) * s["weight"].double() * (z * torch.sigmoid(z))
    r = {} if s["y"] is None else dict(y=y)
    if s["codes"] is not None:
        flat = y.reshape(rows, -1)
        scale = torch.stack([p.abs().amax(1).clamp(min=1e-10) / 448.0 for p in flat.split(128, 1)], 1)
        r |= dict(codes=_nearest_e4m3(flat / torch.repeat_interleave(scale, 128, 1)[:, :flat.shape[1]]), scales=scale)
    return r


def _exact_rotary(s):
    r, half, pos = s["rotary"], s["rotary"] // 2, s["positions"].double()
    axis = [0] * half
    if s["inter"]:
        for a in range(1, s["axes"]):
            for j in range(s["sections"][a]):
                if j * s["axes"] + a < half:
                    axis[j * s["axes"] + a] = a
    else:
        axis = [a for a, n in enumerate(s["sections"]) for _ in range(n)]
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                       torch.stack([pos[a] * s["inv_freq"][i].double() for i, a in enumerate(axis)], 1))[:, None]

    def turned(x, weight):
        x = x.double().clone()
        if weight is not None:
            x = x / torch.sqrt((x ** 2).mean(-1, keepdim=True) + s["eps"]) * weight.double()
        first, second = (slice(0, r, 2), slice(1, r, 2)) if s["adjacent"] else (slice(0, half), slice(half, r))
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    return dict(q=turned(s["q"], s["q_weight"]), k=turned(s["k"], s["k_weight"]))


def exact(case, seed):
    state = prepare(case, seed)
    return {"conv": _exact_conv, "delta": _exact_delta, "gated": _exact_gated, "rotary": _exact_rotary}[case["op"]](state)
