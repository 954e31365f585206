"""The attention layer's steps around a paged 8-bit KV cache, and the residual
norm between blocks: token by token and row by row, double precision.

Test infrastructure (CPU oracle); see the package docstring for who may use it.

The cache: E4M3 codes [pages, heads, page, D] and one scale byte per (page,
head); a value is e4m3(code) * 2^(byte - 127). A slot is page * page_size +
offset.
"""

from __future__ import annotations

import numpy as np

from .formats import e4m3_decode_lut, e4m3_encode_rne_sat, f64_to_bf16_bits

MIN_EXP, MAX_EXP = -40, 40


def block_plan(ctx, new, free, table, page, capacity):
    """One step's plan, request by request and token by token.
    Returns (table, q_offsets, kv_len, slots, positions, counts)."""
    table = np.array(table, dtype=np.int64)
    ctx, new = [max(0, int(c)) for c in ctx], [max(0, int(n)) for n in new]
    slots, positions = np.full(capacity, -1, np.int64), np.full(capacity, -1, np.int64)
    offsets, wanted, short, homeless = [0], 0, 0, 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        width = table.shape[1]
        for j in range(min(-(-c // page), width), min(-(-(c + n) // page), width) if n else 0):
            table[b, j] = free[wanted] if wanted < len(free) else -1
            short += wanted >= len(free)
            wanted += 1
        for i in range(n):
            j, t = (c + i) // page, offsets[-1] + i
            pg = table[b, j] if j < width else -1
            homeless += pg < 0
            if t < capacity:
                positions[t] = c + i
                if pg >= 0:
                    slots[t] = int(pg) * page + (c + i) % page
        offsets.append(offsets[-1] + n)
    kv_len = [c + n for c, n in zip(ctx, new)]
    return table, np.array(offsets), np.array(kv_len, np.int64), slots, positions, [wanted - short, short, homeless]


def scale_exponent(amax: float) -> int:
    """Least e in [MIN_EXP, MAX_EXP] with amax <= 448 * 2^e (MAX_EXP if none)."""
    for e in range(MIN_EXP, MAX_EXP + 1):
        if amax <= 448.0 * 2.0 ** e:
            return e
    return MAX_EXP


def append(x, slots, codes, exps):
    """x float64 [T, H, D] into codes uint8 [P, H, page, D], exps uint8 [P, H]; returns new (codes, exps)."""
    codes, exps = np.array(codes), np.array(exps)
    lut, page = e4m3_decode_lut(), codes.shape[2]
    rows = {}
    for t, s in enumerate(np.asarray(slots).tolist()):
        if 0 <= s < codes.shape[0] * page:
            rows.setdefault(s // page, []).append((s % page, t))
    for p, where in rows.items():
        first = min(where)[0]
        for h in range(codes.shape[1]):
            vals = np.abs(np.stack([x[t, h] for _, t in where]))
            vals = vals[~np.isnan(vals)]
            e = scale_exponent(float(vals.max()) if vals.size else 0.0)
            if first > 0:
                old = int(exps[p, h]) - 127
                if e > old:
                    codes[p, h, :first] = e4m3_encode_rne_sat(lut[codes[p, h, :first]] * 2.0 ** (old - e))
                e = max(e, old)
            exps[p, h] = e + 127
            for off, t in where:
                codes[p, h, off] = e4m3_encode_rne_sat(x[t, h] * 2.0 ** -e)
    return codes, exps


def dequantize(codes, exps):
    return e4m3_decode_lut()[codes] * 2.0 ** (exps.astype(np.float64) - 127)[:, :, None, None]


def attention(q, k_cache, v_cache, table, q_offsets, kv_len, scale, window=-1):
    """q float64 [T, Hq, D]; caches float64 [P, H, page, D] (dequantized; NaN where nothing was written).
    Row i of a request with n new tokens and length L sits at position L - n + i and sees the positions up to
    its own, at most `window` before it (all if window < 0), in pages that exist. A row that sees nothing gives
    0 and -inf. Returns (out [T, Hq, D], lse [T, Hq])."""
    T, Hq, D = q.shape
    P, H, page, _ = k_cache.shape
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    for b in range(len(kv_len)):
        r0, r1, L = int(q_offsets[b]), int(q_offsets[b + 1]), int(kv_len[b])
        places = np.arange(L)
        pages = np.array([table[b][i // page] for i in range(L)], np.int64).reshape(L)
        there = (pages >= 0) & (pages < P)
        for t in range(r0, r1):
            pos = L - (r1 - r0) + (t - r0)
            see = there & (places <= pos)
            if window >= 0:
                see &= places >= pos - window
            i = places[see]
            if not i.size:
                continue
            for h in range(Hq):
                g = h // (Hq // H)
                z = k_cache[pages[i], g, i % page] @ q[t, h] * scale
                m = z.max()
                p = np.exp(z - m)
                out[t, h] = (p / p.sum()) @ v_cache[pages[i], g, i % page]
                lse[t, h] = m + np.log(p.sum())
    return out, lse


def residual_norm(y, residual, w_post=None, w_pre=None, gate=None, residual_scale=1.0, eps=1e-6, offset=0.0):
    """All float64, [T, H] and [H]. Returns (h, n), unrounded."""
    h = residual_scale * residual
    if y is not None:
        u = y if w_post is None else y / np.sqrt(np.mean(y * y, axis=1, keepdims=True) + eps) * (w_post + offset)
        h = h + (u if gate is None else gate * u)
    n = None
    if w_pre is not None:
        n = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * (w_pre + offset)
    return h, n


def bf16(x):
    return (f64_to_bf16_bits(np.asarray(x, np.float64)).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
