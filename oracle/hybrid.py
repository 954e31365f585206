"""The operators of a hybrid decoder's layers, token by token in double precision:
the causal convolution, the gated delta rule and the gated norm of its
linear-attention layers, and rotary positions of several axes.

Test infrastructure (CPU oracle); see the package docstring for who may use it.
"""

from __future__ import annotations

import numpy as np


def _sigmoid(x):
    return 1 / (1 + np.exp(-x))


def causal_conv(x, weight, bias, first, silu=True):
    """One request: x [n, C], weight [C, W], first [W - 1, C] the inputs ahead of x.
    Returns (out [n, C], the last W - 1 inputs, the sums' sizes sum |w x| + |bias|)."""
    n, W = x.shape[0], weight.shape[1]
    every = np.concatenate([first, x])
    y, size = np.zeros(x.shape), np.zeros(x.shape)
    for t in range(n):
        for j in range(W):
            y[t] += weight[:, j] * every[t + j]
            size[t] += np.abs(weight[:, j] * every[t + j])
        if bias is not None:
            y[t] += bias
            size[t] += np.abs(bias)
    return (y * _sigmoid(y) if silu else y), every[n:], size


def delta_gates(a, b, a_log, dt_bias):
    """The logarithm of each token's decay, and beta; a, b [n, v heads]."""
    z = a + dt_bias
    g = -np.exp(a_log) * (np.maximum(z, 0) + np.log1p(np.exp(-np.abs(z))))
    return g, _sigmoid(b)


def delta_rule(q, k, v, a, b, a_log, dt_bias, state, scale, eps):
    """One request: q, k [n, qk heads, 128], v [n, v heads, 128], state [v heads, 128 values,
    128 keys]. Returns (out [n, v heads, 128], the new state, and two sums for error bounds):
    an error of c (1 + |g|) (alpha |S_row| + |v|) a token in a row of the state, c as small as
    one likes, grows no faster than c times `grown` [v heads, 128], because alpha (1 - beta k'
    k'^T) shortens what it multiplies; `met` [n, v heads, 128] is its value plus |S_row| at each token."""
    n, hv, D = v.shape
    group = hv // q.shape[1]
    g, beta = delta_gates(a, b, a_log, dt_bias)
    S, out = np.array(state, dtype=np.float64), np.zeros(v.shape)
    grown, met = np.zeros((hv, D)), np.zeros((n, hv, D))
    for t in range(n):
        kt = np.repeat(k[t] / np.sqrt((k[t] ** 2).sum(-1, keepdims=True) + eps), group, 0)
        qt = np.repeat(q[t] / np.sqrt((q[t] ** 2).sum(-1, keepdims=True) + eps) * scale, group, 0)
        alpha = np.exp(g[t])[:, None]
        grown = alpha * grown + (1 + np.abs(g[t])[:, None]) * (alpha * np.linalg.norm(S, axis=2) + np.abs(v[t]))
        S *= alpha[..., None]
        u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", S, kt))
        S += u[:, :, None] * kt[:, None, :]
        out[t] = np.einsum("hvk,hk->hv", S, qt)
        met[t] = grown + np.linalg.norm(S, axis=2)
    return out, S, grown, met


def gated_norm(x, gate, weight, eps, offset=0.0, sigmoid=False):
    """x, gate [T, H, D]; weight [D] or None."""
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (weight + offset)
    act = _sigmoid(gate)
    return x * (act if sigmoid else gate * act)


def axis_of_pair(half, sections, interleaved):
    if not interleaved:
        return [n for n, s in enumerate(sections) for _ in range(s)]
    axes = len(sections)
    return [i % axes if i // axes < sections[i % axes] else 0 for i in range(half)]


def rotary(x, positions, inv_freq, sections, interleaved=False, adjacent=False, weight=None, eps=1e-6, offset=0.0,
           factor=1.0):
    """x [T, H, D], positions int [axes, T], inv_freq float32 [half]. A token with a
    negative position keeps NaN. Returns (y, the size |a| + |b| of each column's pair)."""
    T, H, D = x.shape
    half = len(inv_freq)
    x = np.array(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (weight + offset)
    y, size = x.copy(), np.abs(x)
    axis = axis_of_pair(half, sections, interleaved)
    for i in range(half):
        # a position below 2^31 times a float32 has 55 bits: float64 rounds it by 2^-54 relative,
        # under 2^-20 of a radian at the far end with inv_freq 1, so the product is split in two
        f = float(np.float32(inv_freq[i]))
        lo = positions[axis[i]] & 0xFFFF
        angle, more = (positions[axis[i]] - lo) * f, lo * f      # each exact (15 + 24 and 16 + 24 bits)
        c = (np.cos(angle) * np.cos(more) - np.sin(angle) * np.sin(more))[:, None]
        s = (np.sin(angle) * np.cos(more) + np.cos(angle) * np.sin(more))[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        y[..., a] = factor * (x[..., a] * c - x[..., b] * s)
        y[..., b] = factor * (x[..., b] * c + x[..., a] * s)
        size[..., a] = size[..., b] = abs(factor) * (np.abs(x[..., a]) + np.abs(x[..., b]))
    y[(positions < 0).any(0)] = np.nan
    return y, size
