"""bfp8_kv_attention against float64 within what its own arithmetic may cost, term by term.

With weights w_i (of sum 1), values v_i = code_i 2^ev_i, x_i = score_i log2(e) + ev_i and the kernel's
weights P_i = 2^(x_i - M), M the largest x less 4 or below, an element of the output may be off by
  * P's rounding to F16, 11 bits: independent errors of 2^-11 at most, a standard deviation of
    2^-11 / sqrt(3) sqrt(sum w_i^2 v_i^2); six of those;
  * P's of less than 2^-14, F16's subnormals: 2^-25 each, so 2^-25 sum |code_i| / sum P_j 2^-ev_j over them;
  * the scores' errors d_i, twice (in the weight and in the weights' sum): 2 sum w_i |v_i| d_i. With
    A_i = scale sum_d |q_d k_id|: eight products' sums of 32 terms, aligned to the largest and cut at
    FP32's last bit, are 8 * 33 * 2^-25 A_i off at most, below 2^-17 A_i; entries of q below 2^-13 of the
    row's largest are carried to 2^-21 of it; scaling, the subtraction and 2^x cost 2^-22 (1 + |score_i|);
  * the value products' FP32 sums, 17 terms a step of 16 tokens: below n 2^-23 sum w_i |v_i|;
  * the weights' sum and the division, 2^-20 of the output, and the output's rounding to BF16, 2^-8 of it.
lse is off by the largest d_i that has any weight and 2^-20 (1 + |lse|).

Weights of 8 bits, as two E4M3 terms would give them, and queries of two E4M3 terms, whose small entries
are only carried to 2^-18 of the largest, are outside of these bounds: the tests without a GPU plant both.
"""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kv as KV
from test_gpu_kv_attention import D, _run, _setup

LUT = F.e4m3_decode_lut()


def _row(q, k, code, ev, scale):
    """(out, lse, bound of out, bound of lse) of one query row [D] over k, code [n, D] and ev [n]."""
    z, v = k @ q * scale, code * 2.0 ** ev[:, None]
    x = z * np.log2(np.e) + ev
    w = np.exp(z - z.max())
    total = w.sum()
    w /= total
    P = 2.0 ** (x - x.max() + 4)
    size = np.abs(k) @ np.abs(q) * abs(scale)
    top = np.abs(q).max()
    small = np.abs(q) < 2.0 ** -13 * top
    d = 2.0 ** -17 * size + 2.0 ** -21 * top * np.abs(k[:, small]).sum(1) * abs(scale) + 2.0 ** -22 * (1 + np.abs(z))
    want, mass = w @ v, w @ np.abs(v)
    bound = (6 * 2.0 ** -11 / 3 ** 0.5 * np.sqrt(w ** 2 @ v ** 2)
             + 2.0 ** -25 * np.abs(code[P < 2.0 ** -14]).sum(0) / (P @ 2.0 ** -ev)
             + 2 * (w * d) @ np.abs(v) + len(z) * 2.0 ** -23 * mass + (2.0 ** -20 + 2.0 ** -8) * np.abs(want))
    lse = z.max() + np.log(total)
    return want, lse, bound, d[w > 2.0 ** -30].max() + 2.0 ** -20 * (1 + abs(lse))


def _requests(s):
    """(first row, positions from, heads' keys, codes and exponents) of each request and KV head."""
    table, off = s["table"].cpu().numpy(), s["off"].cpu().numpy()
    (kc, ke), (vc, ve) = ((t.cpu().numpy() for t in s[x]) for x in ("k", "v"))
    page = kc.shape[2]
    for b, (kv, n) in enumerate(s["lengths"]):
        pages = table[b, :-(-kv // page)]
        for h in range(kc.shape[1]):
            k = KV.dequantize(kc[pages][:, h:h + 1], ke[pages][:, h:h + 1]).reshape(-1, D)[:kv]
            code = LUT[vc[pages, h].reshape(-1, D)[:kv]]
            ev = np.repeat(ve[pages, h].astype(np.float64) - 127, page)[:kv]
            yield off[b], kv - n, n, h, k, code, ev


def _check(s, out, lse, scale=D ** -0.5, every=1):
    q, out, lse = (t.double().cpu().numpy() for t in (s["q"], out, lse))
    worst = 0.0
    for r0, pos0, n, h, k, code, ev in _requests(s):
        for i in sorted(set(range(0, n, every)) | {n - 1}):
            end = pos0 + i + 1
            for g in range(h * s["G"], (h + 1) * s["G"]):
                want, want_lse, bound, lse_bound = _row(q[r0 + i, g], k[:end], code[:end], ev[:end], scale)
                err = np.abs(out[r0 + i, g] - want)
                worst = max(worst, float((err / bound).max()))
                assert np.all(err <= bound), (r0 + i, g, worst)
                assert abs(lse[r0 + i, g] - want_lse) <= lse_bound, (r0 + i, g)
    return worst


SHAPES = [[(n, 1) for n in (1, 2, 17, 33, 64, 100, 129, 300)], [(100, 3), (257, 4), (65, 2)], [(290, 200)],
          [(300, 90), (70, 1), (130, 64), (64, 64)]]


@pytest.mark.gpu
@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("gain", [0.05, 1.0])
def test_within_its_arithmetic(bfp8, cuda_device, shape, gain):
    """Nearly equal weights, where the rounding of each shows most, and ordinary ones."""
    rng = np.random.default_rng(50 + shape)
    s = _setup(cuda_device, rng, SHAPES[shape], 2, 4, 32, q_gain=gain)
    worst = _check(s, *_run(bfp8, s), every=7)
    print(f"largest error over its bound: {worst:.3f}")


def _one_large_entry(q, k):
    """Queries with one entry of 1, where the keys are 0, and others of 2^-13 to 2^-12, which make the
    scores; returns the scale that brings those to ordinary size."""
    q[..., 1:] = np.sign(q[..., 1:]) * 2.0 ** -13 * (1 + np.minimum(np.abs(q[..., 1:]), 1))
    q[..., 0] = 1.0
    k[..., 0] = 0
    return 2.0 ** 12 * 0.1


@pytest.mark.gpu
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_small_entries_of_a_query_count(bfp8, cuda_device, shape):
    rng = np.random.default_rng(60 + shape)
    s = _setup(cuda_device, rng, SHAPES[shape], 2, 4, 32)
    q, k = s["q"].float().cpu().numpy(), s["k"][0].cpu().numpy()
    scale = _one_large_entry(q, k)
    s["q"].copy_(torch.from_numpy(q))
    s["k"][0].copy_(torch.from_numpy(k))
    print(f"largest error over its bound: {_check(s, *_run(bfp8, s, scale=scale), scale, every=7):.3f}")


# ---- the bounds themselves, without a GPU ----------------------------------------


def _bits(x, n):
    """x to n significant bits."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, n)), e - n)


def _e4m3(x):
    return LUT[F.e4m3_encode_rne_sat(x)]


def _e5m2(x):
    return torch.from_numpy(x).to(torch.float8_e5m2).double().numpy()


def _emulate(q, k, code, ev, scale, round_p, first=_e5m2, top=11):
    """The kernels' arithmetic in float64 but for the roundings of P and of the query's two terms; its
    largest entry is brought to 2^top."""
    up = 2.0 ** (top - np.floor(np.log2(np.abs(q).max())))
    hi = first(q * up)
    z = k @ ((hi + _e4m3(q * up - hi)) / up) * scale
    x = z * np.log2(np.e) + ev
    M = x.max() - 4
    P = 2.0 ** (x - M)
    Z = P @ 2.0 ** -ev
    return KV.bf16(round_p(P) @ code / Z), np.log(2) * (M + np.log2(Z))


def _cases(one_large):
    rng = np.random.default_rng(7)
    for n in (17, 64, 129, 300):
        for gain in (0.05, 1.0):
            q = KV.bf16(rng.normal(size=D) * gain)
            k, code = _e4m3(rng.normal(0, 85, (n, D))) * 2.0 ** -7, _e4m3(rng.normal(0, 85, (n, D)))
            ev = np.repeat(rng.integers(-9, -4, -(-n // 32)), 32)[:n].astype(np.float64)
            scale = D ** -0.5
            if one_large:
                scale = _one_large_entry(q, k)
                q = KV.bf16(q)
            yield q, k, code, ev, scale


@pytest.mark.parametrize("one_large", [False, True])
def test_bounds_hold_the_kernels_arithmetic(one_large):
    for c in _cases(one_large):
        want, lse, bound, lse_bound = _row(*c)
        got, got_lse = _emulate(*c, lambda P: P.astype(np.float16).astype(np.float64))
        assert np.all(np.abs(got - want) <= bound) and abs(got_lse - lse) <= lse_bound


def test_bounds_refuse_weights_of_eight_bits():
    out = [np.any(np.abs(_emulate(*c, lambda P: _bits(P, 8))[0] - _row(*c)[0]) > _row(*c)[2])
           for c in _cases(False)]
    assert np.mean(out) > 0.7, out


def test_bounds_refuse_queries_of_two_e4m3_terms():
    for c in _cases(True):
        want, lse, bound, lse_bound = _row(*c)
        got, got_lse = _emulate(*c, lambda P: P, _e4m3, 8)
        assert np.any(np.abs(got - want) > bound) or abs(got_lse - lse) > lse_bound
