"""Pins for oracle/kv.py: block plans written out by hand, scale exponents from
their definition in exact rationals, appends against torch's float8 cast, and
attention against closed forms (uniform weights, one key, a window of one).
"""

from fractions import Fraction

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kv as KV


def test_plan_by_hand():
    # page 4: request 0 holds 5 tokens (2 pages) and gets 4 more (1 new page);
    # request 1 holds none and gets 1; request 2 holds 4 (full page), gets none
    table = [[7, 3, -1], [-1, -1, -1], [9, -1, -1]]
    t, off, kv, slots, pos, counts = KV.block_plan([5, 0, 4], [4, 1, 0], [11, 12, 13], table, 4, 7)
    assert t.tolist() == [[7, 3, 11], [12, -1, -1], [9, -1, -1]]
    assert off.tolist() == [0, 4, 5, 5] and kv.tolist() == [9, 1, 4]
    assert slots.tolist() == [13, 14, 15, 44, 48, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 0, -1, -1] and counts == [2, 0, 0]


def test_plan_short_of_pages_and_of_width():
    t, off, kv, slots, pos, counts = KV.block_plan([0, 0], [3, 9], [5], [[-1, -1], [-1, -1]], 4, 12)
    assert t.tolist() == [[5, -1], [-1, -1]] and counts == [1, 2, 9]
    assert slots.tolist() == [20, 21, 22] + [-1] * 9
    assert pos.tolist() == [0, 1, 2] + list(range(9))


def test_plan_counts_every_token_without_a_page():
    # page 4: request 0 continues a page that is not there (2 tokens) and gets a new one (1 token);
    # request 1 continues one that is; request 2 needs no page, with 4 tokens on a missing page ahead of its own
    t, off, kv, slots, pos, counts = KV.block_plan([2, 1, 4], [3, 2, 1], [9, 8], [[-1, -1], [6, -1], [-1, -1]], 4, 6)
    assert slots.tolist() == [-1, -1, 36, 25, 26, 32] and counts == [2, 0, 2]


@pytest.mark.parametrize("amax", [0.0, 1e-30, 448.0, 448.0000001, 449.0, 1.0, 0.875, 0.8750001, 3.5, 3.4e38])
def test_scale_exponent_is_the_least(amax):
    e = KV.scale_exponent(amax)
    a = Fraction(amax)
    fits = lambda k: a <= 448 * Fraction(2) ** k   # noqa: E731
    assert (fits(e) or e == KV.MAX_EXP) and (e == KV.MIN_EXP or not fits(e - 1))


def test_append_matches_torch_cast_and_moves_old_codes():
    rng = np.random.default_rng(0)
    x = rng.normal(size=(3, 1, 8))
    codes, exps = KV.append(x, [4, 5, 9], np.zeros((3, 1, 4, 8), np.uint8), np.full((3, 1), 87, np.uint8))
    for p, rows, off in ((1, [0, 1], 0), (2, [2], 1)):
        e = int(exps[p, 0]) - 127
        want = torch.tensor(x[rows, 0] * 2.0 ** -e, dtype=torch.float32).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes[p, 0, off:off + len(rows)], want)
    # a value 2^6 times the page's loudest raises its exponent by 6 and keeps the old values
    before = KV.dequantize(codes, exps)[1, 0, :2]
    loud = np.zeros((1, 1, 8))
    loud[0, 0, 0] = np.abs(x[:2]).max() * 64
    c2, e2 = KV.append(loud, [6], codes, exps)
    assert int(e2[1, 0]) == int(exps[1, 0]) + 6
    after = KV.dequantize(c2, e2)[1, 0, :2]
    assert np.all(np.abs(after - before) <= 2.0 ** (int(e2[1, 0]) - 127 - 10))   # half a subnormal step


def test_attention_closed_forms():
    rng = np.random.default_rng(1)
    k, v = rng.normal(size=(3, 1, 2, 4)), rng.normal(size=(3, 1, 2, 4))
    table = [[2, 0]]
    zero = np.zeros((1, 2, 4))
    out, lse = KV.attention(zero, k, v, table, [0, 1], [3], 1.0)      # equal weights
    want = (v[2, 0, 0] + v[2, 0, 1] + v[0, 0, 0]) / 3
    assert np.allclose(out[0], want, rtol=1e-14) and np.allclose(lse, np.log(3.0), rtol=1e-14)
    q = rng.normal(size=(2, 2, 4))
    out, lse = KV.attention(q, k, v, table, [0, 2], [3], 0.5, window=0)   # only itself
    assert np.allclose(out[0], v[2, 0, 1]) and np.allclose(out[1], v[0, 0, 0])
    assert np.allclose(lse[1], q[1] @ k[0, 0, 0] * 0.5)
    out, lse = KV.attention(q, k, v, table, [0, 2], [1], 0.5)         # row 0 before the first position
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(out[1], v[2, 0, 0])
    out, lse = KV.attention(q, k, v, [[-1, 0]], [0, 2], [2], 0.5)     # a missing page
    assert np.all(out == 0) and np.all(np.isneginf(lse))


def test_residual_norm_closed_forms():
    h, n = KV.residual_norm(np.full((1, 4), 3.0), np.ones((1, 4)), np.full(4, 2.0), np.ones(4), 0.5, 0.25, 0.0)
    assert np.allclose(h, 0.25 + 0.5 * 2.0) and np.allclose(n, 1.0)
    h, n = KV.residual_norm(None, np.array([[3.0, 4.0]]), w_pre=np.zeros(2), offset=1.0, eps=0.0)
    assert np.allclose(n, np.array([[3.0, 4.0]]) / np.sqrt(12.5))


def test_bf16_is_half_a_step_away_at_most():
    x = np.random.default_rng(2).normal(size=1000)
    assert np.max(np.abs(KV.bf16(x) - x) / np.abs(x)) <= 2.0 ** -8      # 8 significant bits
    assert F.f64_to_bf16_bits(KV.bf16(x)).tolist() == F.f64_to_bf16_bits(x).tolist()
