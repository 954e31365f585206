"""The hybrid layers' oracle against closed forms (float64 on the CPU)."""

import math

import numpy as np
import pytest

from oracle import hybrid as HY


def test_convolution_of_an_impulse_is_the_weights_backwards():
    w = np.array([[1.0, 2.0, 4.0, 8.0], [0.5, 0.0, -1.0, 3.0]])
    x = np.zeros((6, 2))
    x[1] = 1.0
    out, last, size = HY.causal_conv(x, w, None, np.zeros((3, 2)), silu=False)
    assert np.array_equal(out[1:5], w[:, ::-1].T) and not out[0].any() and not out[5].any()
    assert np.array_equal(last, x[3:]) and np.array_equal(size, np.abs(out))


def test_convolution_in_two_steps_is_that_in_one():
    rng = np.random.default_rng(1)
    x, w, b = rng.normal(size=(9, 5)), rng.normal(size=(5, 4)), rng.normal(size=5)
    first = rng.normal(size=(3, 5))
    whole, last, _ = HY.causal_conv(x, w, b, first)
    for cut in (1, 2, 3, 8):
        one, mid, _ = HY.causal_conv(x[:cut], w, b, first)
        two, end, _ = HY.causal_conv(x[cut:], w, b, mid)
        assert np.allclose(np.concatenate([one, two]), whole, rtol=1e-13) and np.array_equal(end, last)


def _rule(q, k, v, a, b, a_log, dt, S, scale=1.0):
    return HY.delta_rule(q, k, v, a, b, a_log, dt, S, scale, 0.0)


def test_delta_rule_stores_what_it_is_told():
    """beta = 1 and no decay: a key met again returns its latest value, orthogonal keys do not disturb it."""
    rng = np.random.default_rng(2)
    k = np.linalg.qr(rng.normal(size=(128, 128)))[0][:4].reshape(4, 1, 128)[[0, 1, 2, 0]] * 3.0
    v = rng.normal(size=(4, 1, 128))
    a, b = np.full((4, 1), -800.0), np.full((4, 1), 800.0)
    out, S, *_ = _rule(k, k, v, a, b, np.zeros(1), np.zeros(1), np.zeros((1, 128, 128)))
    assert np.allclose(out, v, atol=1e-12)                       # each key, asked at once
    unit = k[:, 0] / 3.0
    assert np.allclose(S[0] @ unit[0], v[3, 0], atol=1e-12)      # the second value of key 0
    assert np.allclose(S[0] @ unit[1], v[1, 0], atol=1e-12)


def test_delta_rule_decays_alone():
    """beta = 0: the state shrinks by exp(-exp(a_log) softplus(a + dt)) a token, and queries are scaled."""
    S = np.random.default_rng(3).normal(size=(2, 128, 128))
    q = np.zeros((3, 1, 128))
    q[:, 0, 5] = 7.0
    a, a_log, dt = np.full((3, 2), 0.25), np.log([1.0, 4.0]), np.array([-0.25, 0.5])
    out, end, grown, met = _rule(q, q, np.zeros((3, 2, 128)), a, np.full((3, 2), -800.0), a_log, dt, S, scale=0.5)
    for h, keep in enumerate([0.5, math.exp(-4 * math.log1p(math.exp(0.75)))]):
        assert np.allclose(end[h], S[h] * keep ** 3, rtol=1e-13)
        assert np.allclose(out[2, h], 0.5 * S[h, :, 5] * keep ** 3, rtol=1e-13)
    assert np.all(grown > 0) and np.all(met[-1] > grown)


def test_delta_rule_bound_holds_an_error_in_the_state():
    """An error put into a row of the state comes out no longer than the bound's recursion says."""
    rng = np.random.default_rng(4)
    n = 20
    q, k, v = rng.normal(size=(n, 1, 128)), rng.normal(size=(n, 1, 128)), rng.normal(size=(n, 2, 128))
    a, b = rng.normal(size=(n, 2)), rng.normal(size=(n, 2))
    rest = (a, b, np.array([-3.0, 0.0]), np.zeros(2))
    S = rng.normal(size=(2, 128, 128))
    e = 1e-6 * rng.normal(size=S.shape)
    _, one, *_ = _rule(q, k, v, *rest, S)
    _, two, *_ = _rule(q, k, v, *rest, S + e)
    keep = np.exp(HY.delta_gates(*rest)[0].sum(0))[:, None]
    assert np.all(np.linalg.norm(two - one, axis=2) <= keep * np.linalg.norm(e, axis=2) * (1 + 1e-6) + 1e-14)


def test_gated_norm_of_a_constant_row():
    x = np.full((1, 2, 64), 3.0)
    z = np.zeros((1, 2, 64))
    w = np.arange(64.0)
    assert np.allclose(HY.gated_norm(x, z, w, 0.0, 1.0, sigmoid=True), 0.5 * (w + 1))
    assert not HY.gated_norm(x, z, w, 0.0).any()
    assert np.allclose(HY.gated_norm(x, z + 1, None, 0.0), 3.0 / (1 + math.exp(-1)))


def test_axes_of_the_pairs():
    assert HY.axis_of_pair(6, [3, 2, 1], False) == [0, 0, 0, 1, 1, 2]
    assert HY.axis_of_pair(8, [4, 2, 2], True) == [0, 1, 2, 0, 1, 2, 0, 0]


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotary_turns_by_quarters_and_back(adjacent):
    """A quarter turn swaps a pair's members; turning by p and then reading at -p's angle gives the row back."""
    rng = np.random.default_rng(5)
    x = rng.normal(size=(3, 1, 64))
    pos = np.array([[0, 1, 2]])
    f = np.full(16, math.pi / 2, dtype=np.float32)
    y, size = HY.rotary(x, pos, f, [16], adjacent=adjacent)
    a, b = (x[1, 0, 0:32:2], x[1, 0, 1:32:2]) if adjacent else (x[1, 0, :16], x[1, 0, 16:32])
    ya, yb = (y[1, 0, 0:32:2], y[1, 0, 1:32:2]) if adjacent else (y[1, 0, :16], y[1, 0, 16:32])
    assert np.allclose(y[0], x[0]) and np.allclose(ya, -b, atol=1e-7) and np.allclose(yb, a, atol=1e-7)
    assert np.array_equal(y[..., 32:], x[..., 32:]) and np.all(size >= np.abs(y) - 1e-12)
    back, _ = HY.rotary(y, pos, -f, [16], adjacent=adjacent)
    assert np.allclose(back, x)


def test_rotary_counts_far_positions_in_whole_turns():
    """A frequency of 2^-k radians and a position: against exact remainders of integer arithmetic."""
    pos = np.array([[2 ** 31 - 1, 1_000_003, -1]])
    f = np.array([0.75], dtype=np.float32)
    y, _ = HY.rotary(np.tile([1.0, 0.0], (3, 1, 1)), pos, f, [1])
    pi = 314159265358979323846264338327950288419716939937510     # 50 digits
    for t, p in enumerate(pos[0][:2]):
        rest = ((int(p) * 3 * 10 ** 50) % (8 * pi)) / 4 / 10 ** 50
        assert abs(y[t, 0, 0] - math.cos(rest)) < 1e-9 and abs(y[t, 0, 1] - math.sin(rest)) < 1e-9
    assert np.isnan(y[2]).all()
