"""Drawn cases of the attention layer's operators against their definitions in 64 bits.

Whole numbers, codes and scale bytes of the plan and the append are equal. Attention: values are
v <= 448 * 2^-6 = 7 in size, weights are rounded to F16: 2^-9 of the largest value bounds six standard
deviations however the weights lie, and BF16 adds 2^-8 of the output; a score's products sum to 2^-17 of
at most 12 (128 entries of 0.8 and 1.3 on average, / sqrt(128)), so lse is within 2^-13. Residual norm: as
its own tests have it, 2^-18 of the terms and BF16's 2^-8; a code may fall one step aside where its
quotient lies between two, which a few in 100,000 do.
"""

import random

import numpy as np
import pytest
import torch

from perf import operators as O

pytestmark = pytest.mark.gpu


def _drawn(op, count, flops, seed):
    rng, out = random.Random(seed), []
    while len(out) < count:
        case = O.draw(rng)
        if case["op"] == op and O.work(case)["flops"] <= flops:
            out.append(case)
    return out


@pytest.fixture
def own(monkeypatch, bfp8, cuda_device):
    monkeypatch.setattr(O, "own", True)


def _np(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("case", _drawn("plan", 8, 0, 1), ids=str)
def test_plan(own, monkeypatch, case):
    got = O.run(O.prepare(case, 3))
    monkeypatch.setattr(O, "own", False)
    want = O.run(O.prepare(case, 3))
    for name in want:
        assert torch.equal(got[name], want[name]), name


@pytest.mark.parametrize("case", _drawn("append", 6, 1e9, 2), ids=str)
def test_append(own, case):
    got, want = O.run(O.prepare(case, 4)), O.exact(case, 4)
    for name in want:
        assert np.array_equal(_np(got[name]), want[name].astype(np.float64), equal_nan=True), name


@pytest.mark.parametrize("case", _drawn("attn", 10, 3e10, 3), ids=str)
def test_attention(own, case):
    got, want = O.run(O.prepare(case, 5)), O.exact(case, 5)
    out, lse = (x.cpu().numpy() for x in (want["out"], want["lse"]))
    assert np.all(np.abs(_np(got["out"]) - out) <= 2.0 ** -8 * np.abs(out) + 2.0 ** -9 * 7)
    assert np.all(np.abs(_np(got["lse"]) - lse) <= 2.0 ** -13 * (1 + np.abs(lse)))


@pytest.mark.parametrize("case", _drawn("norm", 8, 1e8, 4), ids=str)
def test_norm(own, case):
    s = O.prepare(case, 6)
    got, want = O.run(s), O.exact(case, 6)
    h = want["residual"]
    size = np.abs(h) + 2 * np.abs(s["res_scale"] * _np(s["res"]))
    assert np.all(np.abs(_np(got["residual"]) - h) <= 2.0 ** -8 * np.abs(h) + 2.0 ** -18 * size)
    tol = 2.0 ** -18 * 2 * size / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + s["eps"]) * np.abs(_np(s["w_pre"]))
    if "normed" in want:
        assert np.all(np.abs(_np(got["normed"]) - want["normed"]) <= tol + 2.0 ** -8 * (np.abs(want["normed"]) + tol))
    if "codes" in want:
        off = np.abs(_np(got["codes"]) - want["codes"])
        assert np.all(off <= 2.0 ** -3 * np.abs(want["codes"]) + 2.0 ** -9)
        assert np.mean(off > 0) <= 1e-4 + 3 / off.size
        assert np.allclose(_np(got["scales"]), want["scales"], rtol=2.0 ** -17, atol=0)
