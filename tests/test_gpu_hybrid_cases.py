"""Drawn cases of the hybrid layers' operators against their definitions in 64 bits.

Each output's error over the whole tensor, in the mean square. BF16 rounding is uniform within half a step:
2^-8 / sqrt(3) = 2.3e-3 of a value at most (of one just above a power of two). FP32 states: a handful of
roundings of 2^-24 a token, which the decay and the rule shorten, and 2^-22 of a chunk's products: 2^-19 is
allowed. Codes: one step, 2^-3 of the value at most, of the few in 100,000 whose quotient lies within 2^-20 of a
border; one in 10,000 gives sqrt(1e-4) 2^-3.
"""

import random

import pytest
import torch

from perf import more_operators as O

pytestmark = pytest.mark.gpu
LIMITS = dict(out=2.4e-3, y=2.4e-3, q=2.4e-3, k=2.4e-3, state=2.0 ** -19, scales=2.0 ** -20, codes=1.3e-3)


def _drawn(op, count, flops, seed):
    rng, out = random.Random(seed), []
    while len(out) < count:
        case = O.draw(rng)
        if case["op"] == op and O.work(case)["flops"] <= flops:
            out.append(case)
    return out


@pytest.mark.parametrize("case", _drawn("conv", 6, 1e9, 1) + _drawn("delta", 16, 6e9, 2) + _drawn("gated", 6, 1e9, 3)
                         + _drawn("rotary", 6, 1e9, 4), ids=str)
def test_drawn_case(monkeypatch, bfp8, cuda_device, case):
    monkeypatch.setattr(O, "own", True)
    got, want = O.run(O.prepare(case, 7)), O.exact(case, 7)
    assert bfp8.bfp8_device_status() == 0
    for name, ref in want.items():
        off = float((got[name].to(torch.float64) - ref).norm() / ref.norm().clamp(min=1e-300))
        assert off <= LIMITS[name], (name, off)
