"""bfp8_delta_rule: one long prompt with more and more single tokens beside it. How many segments its chunks are walked in
goes by all of the call's requests, so its last bits may differ, and each call keeps the bounds of the delta rule's tests."""

import pytest
import torch

from hybrid_util import delta_inputs, nan_like, offsets
from test_gpu_delta_rule import _check, _run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,hk,hv", [(3000, 2, 4), (2500, 1, 8)])
def test_a_long_prompt_alone_and_among_others(bfp8, cuda_device, n, hk, hv):
    dev, most = cuda_device, 60
    t = delta_inputs(dev, [n] + [1] * most, hk, hv, 83 + n, decay=0.05)
    start, got = t["state"].clone(), {}
    for beside in (0, 3, 9, 18, 40, most):           # 4 heads: segments up to 18 single tokens, one walk from 37 on
        lens = [n] + [1] * beside
        T = sum(lens)
        part = dict(t, **{k: t[k][:T] for k in ("q", "k", "v", "a", "b")}, **{k: t[k][:len(lens)] for k in ("slots_in", "slots_out")},
                    q_offsets=offsets(dev, lens), state=start.clone(), out=nan_like((T, hv, 128), dev))
        _check(part, lens, _run(bfp8, part, lens))
        got[beside] = part["out"][:n], part["state"][part["slots_out"][0]]
    for a, b in zip(got[40], got[most]):             # the same way through: the same bits
        assert torch.equal(a, b)
