"""bfp8_causal_conv on the GPU against the oracle in float64.

Tolerances. The sum of W products and the bias is within (W + 1) 2^-24 of its terms' sizes; SiLU has a slope of
at most 1.1 and, with the approximate exponential, is within (4 + 1.2 max(0, -y)) 2^-23 of itself and two more
roundings; BF16 adds half a step, 2^-8. The state holds inputs, unchanged.
"""

import numpy as np
import pytest
import torch

from hybrid_util import f64, i32, nan_like, offsets
from oracle import hybrid as HY

pytestmark = pytest.mark.gpu


def _inputs(dev, lens, C, W, dtype, bias, seed, extra=0, pitch=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    T, B = sum(lens) + extra, len(lens)
    order = torch.randperm(2 * B + 1, generator=g).tolist()
    wide = (2 * r(T, C + pitch)).to(torch.bfloat16).to(dev)
    return dict(x=wide[:, pitch:], weight=r(C, W).to(dtype).to(dev), bias=r(C).to(dtype).to(dev) if bias else None,
                state=r(2 * B + 1, W - 1, C).to(torch.bfloat16).to(dev), q_offsets=offsets(dev, lens),
                slots_in=i32(dev, [-1 if b % 3 == 2 else order[b] for b in range(B)]), slots_out=i32(dev, order[B:2 * B]),
                out=nan_like((T, C), dev))


def _check(t, lens, before, silu=True):
    x, w, b = f64(t["x"]), f64(t["weight"]), f64(t["bias"])
    W, at = w.shape[1], 0
    want_state = f64(before)
    out, state = f64(t["out"]), f64(t["state"])
    for n, src, dst in zip(lens, t["slots_in"].tolist(), t["slots_out"].tolist()):
        first = f64(before)[src] if src >= 0 else np.zeros((W - 1, x.shape[1]))
        want, last, size = HY.causal_conv(x[at:at + n], w, b, first, silu)
        err = (W + 1) * 2.0 ** -24 * size
        if silu:
            y = HY.causal_conv(x[at:at + n], w, b, first, False)[0]
            err = 1.1 * err + (6 + 1.2 * np.maximum(0, -y)) * 2.0 ** -23 * np.abs(want)
        assert np.all(np.abs(out[at:at + n] - want) <= err + 2.0 ** -8 * (np.abs(want) + err) + 1e-38)
        if n and 0 <= dst < len(want_state):
            want_state[dst] = last
        at += n
    assert np.isnan(out[at:]).all()                  # rows behind the last request
    assert np.array_equal(state, want_state)


def _run(bfp8, t, **kw):
    before = t["state"].clone()
    bfp8.bfp8_causal_conv(t["x"], t["weight"], t["out"], t["q_offsets"], t["state"], t["slots_in"], t["slots_out"],
                          bias=t["bias"], **kw)
    torch.cuda.synchronize()
    return before


LENS = [[1], [1, 1, 1, 1, 1], [2, 0, 3, 1, 4], [0, 0, 0], [5, 31, 32, 33], [64, 1, 0, 100, 2], [300], [3] * 40, [1] * 200]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("C,W,dtype,bias", [(8, 4, torch.bfloat16, False), (1032, 4, torch.float32, True), (256, 3, torch.bfloat16, True),
                                            (520, 2, torch.float32, False)])
def test_matches_oracle(bfp8, cuda_device, lens, C, W, dtype, bias):
    t = _inputs(cuda_device, lens, C, W, dtype, bias, C + sum(lens), extra=3, pitch=16)
    _check(t, lens, _run(bfp8, t))


def test_without_activation_and_without_state(bfp8, cuda_device):
    lens = [7, 1, 40]
    t = _inputs(cuda_device, lens, 64, 4, torch.bfloat16, True, 1)
    _check(t, lens, _run(bfp8, t, silu=False), silu=False)
    t["slots_in"].fill_(-1)
    want = nan_like(t["out"].shape, cuda_device)
    before = t["state"].clone()
    bfp8.bfp8_causal_conv(t["x"], t["weight"], want, t["q_offsets"], t["state"], t["slots_in"], None, bias=t["bias"])
    bfp8.bfp8_causal_conv(t["x"], t["weight"], t["out"], t["q_offsets"], bias=t["bias"])
    assert torch.equal(want, t["out"]) and torch.equal(before, t["state"])


@pytest.mark.parametrize("cuts", [[1] * 9, [2, 7], [4, 1, 1, 3], [8, 1]])
def test_steps_in_one_slot_are_the_whole_prompt(bfp8, cuda_device, cuts):
    """The same slot read and written, in pieces: bit for bit what one call over the prompt gives."""
    dev = cuda_device
    t = _inputs(dev, [9], 128, 4, torch.bfloat16, True, 3)
    slot = i32(dev, [1])
    t["state"][1] = 0
    bfp8.bfp8_causal_conv(t["x"], t["weight"], t["out"], t["q_offsets"], bias=t["bias"])
    got, at = torch.empty_like(t["out"]), 0
    for n in cuts:
        bfp8.bfp8_causal_conv(t["x"][at:at + n], t["weight"], got[at:at + n], offsets(dev, [n]), t["state"], slot, slot,
                              bias=t["bias"])
        at += n
    assert torch.equal(got, t["out"]) and torch.equal(t["state"][1], t["x"][-3:])


def test_slots_outside_the_pool_and_offsets_outside_the_rows(bfp8, cuda_device):
    dev = cuda_device
    lens = [3, 40, 2]
    t = _inputs(dev, lens, 64, 4, torch.bfloat16, False, 4)
    t["slots_in"][:] = i32(dev, [7, -5, 2 ** 31 - 1])
    t["slots_out"][:] = i32(dev, [2 ** 31 - 1, 6, -1])
    before = _run(bfp8, t)
    t["slots_in"][:] = -1                            # what the oracle is told: all three begin from zeros
    t["slots_out"][:] = i32(dev, [-1, 6, -1])
    _check(t, lens, before)
    t["q_offsets"][:] = i32(dev, [-4, 3, 43, 1000])  # clamped to the rows
    again = t["out"].clone()
    _run(bfp8, t)
    assert torch.equal(t["out"], again)


def test_nan_stays_in_its_request_and_window(bfp8, cuda_device):
    dev = cuda_device
    lens = [50, 50, 50]
    t = _inputs(dev, lens, 64, 4, torch.float32, True, 5)
    _run(bfp8, t)
    clean = t["out"].clone()
    t["x"][70, 9] = float("nan")
    _run(bfp8, t)
    bad = torch.isnan(t["out"])
    assert bad[70:74, 9].all() and bad.sum() == 4
    assert torch.equal(t["out"][~bad], clean[~bad])


def test_largest_offsets(bfp8, cuda_device):
    """More than 2^32 bytes of rows: 70000 tokens of 32768 channels, a request that ends in the last of them."""
    dev = cuda_device
    T, C = 70000, 32768
    x = torch.zeros(T, C, dtype=torch.bfloat16, device=dev)
    x[-5:] = torch.randn(5, C, device=dev).to(torch.bfloat16)
    w = torch.randn(C, 4, device=dev).to(torch.bfloat16)
    out = torch.empty_like(x)
    bfp8.bfp8_causal_conv(x, w, out, offsets(dev, [10, T - 10]))
    want, _, size = HY.causal_conv(f64(x[-5:]), f64(w), None, np.zeros((3, C)))
    assert np.all(np.abs(f64(out[-5:]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * (size + 1) * (1 + size))
    assert not out[:-5].any()


def test_captured_step_follows_its_inputs(bfp8, cuda_device):
    """Captured once, replayed with other lengths, slots and inputs, on a stream of its own."""
    dev = cuda_device
    t = _inputs(dev, [5, 60, 0, 2], 256, 4, torch.bfloat16, True, 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bfp8.bfp8_causal_conv(t["x"], t["weight"], t["out"], t["q_offsets"], t["state"], t["slots_in"], t["slots_out"],
                              bias=t["bias"])
    for lens in ([5, 60, 0, 2], [1, 1, 1, 1], [0, 0, 67, 0], [33, 2, 30, 2]):
        t["q_offsets"].copy_(offsets(dev, lens))
        t["x"].copy_(torch.randn(t["x"].shape, device=dev))
        t["out"].fill_(float("nan"))
        before = t["state"].clone()
        graph.replay()
        torch.cuda.synchronize()
        _check(t, lens, before)


def test_refusals(bfp8, cuda_device):
    dev = cuda_device
    t = _inputs(dev, [4], 64, 4, torch.bfloat16, True, 7)
    call = lambda **kw: bfp8.bfp8_causal_conv(**({k: t[k] for k in ("x", "weight", "out", "q_offsets", "state", "slots_in",
                                                                      "slots_out", "bias")} | kw))   # noqa: E731
    call()
    for bad in (dict(x=t["x"].float()), dict(out=t["out"][:3]), dict(weight=t["weight"].t()), dict(bias=t["bias"][:8]),
                dict(bias=t["bias"].float()), dict(state=t["state"][:, :2]), dict(state=t["state"].float()),
                dict(state=None), dict(slots_in=t["slots_in"].long()), dict(q_offsets=t["q_offsets"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad, status in ((dict(out=t["x"]), "INVALID_ARG"), (dict(weight=t["weight"].half(), bias=None), "SCALE_DTYPE")):
        with pytest.raises(bfp8.Bfp8Error, match=status):
            call(**bad)
