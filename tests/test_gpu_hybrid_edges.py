"""Calls of the hybrid layers' operators that their own tests do not make: two at once on two streams,
memory that is not the GPU's, addresses past 2^32 bytes, and values of very different sizes in one chunk."""

import ctypes

import numpy as np
import pytest
import torch

from hybrid_util import delta_inputs, f64, i32, nan_like, offsets
from oracle import hybrid as HY
from test_gpu_delta_rule import NAMES, _check, _run

pytestmark = pytest.mark.gpu


def test_delta_rules_on_two_streams_at_once(bfp8, cuda_device):
    """Prompts and steps of two batches, each on a stream and with a workspace of its own."""
    dev = cuda_device
    lens = [[300, 1, 70], [2000, 5]]
    t = [delta_inputs(dev, n, 2, 4, 31 + i) for i, n in enumerate(lens)]
    before = [x["state"].clone() for x in t]
    ws = [torch.empty(bfp8.bfp8_delta_rule_workspace(len(n), sum(n), max(n), 2, 4), dtype=torch.uint8, device=dev) for n in lens]
    streams = [torch.cuda.Stream() for _ in lens]
    torch.cuda.synchronize()
    for turn in range(3):
        for x, b in zip(t, before):
            x["state"].copy_(b)
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            bfp8.bfp8_delta_rule(*(t[i][k] for k in NAMES), max(lens[i]), workspace=ws[i], stream=s)
        torch.cuda.synchronize()
        assert bfp8.bfp8_device_status() == 0
        for i, n in enumerate(lens):
            _check(t[i], n, before[i])


def test_state_pool_and_rows_past_2_32_bytes(bfp8, cuda_device):
    """Slots and token rows at both ends of tensors of more than 2^32 bytes; a first request that does not
    begin at row 0."""
    dev = cuda_device
    n_slots, hv, T, wide = 9000, 8, 200000, 12000
    lens = [150, 3]
    t = delta_inputs(dev, lens, 4, hv, 37)
    rows = torch.empty(T, wide, dtype=torch.bfloat16, device=dev)
    big = dict(t, state=torch.zeros(n_slots, hv, 128, 128, device=dev), q_offsets=i32(dev, [T - 153, T - 3, T]))
    at = 0
    for name in ("q", "k", "v"):
        h = t[name].shape[1]
        big[name] = rows[:, at:at + h * 128].view(T, h, 128)
        big[name][T - 153:] = t[name]
        at += h * 128
    big["out"] = rows[:, at:at + hv * 128].view(T, hv, 128)
    big["out"][:] = float("nan")
    at += hv * 128
    for name in ("a", "b"):
        big[name] = rows[:, at:at + hv]
        big[name][T - 153:] = t[name]
        at += 8
    big["state"][n_slots - 2:] = t["state"][:2]
    big["slots_in"], big["slots_out"] = i32(dev, [n_slots - 1, n_slots - 2]), i32(dev, [n_slots - 1, n_slots - 2])
    before = big["state"][n_slots - 2:].clone()
    ws = torch.empty(bfp8.bfp8_delta_rule_workspace(2, T, 150, 4, hv), dtype=torch.uint8, device=dev)
    bfp8.bfp8_delta_rule(*(big[k] for k in NAMES), 150, workspace=ws)
    torch.cuda.synchronize()
    assert bfp8.bfp8_device_status() == 0
    assert not big["state"][:n_slots - 2].any() and torch.isnan(big["out"][:T - 153]).all()
    small = dict(t, out=big["out"][T - 153:], state=big["state"][n_slots - 2:], slots_in=i32(dev, [1, 0]), slots_out=i32(dev, [1, 0]))
    _check(small, lens, before)


def _near(x, S0):
    """What a row may be off because a chunk's products carry its state and values to 2^-22 of the largest of
    them: at each token, and at the end.

    A row's power of two keeps M = max(Gamma_C |S|, the updates of the chunk before, |v| of this one) times it at
    2^-3 or more, and what F16's parts leave out of a number is 2^-22 of it or 2^-25, so 2^-22 of it or of M. Of S
    that is sqrt(128) 2^-22 M in length, and so much in S k', hence in r (whose factors are at most 1); r and u are
    cut once each, 2^-22 M. An error e in r of one token is one of at most e in the row of S (|k'| <= 1), which
    nothing lengthens after that; 64 tokens of 14 2^-22 M each are 896 2^-22 M. (M counts |S| at the chunk's
    begin too, and twice as far as its values' largest, for what S grows to inside the chunk.)"""
    q, k, v = x["q"], x["k"], x["v"]
    g, beta = HY.delta_gates(x["a"], x["b"], x["a_log"], x["dt_bias"])
    n, hv = v.shape[:2]
    group = hv // k.shape[1]
    S, near, updates = np.array(S0), np.zeros(S0.shape[:2]), np.abs(S0).max(-1)
    at = np.zeros((n, hv, 128))
    for c in range(0, n, 64):
        rows = range(c, min(n, c + 64))
        M = np.maximum(np.maximum(updates, np.linalg.norm(S, axis=2)), 2 * np.abs(v[c:c + 64]).max(0))
        add = 896 * 2.0 ** -22 * M
        at[c:c + 64] = near + add
        near = near * np.exp(g[c:c + 64].sum(0))[:, None] + add
        updates = np.zeros_like(updates)
        for t in rows:
            kt = np.repeat(k[t] / np.sqrt((k[t] ** 2).sum(-1, keepdims=True) + 1e-6), group, 0)
            S *= np.exp(g[t])[:, None, None]
            u = beta[t][:, None] * (v[t] - np.einsum("hvk,hk->hv", S, kt))
            S += u[:, :, None] * kt[:, None, :]
            updates = np.maximum(updates * np.exp(g[t])[:, None], np.abs(u))
    return at, near


def _check_near(t, n, before):
    x = {k: f64(t[k])[:n] if k in ("q", "k", "v", "a", "b") else f64(t[k]) for k in ("q", "k", "v", "a", "b", "a_log", "dt_bias")}
    src, dst = int(t["slots_in"][0]), int(t["slots_out"][0])
    S0 = f64(before)[src] if src >= 0 else np.zeros(before.shape[1:])
    want, S, grown, met = HY.delta_rule(x["q"], x["k"], x["v"], x["a"], x["b"], x["a_log"], x["dt_bias"], S0, 128 ** -0.5, 1e-6)
    at, near = _near(x, S0)
    tol = 128 ** -0.5 * (512 * 2.0 ** -24 * met + at)
    out = f64(t["out"])[:n]
    assert np.all(np.abs(out - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    assert np.all(np.linalg.norm(f64(t["state"])[dst] - S, axis=2) <= 512 * 2.0 ** -24 * grown + near)


@pytest.mark.parametrize("ratio", [2.0 ** 10, 2.0 ** 20])
def test_values_of_very_different_sizes_in_a_chunk(bfp8, cuda_device, ratio):
    dev, n = cuda_device, 200
    t = delta_inputs(dev, [n], 1, 2, 41, decay=0.2)
    t["v"][::7] *= ratio
    _check_near(t, n, _run(bfp8, t, [n]))


def test_the_state_turns_tiny_and_huge(bfp8, cuda_device):
    """A row's power of two follows it over 2^-100 .. 2^100 from chunk to chunk, zeros between."""
    dev, n = cuda_device, 64 * 9
    t = delta_inputs(dev, [n], 1, 2, 43, decay=3.0)
    for c, e in enumerate([0, 60, -60, 0, -100, 100, 10, 3, -20]):
        t["v"][64 * c:64 * (c + 1)] *= 2.0 ** e
    t["v"][64 * 3:64 * 4] = 0
    t["a"][:] = 6.0                                  # a decay that leaves nothing of a chunk in the next one's middle
    _check_near(t, n, _run(bfp8, t, [n]))


def test_host_memory_is_refused(bfp8, cuda_device):
    """Pinned or pageable, whoever the caller: by the binding as ValueError, by the library as INVALID_ARG."""
    dev = cuda_device
    t = delta_inputs(dev, [3], 1, 1, 47)
    for name in ("q", "k", "v", "a", "b", "a_log", "dt_bias", "state", "slots_in", "slots_out", "q_offsets", "out"):
        for host in (t[name].cpu(), t[name].cpu().pin_memory()):
            with pytest.raises(ValueError):
                bfp8.bfp8_delta_rule(*((t | {name: host})[k] for k in NAMES), 3)
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device=dev)
    f = torch.ones(32, device=dev)
    pos = i32(dev, [0, 1, 2, 3])
    with pytest.raises(ValueError):
        bfp8.bfp8_rotary(x.cpu(), x, pos, f)
    with pytest.raises(ValueError):
        bfp8.bfp8_rotary(x, x, pos.cpu().pin_memory(), f)
    with pytest.raises(ValueError):
        bfp8.bfp8_gated_norm(x, x.cpu().pin_memory(), None, x)
    c = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev)
    w = torch.zeros(64, 4, dtype=torch.bfloat16, device=dev)
    with pytest.raises(ValueError):
        bfp8.bfp8_causal_conv(c, w.cpu().pin_memory(), torch.empty_like(c), offsets(dev, [4]))
    pinned = torch.zeros(4096, dtype=torch.uint8).pin_memory().data_ptr()
    p = x.data_ptr()
    s = bfp8.bfp8_gated_norm_args(x_bf16=p, x_stride_token=64, x_stride_head=64, gate_bf16=pinned, gate_stride_token=64,
                                  gate_stride_head=64, out_bf16=p, out_stride_token=64, out_stride_head=64, tokens=4, heads=1,
                                  head_dim=64)
    assert bfp8._lib.bfp8_gated_norm(ctypes.byref(s), None) == 1


def test_a_workspace_on_the_host_or_too_small(bfp8, cuda_device):
    dev, n = cuda_device, 100
    t = delta_inputs(dev, [n], 1, 1, 53)
    size = bfp8.bfp8_delta_rule_workspace(1, n, n, 1, 1)
    assert size > 0 and bfp8.bfp8_delta_rule_workspace(1, n, 20, 1, 1) == 0
    for ws in (None, torch.empty(size - 256, dtype=torch.uint8, device=dev)):
        with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
            bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), n, workspace=ws)
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):
        bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), n, workspace=torch.empty(size + 256, dtype=torch.uint8, device=dev)[16:])
    with pytest.raises(ValueError):
        bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), n, workspace=torch.empty(size, dtype=torch.uint8).pin_memory())
    before = _run(bfp8, t, [n])
    _check(t, [n], before)


def test_workspace_grows_with_every_argument(bfp8, cuda_device):
    sizes = lambda **kw: bfp8.bfp8_delta_rule_workspace(**(dict(batch=3, tokens=3000, max_q_len=900, qk_heads=4, v_heads=8) | kw))   # noqa: E731
    for name, steps in (("batch", [1, 2, 3, 7, 64, 500]), ("tokens", [900, 3000, 3001, 20000, 10 ** 6]),
                        ("max_q_len", [1, 20, 21, 64, 900, 1500, 3000, 10 ** 6]), ("qk_heads", [1, 2, 4, 8]), ("v_heads", [4, 8, 16, 64])):
        got = [sizes(**{name: v}) for v in steps]
        assert got == sorted(got), (name, got)
