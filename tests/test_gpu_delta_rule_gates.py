"""bfp8_delta_rule where its write gates beta are small: a state that many small writes make has the digits of its own
size, by chunks as by single tokens.

Tolerances. A token adds beta (v - alpha S k') k'^T to the state, so what FP32 leaves out of a row of it is at most
c (1 + |g|) 2^-24 (alpha |S_row| + beta |v|), c = 512 by chunks and 64 by steps (the reasons are those of the delta rule's
other tests, with beta |v| for |v|: beta is a factor of the whole of u). By chunks there is 2^-22 of M too, the largest of the
row's state at the chunk's begin, its updates, and the chunk's largest beta times its largest |v|: M times the row's power of
two is 2^-3 or more, and F16's two parts leave out 2^-22 of a number or 2^-25, hence 2^-22 of M. Of S that is
sqrt(128) 2^-22 M in length, and as much in S k'; r and u are cut once each: 14 2^-22 M a token, 896 2^-22 M a chunk of 64,
which nothing after it lengthens.
"""

import numpy as np
import pytest
import torch

from hybrid_util import delta_inputs, f64
from oracle import hybrid as HY
from test_gpu_delta_rule import _run

pytestmark = pytest.mark.gpu


def _check_written(t, n, before, by_chunks):
    x = {k: f64(t[k])[:n] if k in ("q", "k", "v", "a", "b") else f64(t[k]) for k in ("q", "k", "v", "a", "b", "a_log", "dt_bias")}
    src, dst = int(t["slots_in"][0]), int(t["slots_out"][0])
    S = f64(before)[src] if src >= 0 else np.zeros(before.shape[1:])
    g, beta = HY.delta_gates(x["a"], x["b"], x["a_log"], x["dt_bias"])
    hv, group, scale = x["v"].shape[1], x["v"].shape[1] // x["k"].shape[1], 128 ** -0.5
    unit = lambda r: np.repeat(r / np.sqrt((r ** 2).sum(-1, keepdims=True) + 1e-6), group, 0)   # noqa: E731
    c = 512 if by_chunks else 64
    out, rows = f64(t["out"]), np.zeros((hv, 128))
    updates = np.abs(S).max(-1)
    for at in range(0, n, 64):
        some = range(at, min(n, at + 64))
        written = beta[some].max(0)[:, None] * np.abs(x["v"][some]).max(0)
        if by_chunks:
            rows += 896 * 2.0 ** -22 * np.maximum(np.maximum(updates, np.linalg.norm(S, axis=2)), 2 * written)
        updates = np.zeros_like(updates)
        for i in some:
            alpha, write = np.exp(g[i])[:, None], beta[i][:, None]
            kt, qt = unit(x["k"][i]), unit(x["q"][i]) * scale
            rows = (rows if by_chunks else alpha * rows) + c * 2.0 ** -24 * (1 + np.abs(g[i])[:, None]) * (alpha * np.linalg.norm(S, axis=2) + write * np.abs(x["v"][i]))
            S = alpha[..., None] * S
            u = write * (x["v"][i] - np.einsum("hvk,hk->hv", S, kt))
            S = S + u[:, :, None] * kt[:, None, :]
            updates = np.maximum(updates * alpha, np.abs(u))
            want = np.einsum("hvk,hk->hv", S, qt)
            tol = scale * (rows + c * 2.0 ** -24 * np.linalg.norm(S, axis=2))
            off = np.abs(out[i] - want)
            assert np.all(off <= tol + 2.0 ** -8 * (np.abs(want) + tol)), (i, float(np.max(off / (tol + 2.0 ** -8 * np.abs(want)))))
    off = np.linalg.norm(f64(t["state"])[dst] - S, axis=2)
    assert np.all(off <= rows), float(np.max(off / rows))


@pytest.mark.parametrize("b", [-6.0, -10.0, -14.0, -20.0, -60.0])
@pytest.mark.parametrize("n", [3, 20, 21, 64, 200])
@pytest.mark.parametrize("held", [0.0, 1e-6])
def test_small_write_gates(bfp8, cuda_device, n, b, held):
    t = delta_inputs(cuda_device, [n], 1, 2, 61 + n, decay=0.01)
    t["b"].copy_(t["b"].float() * 0.3 + b)
    t["state"] *= held
    t["slots_in"].fill_(-1 if held == 0.0 else int(t["slots_in"][0]))
    before = _run(bfp8, t, [n])
    _check_written(t, n, before, n > 20)


@pytest.mark.parametrize("b", [-10.0, -16.0])
def test_small_write_gates_of_long_prompts(bfp8, cuda_device, b):
    """Chunks walked in segments."""
    n = 2500
    t = delta_inputs(cuda_device, [n], 1, 1, 71, decay=0.002)
    t["b"].copy_(t["b"].float() * 0.3 + b)
    t["slots_in"].fill_(-1)
    _check_written(t, n, _run(bfp8, t, [n]), True)


def test_write_gates_that_change_from_chunk_to_chunk(bfp8, cuda_device):
    """From shut to open and back, with heads that forget in between; a chunk whose gates are all zero writes nothing."""
    n = 64 * 8 + 30
    t = delta_inputs(cuda_device, [n], 1, 2, 73, decay=1.0)
    for i, b in enumerate([-12.0, -3.0, 0.0, -18.0, -float("inf"), -9.0, 4.0, -30.0, -5.0]):
        t["b"][64 * i:64 * i + 64] = b
    t["a"][64 * 3:] += 2.0
    t["slots_in"].fill_(-1)
    _check_written(t, n, _run(bfp8, t, [n]), True)


@pytest.mark.parametrize("b", [-88.0, -87.5, -89.0])
def test_gates_whose_beta_is_subnormal(bfp8, cuda_device, b):
    """beta is 6e-39 at b = -88 and 0 from -89 on; values of 2^100 write with it all the same, beside a smaller state."""
    n = 100
    t = delta_inputs(cuda_device, [n], 1, 2, 79, decay=0.01)
    t["b"][:] = b
    t["v"].copy_(t["v"].float() * 2.0 ** 100)
    t["state"] *= 2.0 ** -100
    before = _run(bfp8, t, [n])
    if b > -89.0:
        _check_written(t, n, before, True)
    else:                                            # nothing is written: the state decays, near its own size
        assert torch.isfinite(t["out"][:n]).all()
        assert (t["state"][int(t["slots_out"][0])].abs() < 2.0 ** -96).all()
