"""bfp8_gated_norm at gates without an end, for the same row in other calls, and at quotients that are exactly the middle
between two codes."""

import numpy as np
import pytest
import torch

from hybrid_util import f64, nan_like
from oracle import formats as F
from oracle import hybrid as HY
from test_gpu_gated_norm import _inputs, _outputs, _run

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("wt", [torch.float32, None])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_gates_without_an_end(bfp8, cuda_device, D, wt, sigmoid):
    """sigmoid(inf) is 1, SiLU(inf) infinite and sigmoid(-inf) 0; gates of +-3e38 are finite and count as far as that.
    Of y the tolerance is that of any gate: tol = (36 + 2.4 max(0, -z)) 2^-24 |y|, and BF16's half step 2^-8."""
    t, o = _inputs(cuda_device, 6, 2, D, D, wt), dict(out=nan_like((6, 2, D), cuda_device))
    gates = [INF, -INF, 3.0e38, -3.0e38]
    for row, z in enumerate(gates):
        t["gate"][row, :, ::3] = z
    t["gate"][4, 0, 5] = INF
    _run(bfp8, t, o, sigmoid=sigmoid)
    z = f64(t["gate"])
    y = HY.gated_norm(f64(t["x"]), np.clip(z, -600, 600), f64(t["weight"]), 1e-6, 0.0, True)   # x times the sigmoid
    with np.errstate(over="ignore", invalid="ignore"):
        want = y if sigmoid else np.where(z <= -3e38, np.where(np.isinf(z), np.nan, -0.0 * y), y * z)
    got = f64(o["out"])
    big = np.abs(want) > 3.39e38                     # BF16's end
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.isinf(got[np.isinf(want)]).all()
    fine = np.isfinite(want) & ~big
    tol = (36 + 2.4 * np.clip(-z, 0, 600)) * 2.0 ** -24 * np.abs(want) + 1e-37
    assert np.all(np.abs(got[fine] - want[fine]) <= (tol + 2.0 ** -8 * (np.abs(want) + tol))[fine])
    assert np.array_equal(np.sign(got[np.isinf(want)]), np.sign(want[np.isinf(want)]))


def test_an_infinite_gate_among_codes(bfp8, cuda_device):
    """The sigmoid of an infinite gate is 1, and its codes are those of a gate of 200, which is 1 too."""
    t, o, far = _inputs(cuda_device, 5, 3, 128, 17), _outputs(cuda_device, 5, 3, 128), _outputs(cuda_device, 5, 3, 128)
    t["gate"][1, 2], t["gate"][3, :, 7], t["gate"][4] = INF, INF, -INF
    _run(bfp8, t, o, sigmoid=True)
    t["gate"].copy_(torch.where(t["gate"] == INF, 200.0, t["gate"]))
    _run(bfp8, t, far, sigmoid=True)
    assert all(torch.equal(o[k], far[k]) for k in o)
    assert not o["out"][4].any() and torch.isfinite(o["out"]).all()


def _tied_rows(T, H, D, largest, seed):
    """BF16 rows whose groups of 128 columns have `largest` as their largest entry, and beside it every entry above
    2^-6 of a code's step that lies in the middle between two codes at a largest of 1.75: 448 / 1.75 is 2^8."""
    g = np.random.default_rng(seed)
    ties = [(1 + (2 * m + 1) / 16) * 2.0 ** e for e in range(-14, 1) for m in range(8)]
    ties = [v for v in ties if v < 1.75]
    x = np.empty((T, H * D))
    for row in x:
        for at in range(0, H * D, 128):
            n = min(128, H * D - at)
            group = np.concatenate([[1.75], g.permutation(ties)[:n - 1], g.uniform(0.01, 1.7, max(0, n - 1 - len(ties)))])
            row[at:at + n] = g.permutation(group) * g.choice([-1.0, 1.0], n)
    return torch.tensor(x * (largest / 1.75)).to(torch.bfloat16).view(T, H, D)


@pytest.mark.parametrize("gate", [1.296875, -2.453125])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_a_row_has_the_same_codes_in_any_call(bfp8, cuda_device, D, gate):
    """Rows full of codes that FP32's last bits decide: alone, next to others, 8192 of them, and over their own input."""
    dev, H = cuda_device, 6144 // D
    row = torch.cat([_tied_rows(1, H, D, 1.75, D), _inputs("cpu", 1, H, D, 5 + D)["x"]]).to(dev)
    calls = []
    for order in ([0], [1, 0], [0] * 40 + [1] * 3 + [0], [0] * 8192):
        t = dict(x=row[order].contiguous(), weight=None)
        t["gate"] = torch.full_like(t["x"], gate)
        o = _outputs(dev, len(order), H, D)
        _run(bfp8, t, o)
        calls.append((order, o))
        over = dict(_outputs(dev, len(order), H, D), out=t["x"])
        _run(bfp8, t, over)
        calls.append((order, over))
    want = {0: calls[0][1], 1: {k: v[:1] for k, v in calls[2][1].items()}}
    for order, o in calls:
        at = torch.tensor(order, device=dev)
        for r in set(order):
            for k in ("q", "scales"):
                assert (o[k][at == r] == want[r][k]).all(), (order[:3], len(order), k)
            assert torch.equal(o["out"][at == r][-1:], want[r]["out"])
@pytest.mark.parametrize("T,H,D", [(1, 1, 128), (3, 4, 64), (40, 3, 128), (9, 5, 256)])
@pytest.mark.parametrize("largest", [1.75, 1.75 * 2.0 ** -9, 1.0, 1.75 * 2.0 ** 20])
@pytest.mark.parametrize("gate,sigmoid", [(0.0, True), (40.0, True), (1.296875, False), (-2.453125, False)])
@pytest.mark.parametrize("weight", [None, 0.75, 1.0])
def test_quotients_in_the_middle_go_to_the_even_code(bfp8, cuda_device, T, H, D, largest, gate, sigmoid, weight):
    """One gate and one weight for a whole row: they cancel from y / max|y|, whose middles are then those of 448 x / max|x|,
    which float64 has without rounding (8 bits by 9, over 1 or 7 / 4). A norm cancels within a head; of heads of 64 there are
    two to a group, so there without."""
    if weight is not None and D == 64:
        return
    dev = cuda_device
    x = _tied_rows(T, H, D, largest, 3 * T + D)
    if largest == 1.0:                               # where the middles are 3 / 2 of powers of two: 448 is 7 / 4 of one
        x.view(T, -1)[:, 1::5] = 1.5 * torch.exp2(-1 - torch.arange(H * D)[1::5] % 12).to(torch.bfloat16)
        x.view(T, -1)[:, ::128] = 1.0
    t = dict(x=x.to(dev), gate=torch.full_like(x, gate).to(dev), weight=None if weight is None else torch.full((D,), weight, device=dev))
    o = _outputs(dev, T, H, D)
    _run(bfp8, t, o, sigmoid=sigmoid)
    flat = f64(t["x"]).reshape(T, -1)
    top = np.repeat(np.maximum.reduceat(np.abs(flat), np.arange(0, H * D, 128), axis=1), 128, axis=1)[:, :H * D]
    quotient = 448 * flat / top
    want = F.e4m3_encode_rne_sat(quotient if gate > 0 or sigmoid else -quotient)
    plain = np.abs(quotient) > 2.0 ** -6 * 1.01
    assert np.array_equal(o["q"].cpu().numpy()[plain], want[plain])
