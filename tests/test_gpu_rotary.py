"""bfp8_rotary on the GPU against the oracle in float64.

Tolerances. The angle in turns is within 2^-64 a position and its float32 within 2^-25 of half a turn: pi 2^-25
radians; sine and cosine add 2 units of 2^-24; with the factor's product each is within 5 2^-24. A pair's turn then
is within (5 + 3) 2^-24 (|a| + |b|) |factor|, the heads' norm adds 20 2^-24 of the same (13 roundings of its sum of
squares, halved, the root, the weight's sum and two products), and BF16 half a step, 2^-8.
"""

import numpy as np
import pytest
import torch

from hybrid_util import f64, nan_like
from oracle import hybrid as HY

pytestmark = pytest.mark.gpu


def _inputs(dev, T, hq, hk, D, r, axes, seed, wt=None, far=5000):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    rows = rn(T, hq + 2 * hk, D).to(torch.bfloat16).to(dev)
    pos = torch.randint(0, far, (axes, T), generator=g).to(torch.int32)
    w = None if wt is None else [(1 + 0.3 * rn(D)).to(wt).to(dev) for _ in range(2)]
    return dict(q=rows[:, :hq], k=rows[:, hq:hq + hk], positions=pos.to(dev),
                inv_freq=(1e6 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().to(dev),
                q_weight=w and w[0], k_weight=w and w[1])


def _check(t, got, sections, eps=1e-6, offset=0.0, factor=1.0, **kw):
    for name in ("q", "k"):
        if t[name] is None:
            continue
        want, size = HY.rotary(f64(t[name]), f64(t["positions"]).astype(np.int64).reshape(len(sections), -1),
                               t["inv_freq"].cpu().numpy(), sections, weight=f64(t[name + "_weight"]), eps=eps, offset=offset,
                               factor=factor, **kw)
        tol = 28 * 2.0 ** -24 * size + 1e-38
        y = f64(got[name])
        assert np.array_equal(np.isnan(y), np.isnan(want))
        ok = ~np.isnan(want)
        assert np.all(np.abs(y - want)[ok] <= (tol + 2.0 ** -8 * (np.abs(want) + tol))[ok])


def _run(bfp8, t, sections=None, out=True, **kw):
    dev = t["q"].device
    got = {n: None if t[n] is None else nan_like(t[n].shape, dev) if out else t[n] for n in ("q", "k")}
    bfp8.bfp8_rotary(t["q"], t["k"], t["positions"], t["inv_freq"], got["q"] if out else None, got["k"] if out else None,
                     sections=sections, q_weight=t["q_weight"], k_weight=t["k_weight"], **kw)
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("T,hq,hk", [(1, 1, 1), (5, 3, 2), (64, 64, 8), (700, 5, 1), (3, 200, 7)])
@pytest.mark.parametrize("D,r", [(64, 64), (64, 48), (128, 128), (128, 32), (256, 64), (256, 176), (256, 256), (128, 16)])
@pytest.mark.parametrize("adjacent,wt", [(False, None), (True, torch.float32), (False, torch.bfloat16)])
def test_one_axis_matches_oracle(bfp8, cuda_device, T, hq, hk, D, r, adjacent, wt):
    t = _inputs(cuda_device, T, hq, hk, D, r, 1, T + D + r, wt)
    _check(t, _run(bfp8, t, adjacent=adjacent), [r // 2], adjacent=adjacent)


@pytest.mark.parametrize("sections", [[64], [40, 24], [24, 20, 20], [16, 16, 16, 16], [0, 64, 0], [63, 1], [1, 0, 63]], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_axes_match_oracle(bfp8, cuda_device, sections, interleaved, adjacent):
    t = _inputs(cuda_device, 37, 6, 2, 128, 128, len(sections), sum(i * s for i, s in enumerate(sections)), torch.bfloat16)
    kw = dict(interleaved=interleaved, adjacent=adjacent, factor=0.75)
    _check(t, _run(bfp8, t, sections, weight_offset=1.0, **kw), sections, offset=1.0, **kw)


def test_far_positions_keep_their_digits(bfp8, cuda_device):
    t = _inputs(cuda_device, 200, 2, 1, 128, 128, 3, 5, far=2 ** 31 - 1)
    t["positions"][:, 0], t["positions"][:, 1] = 2 ** 31 - 1, 0
    _check(t, _run(bfp8, t, [22, 21, 21]), [22, 21, 21])


def test_frequencies_of_any_size(bfp8, cuda_device):
    """Frequencies above one turn a position, negative ones, zero, subnormal ones; NaN for what has no turns."""
    dev = cuda_device
    f = [1.0, -1.0, 6.5, -1000.25, 2.0 ** 23 + 2, 3.0e9, 0.0, 1e-30, 1e-45, 0.1, 2.0 ** 22 + 0.5, 6.2831855]
    t = _inputs(dev, 50, 2, 2, 64, 32, 1, 6, far=1 << 16)
    t["inv_freq"][:len(f)] = torch.tensor(f, device=dev)
    got = _run(bfp8, t)
    _check(t, got, [16])
    t["inv_freq"][:3] = torch.tensor([float("inf"), float("nan"), 2.0 ** 32], device=dev)
    bad = torch.isnan(_run(bfp8, t)["q"])
    assert bad[..., [0, 1, 2, 16, 17, 18]].all() and bad.sum() == 50 * 2 * 6


def test_rows_of_no_request_and_in_place(bfp8, cuda_device):
    """Rows with a negative position on any axis are left as they were, apart and in place."""
    t = _inputs(cuda_device, 40, 4, 2, 128, 64, 3, 7, torch.float32)
    t["positions"][0, 30:], t["positions"][2, 5] = -1, -7
    sections = [12, 10, 10]
    got = _run(bfp8, t, sections)
    _check(t, got, sections)
    before = {n: t[n].clone() for n in ("q", "k")}
    _run(bfp8, t, sections, out=False)
    for n in ("q", "k"):
        left = torch.isnan(got[n])
        assert torch.equal(torch.where(left, before[n], got[n]), t[n])


def test_strides_and_queries_alone(bfp8, cuda_device):
    dev, T = cuda_device, 21
    t = _inputs(dev, T, 3, 1, 64, 64, 2, 8)
    t["q"] = t["q"].transpose(0, 1).contiguous().transpose(0, 1)
    t["positions"] = torch.cat([t["positions"], t["positions"]], 1)[:, 3:3 + T]
    got = _run(bfp8, t, [16, 16])
    _check(t, got, [16, 16])
    assert torch.equal(_run(bfp8, t | dict(k=None), [16, 16])["q"], got["q"])


def test_heads_with_a_nan(bfp8, cuda_device):
    t = _inputs(cuda_device, 9, 4, 2, 64, 32, 1, 9, torch.float32)
    t["q"][3, 1, 40] = float("nan")
    bad = torch.isnan(_run(bfp8, t)["q"])
    assert bad[3, 1].all() and bad.sum() == 64


def test_more_than_2_32_bytes(bfp8, cuda_device):
    dev, T, H, D = cuda_device, 300000, 64, 128
    t = _inputs(dev, 2, H, 1, D, D, 1, 10)
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
    q[-2:] = t["q"]
    pos = torch.zeros(T, dtype=torch.int32, device=dev)
    pos[-2:] = t["positions"][0]
    bfp8.bfp8_rotary(q, None, pos, t["inv_freq"])
    _check(t | dict(k=None), dict(q=q[-2:]), [D // 2])
    assert not q[:-2].any()


def test_captured_on_a_stream_of_its_own(bfp8, cuda_device):
    dev = cuda_device
    t = _inputs(dev, 20, 4, 1, 128, 128, 3, 11, torch.bfloat16)
    got = {n: nan_like(t[n].shape, dev) for n in ("q", "k")}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bfp8.bfp8_rotary(t["q"], t["k"], t["positions"], t["inv_freq"], got["q"], got["k"], sections=[24, 20, 20],
                         q_weight=t["q_weight"], k_weight=t["k_weight"])
    for seed in (12, 13):
        new = _inputs(dev, 20, 4, 1, 128, 128, 3, seed, torch.bfloat16)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        _check(t, got, [24, 20, 20])


def test_refusals(bfp8, cuda_device):
    dev = cuda_device
    t = _inputs(dev, 6, 2, 1, 128, 64, 2, 14, torch.float32)
    for kw in (dict(sections=[32]), dict(sections=[16, 8, 8])):
        with pytest.raises(ValueError):
            _run(bfp8, t, **kw)
    for bad in (dict(q=t["q"].float()), dict(positions=t["positions"].long()), dict(positions=t["positions"][:, :5]),
                dict(inv_freq=t["inv_freq"].double()), dict(q_weight=t["q_weight"][:64]),
                dict(q_weight=t["q_weight"].to(torch.bfloat16)), dict(k=t["k"][:5])):
        with pytest.raises(ValueError):
            _run(bfp8, t | bad, [16, 16])
    for sections in ([16, 15], [33, -1]):
        with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
            _run(bfp8, t, sections)
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):
        _run(bfp8, t | dict(inv_freq=t["inv_freq"][:28].contiguous()), [14, 14])
