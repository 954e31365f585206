"""bfp8_gated_norm on the GPU against the oracle in float64.

Tolerances. The row's factor: 8 fused steps and 5 levels of a tree (13 2^-24, halved by the root), the mean, the
root and its product, 16 2^-24 with the weight's; the gate is within (6 + 1.2 max(0, -z)) 2^-23 of itself and two
more products follow:
  |y - exact| <= (36 + 2.4 max(0, -z)) 2^-24 |y|  =: tol.
BF16 adds half a step, 2^-8. A group's scale is its largest |y| / 448 within that entry's tol and two roundings; a
code lies between the codes of (y - tol) / s and (y + tol) / s, the quotient formed within 2^-22 (a reciprocal and a
product, each rounded).
"""

import numpy as np
import pytest
import torch

from hybrid_util import f64, nan_like
from oracle import formats as F
from oracle import hybrid as HY

pytestmark = pytest.mark.gpu


def _inputs(dev, T, H, D, seed, wt=torch.float32, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    x, z = (spread * r(T, H, D)).to(torch.bfloat16), (4 * r(T, H, D)).to(torch.bfloat16)
    return dict(x=x.to(dev), gate=z.to(dev), weight=None if wt is None else (1 + 0.3 * r(D)).to(wt).to(dev))


def _outputs(dev, T, H, D):
    return dict(out=nan_like((T, H, D), dev), q=torch.full((T, H * D), 0x7F, dtype=torch.uint8, device=dev),
                scales=nan_like((T, -(-H * D // 128)), dev, torch.float32))


def _check(t, o, eps=1e-6, offset=0.0, sigmoid=False):
    z = f64(t["gate"])
    y = HY.gated_norm(f64(t["x"]), z, f64(t["weight"]), eps, offset, sigmoid)
    tol = (36 + 2.4 * np.maximum(0, -z)) * 2.0 ** -24 * np.abs(y) + 1e-37
    if o.get("out") is not None:
        assert np.all(np.abs(f64(o["out"]) - y) <= tol + 2.0 ** -8 * (np.abs(y) + tol))
    if o.get("q") is None:
        return
    y, tol = y.reshape(len(y), -1), tol.reshape(len(y), -1)
    edges = np.arange(0, y.shape[1], 128)
    group = lambda v: np.maximum.reduceat(v, edges, axis=1)   # noqa: E731
    want = np.maximum(group(np.abs(y)), 1e-10) / 448
    got = f64(o["scales"])
    assert np.all(np.abs(got - want) <= group(tol) / 448 + 2.0 ** -23 * want)
    each = np.repeat(got, 128, axis=1)[:, :y.shape[1]]
    lut = F.e4m3_decode_lut()
    code, slack = lut[o["q"].cpu().numpy()], tol + 2.0 ** -22 * np.abs(y)
    assert np.all(code >= lut[F.e4m3_encode_rne_sat((y - slack) / each)])
    assert np.all(code <= lut[F.e4m3_encode_rne_sat((y + slack) / each)])


def _run(bfp8, t, o, **kw):
    bfp8.bfp8_gated_norm(t["x"], t["gate"], t["weight"], o.get("out"), q=o.get("q"), scales=o.get("scales"), **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H", [(1, 1), (3, 2), (2, 5), (64, 48), (301, 7), (1, 300), (2000, 3)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("wt,sigmoid", [(torch.float32, False), (torch.bfloat16, True), (None, True)])
def test_matches_oracle(bfp8, cuda_device, T, H, D, wt, sigmoid):
    t, o = _inputs(cuda_device, T, H, D, T + H + D, wt), _outputs(cuda_device, T, H, D)
    _run(bfp8, t, o, sigmoid=sigmoid, weight_offset=0.25)
    _check(t, o, offset=0.25, sigmoid=sigmoid)
    for name in ("out", "q"):                        # each output alone: the same bytes
        lone = _outputs(cuda_device, T, H, D)
        lone = {k: lone[k] for k in (["out"] if name == "out" else ["q", "scales"])}
        _run(bfp8, t, lone, sigmoid=sigmoid, weight_offset=0.25)
        assert all(torch.equal(lone[k], o[k]) for k in lone)


@pytest.mark.parametrize("T,H,D,wt,sigmoid", [(8000, 16, 128, torch.float32, False), (3001, 33, 64, torch.float32, False),
                                              (4000, 9, 256, torch.float32, True), (700, 40, 128, torch.float32, True)])
def test_codes_are_those_of_exact_arithmetic(bfp8, cuda_device, T, H, D, wt, sigmoid):
    """Where FP32's last bits would decide a code, sums of two floats do: entries within 2^-32, so a quotient within
    2^-31 of the exact one. (One code in a million differs without. Below 2^-6 codes stay as FP32 has them.)"""
    t, o = _inputs(cuda_device, T, H, D, 31 * T + D, wt), _outputs(cuda_device, T, H, D)
    _run(bfp8, t, o, sigmoid=sigmoid, weight_offset=0.125)
    y = HY.gated_norm(f64(t["x"]), f64(t["gate"]), f64(t["weight"]), 1e-6, 0.125, sigmoid).reshape(T, -1)
    largest = np.maximum.reduceat(np.abs(y), np.arange(0, y.shape[1], 128), axis=1)
    v = y / np.repeat(largest / 448, 128, axis=1)[:, :y.shape[1]]
    lut = F.e4m3_decode_lut()
    code, plain = lut[o["q"].cpu().numpy()], np.abs(v) > 2.0 ** -6 * 1.01
    assert np.all((code >= lut[F.e4m3_encode_rne_sat(v - 2.0 ** -31 * np.abs(v))])[plain])
    assert np.all((code <= lut[F.e4m3_encode_rne_sat(v + 2.0 ** -31 * np.abs(v))])[plain])
    for name in ("x", "gate"):                       # the same codes where the row is overwritten by the output
        held, again = t[name].clone(), _outputs(cuda_device, T, H, D)
        _run(bfp8, t, dict(again, out=t[name]), sigmoid=sigmoid, weight_offset=0.125)
        assert all(torch.equal(again[k], o[k]) for k in ("q", "scales")) and torch.equal(t[name], o["out"])
        t[name].copy_(held)


def test_strides_scales_of_either_order_and_in_place(bfp8, cuda_device):
    dev, T, H, D = cuda_device, 33, 6, 128
    t, o = _inputs(dev, T, H, D, 1), _outputs(dev, T, H, D)
    wide = torch.randn(T, H, 2 * D + 8, device=dev).to(torch.bfloat16)
    wide[..., :D], wide[..., D + 8:] = t["x"], t["gate"]
    t["x"], t["gate"] = wide[..., :D], wide[..., D + 8:]
    o["scales"] = nan_like((H, T), dev, torch.float32).t()
    o["out"] = nan_like((H, T, D), dev).transpose(0, 1)
    o["q"] = torch.zeros(T, H * D + 24, dtype=torch.uint8, device=dev)[:, :H * D]
    _run(bfp8, t, o)
    _check(t, o)
    want, before = o["out"].clone(), dict(t, x=t["x"].clone(), gate=t["gate"].clone())
    _run(bfp8, t, dict(out=t["gate"]))               # over the gate
    assert torch.equal(t["gate"], want) and torch.equal(t["x"], before["x"])
    t["gate"].copy_(before["gate"])
    _run(bfp8, t, dict(out=t["x"]))                  # over the input
    assert torch.equal(t["x"], want)


@pytest.mark.parametrize("spread", [0.0, 1e-30, 1e18])
def test_rows_of_nothing_and_of_any_size(bfp8, cuda_device, spread):
    """Rows of zeros (codes 0, the scale's floor), tiny ones that eps outweighs, and squares near the type's end."""
    t, o = _inputs(cuda_device, 9, 3, 128, 2, spread=spread), _outputs(cuda_device, 9, 3, 128)
    _run(bfp8, t, o)
    _check(t, o)
    if spread == 0.0:
        assert not (o["q"] & 0x7F).any() and (o["scales"] == np.float32(1e-10) / np.float32(448)).all()


def test_gates_at_their_ends(bfp8, cuda_device):
    t, o = _inputs(cuda_device, 4, 2, 64, 3), _outputs(cuda_device, 4, 2, 64)
    t["gate"][0], t["gate"][1], t["gate"][2] = -87.0, 200.0, -1000.0
    _run(bfp8, t, o)
    assert torch.isfinite(o["out"]).all() and not o["out"][2].any()
    t = {k: v[[0, 1, 3]] if k != "weight" else v for k, v in t.items()}
    _check(t, {k: v[[0, 1, 3]] for k, v in o.items()})


def test_nan_stays_in_its_head(bfp8, cuda_device):
    t, o = _inputs(cuda_device, 5, 4, 64, 4), _outputs(cuda_device, 5, 4, 64)
    t["x"][2, 1, 7] = float("nan")
    _run(bfp8, t, o)
    bad = torch.isnan(o["out"])
    assert bad[2, 1].all() and bad.sum() == 64
    assert ((o["q"][2, 64:128] & 0x7F) == 0x7F).all() and ((o["q"] & 0x7F) == 0x7F).sum() == 64


def test_more_than_2_32_bytes(bfp8, cuda_device):
    dev, T, H, D = cuda_device, 300000, 64, 128
    x = torch.zeros(T, H, D, dtype=torch.bfloat16, device=dev)
    t = _inputs(dev, 2, H, D, 5)
    x[-2:] = t["x"]
    gate = torch.ones_like(x)
    gate[-2:] = t["gate"]
    out = torch.empty_like(x)
    _run(bfp8, dict(x=x, gate=gate, weight=t["weight"]), dict(out=out))
    _check(t, dict(out=out[-2:]))
    assert not out[:-2].any()


def test_captured_on_a_stream_of_its_own(bfp8, cuda_device):
    dev = cuda_device
    t, o = _inputs(dev, 20, 4, 128, 6), _outputs(dev, 20, 4, 128)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bfp8.bfp8_gated_norm(t["x"], t["gate"], t["weight"], o["out"], q=o["q"], scales=o["scales"])
    for seed in (7, 8):
        new = _inputs(dev, 20, 4, 128, seed)
        for k in t:
            t[k].copy_(new[k])
        graph.replay()
        torch.cuda.synchronize()
        _check(t, o)


def test_refusals(bfp8, cuda_device):
    dev = cuda_device
    t, o = _inputs(dev, 6, 2, 128, 9), _outputs(dev, 6, 2, 128)
    for bad in (dict(x=t["x"].float()), dict(gate=t["gate"][:, :1]), dict(weight=t["weight"][:64]), dict(weight=t["weight"].cpu())):
        with pytest.raises(ValueError):
            _run(bfp8, t | bad, o)
    for bad in (dict(out=o["out"][:5]), dict(q=o["q"][:, :128]), dict(scales=o["scales"][:, :1]), dict(scales=None),
                dict(scales=o["scales"].double()), dict(q=o["q"].float())):
        with pytest.raises(ValueError):
            _run(bfp8, t, o | bad)
    with pytest.raises(bfp8.Bfp8Error, match="SCALE_DTYPE"):
        _run(bfp8, t | dict(weight=t["weight"].half()), o)
    with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
        _run(bfp8, t, {})
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):
        _run(bfp8, {k: v[..., :96].contiguous() for k, v in t.items()}, dict(out=o["out"][..., :96].contiguous()))
