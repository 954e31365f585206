"""bfp8_residual_norm on the GPU against the oracle in float64.

Tolerances. A row's float32 error: the sum of H <= 16384 squares is formed as
32 fused steps a thread and 10 levels of a tree, so it is within 42 * 2^-24;
halved by the square root, plus the mean's division, the root and the
reciprocal, the row's factor is within 24 * 2^-24. u takes three more
roundings, the residual's product one, their sum one:
  |h - exact| <= 28 * 2^-24 (|a res| + |gate u|)  <  2^-19 (|a res| + |gate u|).
n repeats the factor and adds h's error through it (its effect on the row's
factor is below the largest relative error of h's terms once more):
  |n - exact| <= 2^-18 (|n| + (|a res| + |gate u|) * factor * |w|)  =: tol_n.
BF16 results add half a step, 2^-8 relative (8 significant bits); a group's
scale is the group's largest |n| / 448 within the group's largest tol_n and
one rounding; a code lies between the codes of (n - tol) / s and (n + tol) / s.
"""

import numpy as np
import pytest
import torch

from oracle import formats as F
from oracle import kv as KV

pytestmark = pytest.mark.gpu


def _inputs(dev, T, H, gate, wt, seed, post=True, y=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    res = r(T, H)
    res[:, ::max(1, H // 7)] *= 40.0
    t = dict(res=res.to(torch.bfloat16), y=(0.5 * r(T, H)).to(torch.bfloat16) if y else None,
             w_post=(1 + 0.3 * r(H)).to(wt) if post else None, w_pre=(1 + 0.3 * r(H)).to(wt), gate=None)
    if gate:
        t["gate"] = torch.sigmoid(r(*((H,) if gate == "channel" else (T, H)))).to(torch.bfloat16)
    return {k: None if v is None else v.to(dev) for k, v in t.items()}


def _np(t):
    return None if t is None else t.double().cpu().numpy()


def _check(t, out, scale=0.75, eps=1e-6, offset=0.0):
    res_out, norm_out, q, s = out
    y, res, wp, wn, gate = (_np(t[k]) for k in ("y", "res", "w_post", "w_pre", "gate"))
    h, n = KV.residual_norm(y, res, wp, wn, gate, scale, eps, offset)
    size = np.abs(scale * res) + (np.abs(h - scale * res) if y is not None else 0)
    if res_out is not None:
        tol = 2.0 ** -8 * np.abs(h) + 2.0 ** -18 * size
        assert np.all(np.abs(_np(res_out) - h) <= tol)
    factor = 1 / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps)
    tol = 2.0 ** -18 * (np.abs(n) + size * factor * np.abs(wn + offset))
    if norm_out is not None:
        assert np.all(np.abs(_np(norm_out) - n) <= tol + 2.0 ** -8 * (np.abs(n) + tol))
    if q is not None:
        edges = np.arange(0, n.shape[1], 128)
        group = lambda x: np.maximum.reduceat(x, edges, axis=1)   # noqa: E731
        want = np.maximum(group(np.abs(n)), 1e-10) / 448
        got = _np(s)
        assert np.all(np.abs(got - want) <= group(tol) / 448 + 2.0 ** -23 * want)
        each = np.repeat(got, 128, axis=1)[:, :n.shape[1]]
        lut = F.e4m3_decode_lut()
        code = lut[q.cpu().numpy()]
        slack = tol + 2.0 ** -22 * np.abs(n)
        assert np.all(code >= lut[F.e4m3_encode_rne_sat((n - slack) / each)])
        assert np.all(code <= lut[F.e4m3_encode_rne_sat((n + slack) / each)])


def _outputs(dev, T, H):
    return [torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev),
            torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=dev),
            torch.full((T, H), 0x7F, dtype=torch.uint8, device=dev),
            torch.full((T, -(-H // 128)), float("nan"), dtype=torch.float32, device=dev)]


def _run(bfp8, t, out, **kw):
    bfp8.bfp8_residual_norm(t["y"], t["res"], out[0], norm_out=out[1], q=out[2], scales=out[3],
                            w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], **kw)
    torch.cuda.synchronize()


@pytest.mark.parametrize("T,H", [(1, 1), (3, 7), (2, 128), (5, 129), (17, 1000), (300, 2048), (16, 5120), (301, 5120),
                                 (4, 8192), (3, 8193), (2, 16384), (200, 2072), (700, 96)])
@pytest.mark.parametrize("gate,wt", [(None, torch.bfloat16), ("channel", torch.float32), ("token", torch.bfloat16)])
def test_matches_oracle(bfp8, cuda_device, T, H, gate, wt):
    t = _inputs(cuda_device, T, H, gate, wt, T * H)
    out = _outputs(cuda_device, T, H)
    _run(bfp8, t, out, residual_scale=0.75)
    _check(t, out)


@pytest.mark.parametrize("post,y", [(False, True), (False, False)])
def test_without_post_norm_and_without_a_block(bfp8, cuda_device, post, y):
    t = _inputs(cuda_device, 9, 640, "channel" if y else None, torch.bfloat16, 3, post, y)
    out = _outputs(cuda_device, 9, 640)
    _run(bfp8, t, out, residual_scale=1.0, eps=1e-5)
    _check(t, out, 1.0, 1e-5)


def test_each_output_alone(bfp8, cuda_device):
    t = _inputs(cuda_device, 12, 1536, None, torch.float32, 4)
    full = _outputs(cuda_device, 12, 1536)
    _run(bfp8, t, full, weight_offset=1.0)
    _check(t, full, 1.0, offset=1.0)
    for keep in ([0], [1], [2, 3]):
        part = _outputs(cuda_device, 12, 1536)
        _run(bfp8, t, [o if i in keep else None for i, o in enumerate(part)], weight_offset=1.0)
        for i in keep:
            assert torch.equal(part[i], full[i])


def test_in_place_and_strided(bfp8, cuda_device):
    """The residual updated in place inside a wider buffer, y's memory reused for
    the norm, token-contiguous scales, rows of a wider code buffer."""
    dev, T, H = cuda_device, 21, 640
    t = _inputs(dev, T, H, "token", torch.bfloat16, 5)
    want = _outputs(dev, T, H)
    _run(bfp8, t, want, residual_scale=0.5)
    wide = torch.zeros(T, H + 24, dtype=torch.bfloat16, device=dev)
    wide[:, 8:8 + H] = t["res"]
    odd = torch.zeros(T, H + 3, dtype=torch.bfloat16, device=dev)     # rows at odd addresses
    odd[:, 1:1 + H] = t["y"]
    q, s = torch.zeros(T, H + 5, dtype=torch.uint8, device=dev), torch.zeros(5, T, device=dev)
    res, y = wide[:, 8:8 + H], odd[:, 1:1 + H]
    bfp8.bfp8_residual_norm(y, res, res, norm_out=y, q=q[:, 2:2 + H], scales=s, s_stride_m=1, s_stride_kb=T,
                            w_post=t["w_post"], w_pre=t["w_pre"], gate=t["gate"], residual_scale=0.5)
    torch.cuda.synchronize()
    for got, w in ((res, want[0]), (y, want[1]), (q[:, 2:2 + H], want[2]), (s.t(), want[3])):
        assert torch.equal(got, w)
    assert bool((wide[:, :8] == 0).all()) and bool((wide[:, 8 + H:] == 0).all())
    assert bool((q[:, :2] == 0).all()) and bool((q[:, 2 + H:] == 0).all())


def test_zero_rows_and_empty(bfp8, cuda_device):
    t = _inputs(cuda_device, 4, 256, None, torch.bfloat16, 6)
    t["res"][1] = 0
    t["y"][1] = 0
    out = _outputs(cuda_device, 4, 256)
    _run(bfp8, t, out, residual_scale=0.75)
    _check(t, out)
    assert bool((out[2][1] == 0).all()) and bool((out[0][1] == 0).all())
    bfp8.bfp8_residual_norm(t["y"][:0], t["res"][:0], out[0][:0], w_post=t["w_post"])


def test_refusals(bfp8, cuda_device):
    dev = cuda_device
    t = _inputs(dev, 4, 256, None, torch.bfloat16, 7)
    out = _outputs(dev, 4, 256)
    call = bfp8.bfp8_residual_norm
    with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
        call(t["y"], t["res"])                                         # no output
    with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
        call(t["y"], t["res"], norm_out=out[1])                        # no w_pre
    with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
        call(None, t["res"], out[0], w_post=t["w_post"])               # a post-norm of nothing
    with pytest.raises(bfp8.Bfp8Error, match="INVALID_ARG"):
        call(t["y"], t["res"], out[0], eps=-1.0)
    with pytest.raises(bfp8.Bfp8Error, match="SCALE_DTYPE"):
        call(t["y"], t["res"], out[0], w_post=t["w_post"].half())
    with pytest.raises(ValueError, match="scales"):
        call(t["y"], t["res"], q=out[2], w_pre=t["w_pre"])
    with pytest.raises(ValueError, match="shape"):
        call(t["y"][:3], t["res"], out[0])
    with pytest.raises(ValueError, match="same dtype"):
        call(t["y"], t["res"], out[0], w_post=t["w_post"], w_pre=t["w_pre"].float())
    with pytest.raises(ValueError, match="too small"):
        call(t["y"], t["res"], out[0][:3])
    wide = torch.zeros(2, 16392, dtype=torch.bfloat16, device=dev)
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):
        call(None, wide, torch.empty_like(wide))
