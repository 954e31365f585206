"""The decoder-layer example against the same layer in plain float64 arithmetic.

What the example rounds and the plain layer does not: the projections' inputs
(two by residual_norm, the attention's output, silu(gate) * up) and the cache's
keys and values to E4M3, whose relative rounding error is 2^-4 at most and
2^-4 / sqrt(3) = 3.6 % in the mean square; BF16 outputs, 2^-9, are lost in that.
A block's output passes through at most four such roundings (codes, keys,
values, attention output), each a sum over many terms that keeps the relative
size of its error: sqrt(4) * 3.6 % = 7.2 % in the mean square. The first block's
error also enters the second through the residual sum. Twice 7.2 % is allowed;
a row, head, page or position out of place costs 100 %.
"""

import sys
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, str(Path(__file__).resolve().parent.parent / "examples"))
LIMIT = 0.145


def _dequantize(w):
    q, s = w
    grid = s.double().repeat_interleave(128, 0).repeat_interleave(128, 1)[: q.shape[0], : q.shape[1]]
    return q.view(torch.float8_e4m3fn).double() * grid


def _norm(x, w):
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()


def _rotate(x, pos):
    f = pos.double()[:, None] * 1e6 ** (-torch.arange(0, 128, 2, device=x.device).double() / 128)
    cos, sin = f.cos()[:, None], f.sin()[:, None]
    a, b = x[..., :64], x[..., 64:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _plain(layer, x, pos, past):
    """One request's new rows; `past` holds its earlier keys and values."""
    T, H, G = x.shape[0], layer.kv_heads, layer.heads // layer.kv_heads
    x = x.double()
    y = (_norm(x, layer.norms[0]) @ _dequantize(layer.qkv).T).view(T, -1, 128)
    q, k, v = y.split([layer.heads, H, H], 1)
    past.append((_rotate(k, pos), v))
    k, v = (torch.cat([p[i] for p in past]).repeat_interleave(G, 1) for i in range(2))
    s = torch.einsum("thd,shd->hts", _rotate(q, pos), k) / 128 ** 0.5
    s = s.masked_fill(torch.arange(len(k), device=x.device) > pos[:, None], float("-inf"))
    attn = torch.einsum("hts,shd->thd", s.softmax(-1), v).reshape(T, -1) @ _dequantize(layer.o).T
    x = x + _norm(attn, layer.norms[1])
    g, u = (_norm(x, layer.norms[2]) @ _dequantize(layer.gate_up).T).chunk(2, -1)
    ffn = (torch.nn.functional.silu(g) * u) @ _dequantize(layer.down).T
    return attn, ffn, x + _norm(ffn, layer.norms[3])


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


@pytest.mark.parametrize("page", [16, 128])
def test_layer_matches_plain_arithmetic(bfp8, cuda_device, page):
    from decoder_layer import DecoderLayer, PagePool

    torch.manual_seed(page)
    prompts, steps = [37, 1, 130], 3
    layer = DecoderLayer(512, 768, 8, 2, cuda_device)
    pool = PagePool(len(prompts), 2, 64, page, 160, cuda_device)
    past, done = [[] for _ in prompts], [0] * len(prompts)
    for i in range(1 + steps):
        new = prompts if i == 0 else [1, 2 * (i % 2), 1]        # a request may sit a step out
        x = torch.randn(sum(new), 512, device=cuda_device).to(torch.bfloat16)
        x0 = x.clone()
        step = pool.plan(new)
        normed, attn, ffn = layer(x, pool, step)
        torch.cuda.synchronize()
        assert bfp8.bfp8_device_status() == 0
        assert step["counts"][1:].tolist() == [0, 0]
        at = 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            pos = torch.arange(done[b], done[b] + n, device=cuda_device)
            rows = slice(at, at + n)
            want = _plain(layer, x0[rows], pos, past[b])
            assert torch.equal(step["positions"][rows].long(), pos)
            for name, got, ref in zip(("attention", "feed-forward", "residual"),
                                      (attn[rows], ffn[rows], x[rows]), want):
                assert _off(got, ref) < LIMIT, (name, i, b, _off(got, ref))
            assert _off(normed[rows], _norm(want[2], layer.norms[4])) < LIMIT
            done[b] += n
            at += n
