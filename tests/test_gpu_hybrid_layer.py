"""The linear-attention example against the same layer in plain float64 arithmetic, which rounds
where the example does: the norm's and the gated heads' codes to E4M3 with 1x128 scales, and the
projections', the convolution's and the delta rule's outputs to BF16.

What is left: a BF16 value next to a border falls to either side of it. If every output of the
delta rule were one BF16 step aside (2^-8 of it at most), 2^-8 / 2^-4 = 1/16 of the codes, whose
steps are 2^-3 of a value at most, would move by one, sqrt(1/16) 2^-3 = 3.1 % in the mean square;
the state takes 2^-8 / 2 from keys and values so moved. A row, head or slot out of place costs
100 %.
"""

import subprocess
import sys
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu
EXAMPLES = Path(__file__).resolve().parent.parent / "examples"
sys.path.insert(0, str(EXAMPLES))
LIMIT, STATE_LIMIT = 0.032, 0.004


def _weight(w, members):
    q, s = w
    rows = torch.cat([s[a:b].double().repeat_interleave(128, 0)[:n] for (a, b), n in zip(_blocks(members), members)])
    return q.view(torch.float8_e4m3fn).double() * rows.repeat_interleave(128, 1)[:, : q.shape[1]]


def _blocks(members):
    at = 0
    for n in members:
        yield at, at + -(-n // 128)
        at += -(-n // 128)


def _quantized(x):
    T, n = x.shape
    g = torch.nn.functional.pad(x, (0, -n % 128)).view(T, -1, 128)
    s = (g.abs().amax(-1).clamp(min=1e-10) / 448).float().double()
    q = (g / s[..., None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).double() * s[..., None]
    return q.view(T, -1)[:, :n]


def _bf16(x):
    return x.to(torch.bfloat16).double()


def _norm(x, w):
    return x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.double()


def _plain(layer, x, past):
    """One request's new rows; `past` holds its convolution inputs and state."""
    hk, hv, T = layer.qk_heads, layer.v_heads, x.shape[0]
    x = x.double()
    y = _bf16(_quantized(_norm(x, layer.norms[0])) @ _weight(layer.w_in, layer.members).T)
    qkv, z, a, b = y.split(layer.members, 1)
    every = torch.cat([past["conv"], qkv])
    past["conv"] = every[-3:]
    c = (every.unfold(0, 4, 1) * layer.conv.double()).sum(-1)
    q, k, v = _bf16(c * torch.sigmoid(c)).view(T, -1, 128).split([hk, hk, hv], 1)
    unit = lambda t: (t / (t.square().sum(-1, keepdim=True) + 1e-6).sqrt()).repeat_interleave(hv // hk, 1)   # noqa: E731
    q, k = unit(q) / 128 ** 0.5, unit(k)
    keep = torch.exp(-layer.a_log.double().exp() * torch.nn.functional.softplus(a + layer.dt_bias.double()))
    beta, S, out = torch.sigmoid(b), past["state"], []
    for t in range(T):
        S = S * keep[t][:, None, None]
        u = beta[t][:, None] * (v[t] - torch.einsum("hvk,hk->hv", S, k[t]))
        S = S + u[:, :, None] * k[t][:, None]
        out.append(torch.einsum("hvk,hk->hv", S, q[t]))
    past["state"] = S
    o, z = _bf16(torch.stack(out)), z.view(T, hv, 128)
    y = _norm(o, layer.head_norm) * z * torch.sigmoid(z)
    mixer = _bf16(_quantized(y.reshape(T, -1)) @ _weight(layer.w_out, [layer.hidden]).T)
    return mixer, _norm(x + mixer, layer.norms[1])


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_layer_matches_plain_arithmetic(bfp8, cuda_device):
    """Prompts, single tokens, requests that sit a step out, and drafts kept by some requests and dropped by others."""
    from hybrid_layer import LinearAttentionLayer, StatePool

    torch.manual_seed(3)
    dev = cuda_device
    layer = LinearAttentionLayer(512, 2, 4, dev)
    pool = StatePool(4, 2, 4, dev)
    empty = lambda: dict(conv=torch.zeros(3, layer.channels, dtype=torch.float64, device=dev),   # noqa: E731
                         state=torch.zeros(4, 128, 128, dtype=torch.float64, device=dev))
    past = [empty() for _ in range(4)]
    for new, kept in (([37, 1, 130, 66], None), ([1, 1, 1, 1], None), ([1, 0, 2, 70], None), ([3, 3, 3, 3], [0, 2]),
                      ([1, 1, 1, 1], None)):
        x = torch.randn(sum(new), 512, device=dev).to(torch.bfloat16)
        x0 = x.clone()
        normed, mixer = layer(x, pool, pool.plan(new, draft=kept is not None))
        torch.cuda.synchronize()
        assert bfp8.bfp8_device_status() == 0
        if kept is not None:
            pool.accept(kept)
        at = 0
        for b, n in enumerate(new):
            if n == 0:
                continue
            rows, before = slice(at, at + n), dict(past[b])
            want = _plain(layer, x0[rows], past[b])
            assert _off(mixer[rows], want[0]) < LIMIT, (new, b, _off(mixer[rows], want[0]))
            assert _off(normed[rows], want[1]) < LIMIT
            if kept is not None and b not in kept:
                past[b] = before
            slot = int(pool.now[b])
            assert _off(pool.state[slot], past[b]["state"]) < STATE_LIMIT, (new, b)
            assert _off(pool.conv[slot], past[b]["conv"]) < STATE_LIMIT
            at += n


def test_example_runs(bfp8, cuda_device):
    r = subprocess.run([sys.executable, str(EXAMPLES / "hybrid_layer.py"), "--hidden", "512", "--qk-heads", "2", "--v-heads",
                        "4", "--prompts", "70,3", "--steps", "2"], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert r.stdout.count("\n") == 5 and "nan" not in r.stdout
