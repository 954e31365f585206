"""Inputs and helpers that the hybrid layers' GPU tests share."""

import numpy as np
import torch


def i32(dev, values):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def offsets(dev, lens):
    return i32(dev, np.concatenate([[0], np.cumsum(lens)]).tolist())


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def nan_like(shape, dev, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device=dev)


def delta_inputs(dev, lens, hk, hv, seed, slots=None, extra=0, decay=1.0):
    """Inputs of a ragged step of the delta rule: q, k, v as columns of one matrix of `extra` more rows
    than tokens, slots drawn apart for reading and writing (every third request begins from zeros)."""
    g = torch.Generator().manual_seed(seed)
    T, B = sum(lens) + extra, len(lens)
    n = 2 * B + 1 if slots is None else slots
    r = lambda *s: torch.randn(*s, generator=g)   # noqa: E731
    qkv = torch.nn.functional.silu(1.5 * r(T, 2 * hk + hv, 128)).to(torch.bfloat16).to(dev)
    ab = r(T, 2, hv).to(torch.bfloat16).to(dev)
    order = torch.randperm(n, generator=g).tolist()
    return dict(q=qkv[:, :hk], k=qkv[:, hk:2 * hk], v=qkv[:, 2 * hk:], a=ab[:, 0], b=ab[:, 1],
                a_log=torch.log(decay * (0.02 + 8 * torch.rand(hv, generator=g) ** 3)).to(dev),
                dt_bias=r(hv).to(dev) - 2, state=(0.3 * r(n, hv, 128, 128)).to(dev),
                slots_in=i32(dev, [-1 if b % 3 == 2 else order[b] for b in range(B)]), slots_out=i32(dev, order[B:2 * B]),
                q_offsets=offsets(dev, lens), out=nan_like((T, hv, 128), dev))
