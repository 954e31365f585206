"""One linear-attention layer of a hybrid decoder, served with a pool of states: prompts of
different lengths in one ragged step, then a token per request and step, and at the end a step
of drafted tokens of which only some are kept.

    residual_norm (pre-norm + 1x128 quant) -> linear_w8a8 (queries, keys, values, gate, a, b)
    -> causal_conv -> delta_rule -> gated_norm (+ 1x128 quant) -> linear_w8a8 (output)
    -> residual_norm (residual sum, the next block's pre-norm)

(The decoder's full-attention layers are those of decoder_layer.py.) Weights and inputs are
random. Run it as

    python examples/hybrid_layer.py --prompts 949,300,17 --steps 16
"""

import argparse
import sys
from pathlib import Path

import torch

sys.path[:0] = [str(Path(__file__).resolve().parent), str(Path(__file__).resolve().parent.parent)]
from block_scaled_fp8_token_gb300 import bfp8  # noqa: E402
from decoder_layer import fp8_weight  # noqa: E402

D, WIDTH = 128, 4   # of a head, and of the convolution


class StatePool:
    """What each request keeps between steps: two slots, one with its present state and one that a
    step may write without giving that up."""

    def __init__(self, batch, qk_heads, v_heads, dev):
        channels = (2 * qk_heads + v_heads) * D
        self.conv = torch.zeros(2 * batch, WIDTH - 1, channels, dtype=torch.bfloat16, device=dev)
        self.state = torch.zeros(2 * batch, v_heads, D, D, dtype=torch.float32, device=dev)
        self.now = torch.arange(batch, dtype=torch.int32, device=dev)
        self.begun = torch.zeros(batch, dtype=torch.bool, device=dev)

    def plan(self, new, draft=False):
        """Offsets and slots of new[b] more tokens of each request; of a draft the states go to the
        other slots, and count only once accept() says so."""
        dev, batch = self.now.device, len(self.now)
        q_offsets = torch.zeros(batch + 1, dtype=torch.int32, device=dev)
        q_offsets[1:] = torch.tensor(new, device=dev).cumsum(0)
        slots_in = torch.where(self.begun, self.now, -1)
        slots_out = (self.now + batch) % (2 * batch) if draft else self.now.clone()
        if not draft:
            self.begun |= torch.tensor(new, device=dev) > 0
        return dict(new=new, q_offsets=q_offsets, slots_in=slots_in, slots_out=slots_out)

    def accept(self, requests):
        """The last draft's states become these requests' own."""
        at = torch.tensor(requests, device=self.now.device)
        self.now[at] = (self.now[at] + len(self.now)) % (2 * len(self.now))


class LinearAttentionLayer:
    def __init__(self, hidden, qk_heads, v_heads, dev, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)

        def randn(*shape):
            return torch.randn(*shape, generator=gen, device=dev)

        self.hidden, self.qk_heads, self.v_heads = hidden, qk_heads, v_heads
        self.channels = (2 * qk_heads + v_heads) * D
        # queries, keys, values | output gate | a | b, each a member with scale blocks of its own
        self.members = [self.channels, v_heads * D, v_heads, v_heads]
        parts = [fp8_weight(n, hidden, gen, dev) for n in self.members]
        self.w_in = tuple(torch.cat(t) for t in zip(*parts))
        self.w_out = fp8_weight(hidden, v_heads * D, gen, dev)
        self.conv = (randn(self.channels, WIDTH) / WIDTH ** 0.5).to(torch.bfloat16)
        self.a_log = torch.log(1 + 15 * torch.rand(v_heads, generator=gen, device=dev))
        self.dt_bias = randn(v_heads) - 4
        self.norms = [(1 + 0.1 * randn(hidden)).to(torch.bfloat16) for _ in range(2)]
        self.head_norm = 1 + 0.1 * randn(D)

    def __call__(self, x, pool, step):
        """x [T, hidden], the residual stream, is updated; returns what the next block's first
        projection would take, and this block's output."""
        T, dev, hv = x.shape[0], x.device, self.v_heads

        def bf16(*shape):
            return torch.empty(shape, dtype=torch.bfloat16, device=dev)

        def codes(n):
            return (torch.empty(T, n, dtype=torch.uint8, device=dev),
                    torch.empty(T, -(-n // 128), dtype=torch.float32, device=dev))

        def linear(a, w, n, members=None):
            y = bf16(T, n)
            ws = torch.empty(bfp8.bfp8_linear_w8a8_workspace(T, n, a[0].shape[1], members), dtype=torch.uint8, device=dev)
            bfp8.bfp8_linear_w8a8(*a, *w, y, member_rows=members, workspace=ws)
            return y

        a = codes(self.hidden)
        bfp8.bfp8_residual_norm(None, x, q=a[0], scales=a[1], w_pre=self.norms[0])
        qkv, z, a_in, b_in = linear(a, self.w_in, sum(self.members), self.members).split(self.members, 1)
        slots = (step["slots_in"], step["slots_out"])
        mixed = bf16(T, self.channels)
        bfp8.bfp8_causal_conv(qkv, self.conv, mixed, step["q_offsets"], pool.conv, *slots)
        q, k, v = mixed.view(T, -1, D).split([self.qk_heads, self.qk_heads, hv], 1)
        o = bf16(T, hv, D)
        most = max(step["new"])
        ws = torch.empty(bfp8.bfp8_delta_rule_workspace(len(step["new"]), T, most, self.qk_heads, hv), dtype=torch.uint8,
                         device=dev)
        bfp8.bfp8_delta_rule(q, k, v, a_in, b_in, self.a_log, self.dt_bias, pool.state, *slots, step["q_offsets"], o, most,
                             workspace=ws)
        y = codes(hv * D)
        bfp8.bfp8_gated_norm(o, z.view(T, hv, D), self.head_norm, q=y[0], scales=y[1])
        mixer = linear(y, self.w_out, self.hidden)
        normed = bf16(T, self.hidden)
        bfp8.bfp8_residual_norm(mixer, x, x, norm_out=normed, w_pre=self.norms[1])
        return normed, mixer


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--qk-heads", type=int, default=16)
    ap.add_argument("--v-heads", type=int, default=48)
    ap.add_argument("--prompts", default="949,300,17", help="lengths of the requests' prompts")
    ap.add_argument("--steps", type=int, default=16, help="decode steps behind them")
    args = ap.parse_args()
    dev, prompts = torch.device("cuda"), [int(n) for n in args.prompts.split(",")]
    layer = LinearAttentionLayer(args.hidden, args.qk_heads, args.v_heads, dev)
    pool = StatePool(len(prompts), args.qk_heads, args.v_heads, dev)

    def run(name, new, draft=False):
        x = torch.randn(sum(new), args.hidden, device=dev).to(torch.bfloat16)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        normed, _ = layer(x, pool, pool.plan(new, draft))
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {sum(new)} tokens, {begin.elapsed_time(end):.3f} ms, output rms "
              f"{normed.float().square().mean().sqrt():.4f}")

    run("prompts", prompts)
    for i in range(args.steps):
        run(f"step {i}", [1] * len(prompts))
    run("draft of 4", [4] * len(prompts), draft=True)
    pool.accept([0])   # the other requests' drafts are dropped: their states are what they were
    run("after it", [1] * len(prompts))
    status = bfp8.bfp8_device_status()
    if status != 0:
        raise SystemExit("device status: " + bfp8.bfp8_status_string(status))


if __name__ == "__main__":
    main()
