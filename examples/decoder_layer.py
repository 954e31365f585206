"""One decoder layer served from a paged 8-bit KV cache: prompts of different
lengths in one ragged step, then a token per request and step.

    kv_plan -> residual_norm (pre-norm + 1x128 quant) -> linear_w8a8 (QKV)
    -> rotary -> kv_append -> kv_attention
    -> act_quant_group -> linear_w8a8 (output)
    -> residual_norm (post-norm, residual sum, pre-norm, quant)
    -> linear_w8a8_silu_quant (gate/up) -> linear_w8a8 (down)
    -> residual_norm (post-norm, residual sum, the next layer's pre-norm)

Weights and inputs are random. Run it as

    python examples/decoder_layer.py --prompts 949,300,17 --steps 16
"""

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parent.parent))
from block_scaled_fp8_token_gb300 import bfp8  # noqa: E402

D = 128   # head width of the cache


def fp8_weight(n, k, gen, dev):
    """A random [n, k] weight as E4M3 codes and a 128x128 scale grid."""
    w = torch.randn(n, k, generator=gen, device=dev) / k ** 0.5
    q = torch.empty(n, k, dtype=torch.uint8, device=dev)
    s = torch.empty(-(-n // 128), -(-k // 128), dtype=torch.float32, device=dev)
    bfp8.bfp8_quantize_weight_block(w, q, s)
    return q, s


class PagePool:
    """The cache of one layer, its requests' block tables and the free pages. The
    host knows every length, so no step waits for the device."""

    def __init__(self, batch, kv_heads, pages, page_size, max_tokens, dev):
        self.page_size, self.used = page_size, 0
        shape = (pages, kv_heads, page_size, D)
        self.k, self.v = (torch.empty(shape, dtype=torch.uint8, device=dev) for _ in range(2))
        self.k_exp, self.v_exp = (torch.empty(pages, kv_heads, dtype=torch.uint8, device=dev) for _ in range(2))
        self.free = torch.randperm(pages, device=dev, dtype=torch.int64).to(torch.int32)
        self.table = torch.full((batch, -(-max_tokens // page_size)), -1, dtype=torch.int32, device=dev)
        self.lengths = [0] * batch

    def plan(self, new):
        """Slots and positions of `new[b]` more tokens of each request. (The free list is passed
        from its first unused page on; a captured step would read the same address each time, and
        the list would have to be moved up to it between replays.)"""
        dev, T = self.free.device, sum(new)

        def i32(x):
            return torch.tensor(x, dtype=torch.int32, device=dev)

        s = dict(new=new, max_new=max(new), q_offsets=torch.empty(len(new) + 1, dtype=torch.int32, device=dev),
                 kv_len=torch.empty(len(new), dtype=torch.int32, device=dev),
                 slots=torch.empty(T, dtype=torch.int64, device=dev),
                 positions=torch.empty(T, dtype=torch.int32, device=dev),
                 counts=torch.empty(3, dtype=torch.int32, device=dev))
        bfp8.bfp8_kv_plan(i32(self.lengths), i32(new), self.free[self.used:], self.table, self.page_size,
                          s["q_offsets"], s["kv_len"], s["slots"], s["positions"], s["counts"])
        for b, n in enumerate(new):
            self.used += -(-(self.lengths[b] + n) // self.page_size) - -(-self.lengths[b] // self.page_size)
            self.lengths[b] += n
        if self.used > len(self.free):
            raise RuntimeError("the cache has no free pages left")
        return s


class DecoderLayer:
    def __init__(self, hidden, inter, heads, kv_heads, dev, seed=0):
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.hidden, self.inter, self.heads, self.kv_heads = hidden, inter, heads, kv_heads
        self.members = [heads * D, kv_heads * D, kv_heads * D]
        self.qkv = fp8_weight(sum(self.members), hidden, gen, dev)
        self.o = fp8_weight(hidden, heads * D, gen, dev)
        self.gate_up = fp8_weight(2 * inter, hidden, gen, dev)
        self.down = fp8_weight(hidden, inter, gen, dev)
        self.norms = [(1 + 0.1 * torch.randn(hidden, generator=gen, device=dev)).to(torch.bfloat16) for _ in range(5)]
        self.inv_freq = (1e6 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().to(dev)

    def __call__(self, x, pool, step):
        """x [T, hidden], the residual stream, is updated; returns what the next
        layer's first projection would take, and the two blocks' outputs."""
        T, dev = x.shape[0], x.device
        pre_attn, post_attn, pre_ffn, post_ffn, pre_next = self.norms

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

        # attention block
        a = codes(self.hidden)
        bfp8.bfp8_residual_norm(None, x, q=a[0], scales=a[1], w_pre=pre_attn)
        qkv = linear(a, self.qkv, sum(self.members), self.members).view(T, -1, D)
        q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
        bfp8.bfp8_rotary(q, k, step["positions"], self.inv_freq)
        cache = (pool.k, pool.v, pool.k_exp, pool.v_exp)
        bfp8.bfp8_kv_append(k, v, step["slots"], *cache)
        out = bf16(T, self.heads, D)
        n = bfp8.bfp8_kv_attention_workspace(len(step["new"]), T, step["max_new"], self.heads, self.kv_heads)
        bfp8.bfp8_kv_attention(q, *cache, pool.table, step["q_offsets"], step["kv_len"], out, step["max_new"],
                               workspace=torch.empty(n, dtype=torch.uint8, device=dev))
        o = codes(self.heads * D)
        bfp8.bfp8_act_quant_group(out.view(T, -1), *o)
        attn = linear(o, self.o, self.hidden)

        # feed-forward block
        bfp8.bfp8_residual_norm(attn, x, x, q=a[0], scales=a[1], w_post=post_attn, w_pre=pre_ffn)
        h = codes(self.inter)
        ws = torch.empty(bfp8.bfp8_linear_w8a8_silu_quant_workspace(T, self.inter, self.hidden), dtype=torch.uint8,
                         device=dev)
        bfp8.bfp8_linear_w8a8_silu_quant(*a, *self.gate_up, *h, workspace=ws)
        ffn = linear(h, self.down, self.hidden)
        normed = bf16(T, self.hidden)
        bfp8.bfp8_residual_norm(ffn, x, x, norm_out=normed, w_post=post_ffn, w_pre=pre_next)
        return normed, attn, ffn


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inter", type=int, default=17408)
    ap.add_argument("--heads", type=int, default=64)
    ap.add_argument("--kv-heads", type=int, default=8)
    ap.add_argument("--page", type=int, default=64, choices=(16, 32, 64, 128))
    ap.add_argument("--prompts", default="949,300,17", help="lengths of the requests' prompts")
    ap.add_argument("--steps", type=int, default=16, help="decode steps behind them")
    args = ap.parse_args()
    dev, prompts = torch.device("cuda"), [int(n) for n in args.prompts.split(",")]
    layer = DecoderLayer(args.hidden, args.inter, args.heads, args.kv_heads, dev)
    longest = max(prompts) + args.steps
    pages = sum(-(-(n + args.steps) // args.page) for n in prompts)
    pool = PagePool(len(prompts), args.kv_heads, pages, args.page, longest, dev)
    for i in range(args.steps + 1):
        new = prompts if i == 0 else [1] * len(prompts)
        x = torch.randn(sum(new), args.hidden, device=dev).to(torch.bfloat16)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        normed, _, _ = layer(x, pool, pool.plan(new))
        end.record()
        torch.cuda.synchronize()
        print(f"step {i}: {sum(new)} tokens, cache lengths {pool.lengths}, {begin.elapsed_time(end):.3f} ms, "
              f"output rms {normed.float().square().mean().sqrt():.4f}")
    if bfp8.bfp8_device_status() != 0:
        raise SystemExit("device status: " + bfp8.bfp8_status_string(bfp8.bfp8_device_status()))


if __name__ == "__main__":
    main()
