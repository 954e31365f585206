"""bfp8_kv_attention on the GPU against the oracle in float64.

Tolerance. The inputs are exact on both sides (codes, powers of two, BF16
queries). The kernels carry a query and a weight as 8 significant bits or more:
  * a score's error comes from entries of q below 2^-10 of the row's largest
    (carried to 2^-18 of it) and FP32 sums: with |k| <= 448 * 2^ek and D = 128,
    |dx| <= 128 * 2^-18 |q|max |k|max scale in the worst case;
  * a weight is rounded to 2^-9 of itself or, far below the maximum, to 2^-14
    of the largest; the weights' rounding errors are independent, so with
    weights w_i summing to 1 and values v_i the output's error has the standard
    deviation 2^-9 / sqrt(3) * sqrt(sum w_i^2 v_i^2) or less; six of those, and
    BF16's half step 2^-8 of the output, bound an element.
The second term is what `_bound` computes; 2^-14 * sum w_i |v_i| covers the
absolute part. lse has FP32's error: 2^-18 (1 + |lse|) covers the sums of up to
2^15 terms and the approximate exponential (2^-22 each) with the score's.
"""

import numpy as np
import pytest
import torch

from gpu_util import bits16
from oracle import kv as KV

pytestmark = pytest.mark.gpu

D = 128


def _setup(dev, rng, lengths, H, G, page, order="heads", spread=2, extra=3, q_gain=1.0):
    """A cache holding requests of (kv length, new rows); NaN codes wherever nothing was written."""
    used = [max(0, -(-kv // page)) for kv, _ in lengths]
    P = sum(used) + extra
    perm = rng.permutation(P)
    table = np.full((len(lengths), max(1, max(used) + 2)), -1, np.int64)
    table[:, -1] = 2 ** 31 - 1                     # never looked at
    caches, deq = [], []
    exps = [rng.integers(120 - spread, 121 + spread, (P, H)).astype(np.uint8) for _ in range(2)]
    codes = [np.full((P, H, page, D), 0x7F, np.uint8) for _ in range(2)]
    at = 0
    for b, (kv, _) in enumerate(lengths):
        table[b, :used[b]] = perm[at:at + used[b]]
        at += used[b]
        for j in range(used[b]):
            n = min(page, kv - j * page)
            for c in codes:
                x = torch.from_numpy(rng.normal(0, 85, (H, n, D))).clamp(-448, 448)
                c[table[b, j], :, :n] = x.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    for c, e in zip(codes, exps):
        deq.append(KV.dequantize(c, e))
        t = torch.from_numpy(c).to(dev)
        if order == "tokens":
            t = t.transpose(1, 2).contiguous().transpose(1, 2)
        caches.append((t, torch.from_numpy(e).to(dev)))
    T = sum(n for _, n in lengths)
    q = torch.from_numpy((rng.normal(size=(T, H * G, D)) * q_gain).astype(np.float32)).to(torch.bfloat16)
    off = np.concatenate([[0], np.cumsum([n for _, n in lengths])])
    i32 = lambda v: torch.tensor(np.asarray(v), dtype=torch.int32, device=dev)   # noqa: E731
    return dict(q=q.to(dev), k=caches[0], v=caches[1], table=i32(table), off=i32(off), kv=i32([kv for kv, _ in lengths]),
                deq=deq, lengths=lengths, T=T, H=H, G=G, maxq=max([n for _, n in lengths] + [1]))


def _run(bfp8, s, window=-1, scale=None, out=None, lse=True, ws=None, fill=0xAB):
    dev = s["q"].device
    out = torch.full(s["q"].shape, float("nan"), dtype=torch.bfloat16, device=dev) if out is None else out
    lse = torch.full(s["q"].shape[:2], float("nan"), dtype=torch.float32, device=dev) if lse else None
    if ws is None:
        n = bfp8.bfp8_kv_attention_workspace(len(s["lengths"]), s["T"], s["maxq"], s["H"] * s["G"], s["H"])
        ws = torch.full((n,), fill, dtype=torch.uint8, device=dev)     # contents are free
    bfp8.bfp8_kv_attention(s["q"], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["off"], s["kv"], out,
                           s["maxq"], softmax_scale=scale, window=window, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert bfp8.bfp8_device_status() == 0
    return out, lse


def _check(bfp8, s, window=-1, scale=None, rows=None, got=None):
    """Compares with the oracle; rows: only these (all by default)."""
    out, lse = got or _run(bfp8, s, window, scale)
    out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
    scale = D ** -0.5 if scale is None else scale
    q = s["q"].double().cpu().numpy()
    table, (kd, vd) = s["table"].cpu().numpy(), s["deq"]
    P, H, page, _ = kd.shape
    off = s["off"].cpu().numpy()
    for b, (kv, n) in enumerate(s["lengths"]):
        pages = table[b, :max(0, -(-kv // page))].astype(np.int64)
        there = (pages >= 0) & (pages < P)
        safe = np.where(there, pages, 0)
        hide = np.repeat(~there, page)[:max(kv, 0)]
        for h in range(H):
            k = kd[safe, h].reshape(-1, D)[:max(kv, 0)]
            v = np.nan_to_num(vd[safe, h].reshape(-1, D)[:max(kv, 0)])
            k = np.nan_to_num(k)
            for t in range(off[b], off[b + 1]):
                if rows is not None and t not in rows:
                    continue
                heads = slice(h * s["G"], (h + 1) * s["G"])
                pos = kv - n + t - off[b]
                place = np.arange(max(kv, 0))
                see = ~hide & (place <= pos)
                if window >= 0:
                    see &= place >= pos - window
                if not see.any():
                    assert np.all(out[t, heads] == 0) and np.all(np.isneginf(lse[t, heads])), (b, h, t)
                    continue
                z = q[t, heads] @ k[see].T * scale
                m = z.max(1, keepdims=True)
                w = np.exp(z - m)
                total = w.sum(1, keepdims=True)
                w /= total
                want = w @ v[see]
                bound = (2.0 ** -8 * np.abs(want) + 6 * 2.0 ** -9 / 3 ** 0.5 * np.sqrt(w ** 2 @ v[see] ** 2)
                         + 2.0 ** -14 * (w @ np.abs(v[see])))
                err = np.abs(out[t, heads] - want)
                assert np.all(err <= bound), (b, h, t, float((err / bound).max()))
                want_lse = (m + np.log(total))[:, 0]
                assert np.all(np.abs(lse[t, heads] - want_lse) <= 2.0 ** -18 * (1 + np.abs(want_lse))), (b, h, t)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 8), (3, 5), (1, 40), (8, 1)])
def test_decode_matches_oracle(bfp8, cuda_device, page, H, G):
    """One new token a request, lengths of one token to several pages, odd ones among them."""
    rng = np.random.default_rng(page * 100 + H * 10 + G)
    lengths = [(n, 1) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700)]
    _check(bfp8, _setup(cuda_device, rng, lengths, H, G, page))


@pytest.mark.parametrize("page,order", [(16, "tokens"), (64, "heads"), (128, "tokens")])
@pytest.mark.parametrize("window", [-1, 0, 1, 37, 100])
def test_drafts_and_windows(bfp8, cuda_device, page, order, window):
    """A few new tokens a request, and requests whose new tokens are all they have."""
    rng = np.random.default_rng(page + window)
    lengths = [(3, 3), (100, 2), (257, 4), (1, 1), (64, 5), (65, 3), (300, 7), (40, 1)]
    _check(bfp8, _setup(cuda_device, rng, lengths, 2, 4, page, order), window)


@pytest.mark.parametrize("page,G,H,window", [(16, 8, 2, -1), (32, 1, 2, -1), (64, 5, 1, -1), (128, 8, 1, 200), (64, 2, 2, 0),
                                             (16, 3, 1, 77)])
def test_prompts_match_oracle(bfp8, cuda_device, page, G, H, window):
    """Prompts and chunks behind cached tokens, next to single tokens and drafts."""
    rng = np.random.default_rng(page * G)
    lengths = [(300, 300), (1, 1), (130, 2), (517, 129), (128, 128), (640, 33), (255, 255), (90, 64), (700, 1)]
    s = _setup(cuda_device, rng, lengths, H, G, page)
    rows = None
    if s["T"] * H * G > 4000:
        rows = set(rng.choice(s["T"], 500, replace=False).tolist()) | {0, 1, 299, 300, s["T"] - 1}
    _check(bfp8, s, window, rows=rows)


def test_long_prompt(bfp8, cuda_device):
    rng = np.random.default_rng(21)
    s = _setup(cuda_device, rng, [(2309, 1500), (1111, 1111)], 2, 8, 64)
    _check(bfp8, s, rows=set(rng.choice(s["T"], 150, replace=False).tolist()) | {0, 1499, 1500, s["T"] - 1})


def test_long_cache(bfp8, cuda_device):
    """One request split over every SM, next to short ones; and few rows against a long cache."""
    rng = np.random.default_rng(22)
    s = _setup(cuda_device, rng, [(9, 1), (33333, 1), (130, 1)], 1, 8, 64)
    _check(bfp8, s)
    s = _setup(cuda_device, rng, [(12345, 70)], 1, 2, 128)
    _check(bfp8, s, rows=set(range(0, 70, 9)) | {69})


def test_a_prompt_of_many_heads(bfp8, cuda_device):
    """One prompt with several 256-row items an SM, behind a cached prefix."""
    rng = np.random.default_rng(31)
    s = _setup(cuda_device, rng, [(911, 700)], 16, 16, 32)
    _check(bfp8, s, rows={0, 1, 15, 16, 333, 698, 699})


@pytest.mark.parametrize("batch", [390, 900])
def test_many_requests_with_prompts_among_them(bfp8, cuda_device, batch):
    """More requests than a block has threads; prompts at the ends and between single tokens."""
    rng = np.random.default_rng(batch)
    lengths = [(int(rng.integers(1, 40)), 1) for _ in range(batch)]
    for b in (0, 130, 131, 383, 384, batch - 1):
        n = int(rng.integers(33, 90))
        lengths[b] = (n + int(rng.integers(0, 300)), n)
    _check(bfp8, _setup(cuda_device, rng, lengths, 1, 2, 16))


def test_sharp_and_flat_softmax(bfp8, cuda_device):
    rng = np.random.default_rng(23)
    for gain in (0.0, 30.0):
        s = _setup(cuda_device, rng, [(500, 1), (300, 40), (260, 260)], 2, 4, 32, q_gain=gain)
        _check(bfp8, s)
    s = _setup(cuda_device, rng, [(500, 1), (300, 40), (260, 260)], 2, 4, 32)
    _check(bfp8, s, scale=0.7)
    _check(bfp8, s, scale=-0.1)


def test_scales_far_apart(bfp8, cuda_device):
    """Pages whose value scales differ by up to 2^40 and key scales by 2^8: the weights' common
    maximum takes the value scale into account, so no page is lost."""
    rng = np.random.default_rng(24)
    s = _setup(cuda_device, rng, [(400, 1), (333, 60), (300, 200)], 2, 4, 16)
    P, H = s["k"][1].shape
    ev = rng.integers(100, 141, (P, H)).astype(np.uint8)
    ek = rng.integers(113, 122, (P, H)).astype(np.uint8)
    s["v"][1].copy_(torch.from_numpy(ev))
    s["k"][1].copy_(torch.from_numpy(ek))
    s["deq"] = [KV.dequantize(c[0].cpu().numpy(), e) for c, e in ((s["k"], ek), (s["v"], ev))]
    _check(bfp8, s)


def test_rows_that_see_nothing(bfp8, cuda_device):
    """Empty requests, more new rows than the cache holds, and missing pages."""
    rng = np.random.default_rng(25)
    s = _setup(cuda_device, rng, [(0, 2), (3, 7), (0, 0), (50, 1), (200, 70), (0, 90), (20, 100)], 2, 4, 16)
    _check(bfp8, s)
    s["table"][3, :4] = torch.tensor([-1, 10 ** 6, -5, 2 ** 31 - 1])    # no page of request 3 is there
    s["table"][4, 2] = -1                                                # one of request 4's is not
    s["table"][4, 7] = s["deq"][0].shape[0]
    _check(bfp8, s)


def test_a_table_narrower_than_the_length(bfp8, cuda_device):
    """Tokens past the table's width are not there."""
    rng = np.random.default_rng(26)
    s = _setup(cuda_device, rng, [(100, 1), (90, 80)], 1, 4, 16)
    wide = s["table"].clone()
    wide[:, 3:] = -1
    want = _run(bfp8, dict(s, table=wide))
    got = _run(bfp8, dict(s, table=s["table"][:, :3]))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_strided_rows(bfp8, cuda_device):
    """Queries as columns of a projection, the output inside a wider buffer, padding untouched."""
    rng = np.random.default_rng(27)
    s = _setup(cuda_device, rng, [(70, 1), (200, 3), (100, 100)], 2, 2, 32)
    want, lse = _run(bfp8, s)
    wide = torch.zeros(s["T"], 9, 136, dtype=torch.bfloat16, device=cuda_device)
    wide[:, 1:5, 8:] = s["q"]
    out = torch.full((s["T"], 6, 160), 7.0, dtype=torch.bfloat16, device=cuda_device)
    got, lse2 = _run(bfp8, dict(s, q=wide[:, 1:5, 8:]), out=out[:, 1:5, 16:144])
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    out[:, 1:5, 16:144] = 7.0
    assert bool((out == 7.0).all())


def test_results_repeat_bit_for_bit(bfp8, cuda_device):
    rng = np.random.default_rng(28)
    s = _setup(cuda_device, rng, [(5000, 1), (900, 2), (700, 300), (2, 1)], 2, 8, 64)
    a = _run(bfp8, s, fill=0xFF)
    b = _run(bfp8, s, fill=0x00)
    assert np.array_equal(bits16(a[0]), bits16(b[0])) and torch.equal(a[1], b[1])
    c = _run(bfp8, s, lse=False)
    assert np.array_equal(bits16(a[0]), bits16(c[0]))


def test_a_nan_reaches_the_rows_that_see_it(bfp8, cuda_device):
    rng = np.random.default_rng(29)
    s = _setup(cuda_device, rng, [(60, 1), (60, 1), (200, 100)], 1, 4, 16)
    s["q"][0, 1] = float("nan")
    page = int(s["table"][1, 2])
    s["v"][0][page, 0, 5, 9] = 0x7F
    out, lse = _run(bfp8, s)
    nan = torch.isnan(out.float())
    assert bool(nan[0, 1].all()) and not bool(nan[0, [0, 2, 3]].any())
    assert bool(nan[1, :, 9].all()) and int(nan[1].sum()) == 4
    assert not bool(nan[2:].any())


def test_graph_replay_follows_the_lengths(bfp8, cuda_device):
    """A captured call reads lengths and tables when it is replayed."""
    rng = np.random.default_rng(30)
    s = _setup(cuda_device, rng, [(300, 1), (640, 1)], 2, 4, 64)
    out, lse = torch.empty_like(s["q"]), torch.empty(s["T"], 8, device=cuda_device)
    ws = torch.empty(bfp8.bfp8_kv_attention_workspace(2, 2, 1, 8, 2), dtype=torch.uint8, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bfp8.bfp8_kv_attention(s["q"], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["off"], s["kv"], out, 1,
                               lse=lse, workspace=ws)
    for lengths in ([300, 640], [299, 1], [0, 640], [64, 65]):
        s["kv"].copy_(torch.tensor(lengths, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        _check(bfp8, dict(s, lengths=[(n, 1) for n in lengths]), got=(out, lse))


def test_graph_replay_of_a_mixed_batch(bfp8, cuda_device):
    """Prompts and single tokens in one captured call, replayed with other lengths and row counts."""
    rng = np.random.default_rng(34)
    s = _setup(cuda_device, rng, [(300, 90), (640, 1), (500, 200)], 2, 4, 32)
    out, lse = torch.empty_like(s["q"]), torch.empty(s["T"], 8, device=cuda_device)
    ws = torch.empty(bfp8.bfp8_kv_attention_workspace(3, s["T"], 200, 8, 2), dtype=torch.uint8, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bfp8.bfp8_kv_attention(s["q"], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["off"], s["kv"], out,
                               200, lse=lse, workspace=ws)
    for lengths in ([(300, 90), (640, 1), (500, 200)], [(299, 1), (20, 20), (499, 3)], [(64, 0), (640, 150), (1, 1)]):
        s["kv"].copy_(torch.tensor([kv for kv, _ in lengths], dtype=torch.int32))
        s["off"].copy_(torch.tensor(np.cumsum([0] + [n for _, n in lengths]), dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        assert bfp8.bfp8_device_status() == 0
        _check(bfp8, dict(s, lengths=lengths), got=(out, lse))


def test_appends_and_attention_back_to_back(bfp8, cuda_device):
    """Each call reads what the append before it wrote, with nothing between them that waits."""
    rng = np.random.default_rng(35)
    s = _setup(cuda_device, rng, [(700, 1), (400, 120), (333, 2), (900, 300)], 2, 4, 32)
    slots = torch.cat([s["table"][b, torch.arange(n, device=cuda_device) // 32].long() * 32
                       + torch.arange(n, device=cuda_device) % 32 for b, n in enumerate((700, 400, 333, 900))])
    new = [torch.randn(2, len(slots), 2, D, device=cuda_device).to(torch.bfloat16) for _ in range(6)]
    cache = (s["k"][0], s["v"][0], s["k"][1], s["v"][1])
    n = bfp8.bfp8_kv_attention_workspace(4, s["T"], 300, 8, 2)
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)

    def go(i, out, sync):
        bfp8.bfp8_kv_append(new[i][0], new[i][1], slots, *cache)
        if sync:
            torch.cuda.synchronize()
        bfp8.bfp8_kv_attention(s["q"], *cache, s["table"], s["off"], s["kv"], out, 300, workspace=ws)
        if sync:
            torch.cuda.synchronize()

    outs = [[torch.empty_like(s["q"]) for _ in new] for _ in range(3)]
    for k, sync in enumerate((True, False, False)):
        for i in range(len(new)):
            go(i, outs[k][i], sync)
    torch.cuda.synchronize()
    for i in range(len(new)):
        assert torch.equal(outs[0][i], outs[1][i]) and torch.equal(outs[0][i], outs[2][i]), i


def test_two_streams_at_once(bfp8, cuda_device):
    rng = np.random.default_rng(31)
    a = _setup(cuda_device, rng, [(3000, 1)] * 3 + [(400, 200)], 2, 4, 64)
    b = _setup(cuda_device, rng, [(2000, 2)] * 2, 4, 2, 16)
    wa, wb = _run(bfp8, a), _run(bfp8, b)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for st, s in zip(streams, (a, b)):
        with torch.cuda.stream(st):
            out = torch.empty_like(s["q"])
            ws = torch.empty(bfp8.bfp8_kv_attention_workspace(len(s["lengths"]), s["T"], s["maxq"], 8, s["H"]),
                             dtype=torch.uint8, device=cuda_device)
            for _ in range(3):
                bfp8.bfp8_kv_attention(s["q"], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["off"], s["kv"],
                                       out, s["maxq"], workspace=ws)
            got.append((out, ws))
    torch.cuda.synchronize()
    assert torch.equal(got[0][0], wa[0]) and torch.equal(got[1][0], wb[0])


def test_cache_past_32_bits(bfp8, cuda_device):
    """Pages whose byte offsets need more than 32 bits, found through the table."""
    rng = np.random.default_rng(32)
    P, H, page = 140000, 8, 32
    small = _setup(cuda_device, rng, [(90, 1), (64, 40)], H, 1, page, extra=0)
    want = _run(bfp8, small)
    far = torch.tensor([P - 1, 65536, 131072, 3, 99999], device=cuda_device)
    big = dict(small)
    for x in ("k", "v"):
        codes = torch.zeros(P, H, page, D, dtype=torch.uint8, device=cuda_device)
        exps = torch.zeros(P, H, dtype=torch.uint8, device=cuda_device)
        codes[far], exps[far] = small[x][0], small[x][1]
        big[x] = (codes, exps)
    t = small["table"].clone()
    real = (t >= 0) & (t < 5)
    t[real] = far[t[real].long()].to(torch.int32)
    got = _run(bfp8, dict(big, table=t))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_workspace_holds_every_smaller_call(bfp8, cuda_device):
    """What is enough for a batch, tokens and lengths is enough for fewer of any of them."""
    sizes = [(b, t, q) for b in (1, 2, 17, 300) for t in (1, 40, 700, 5000) for q in (1, 8, 9, 64, 65, 700, 5000)]
    need = {x: bfp8.bfp8_kv_attention_workspace(*x, 64, 8) for x in sizes}
    for a in sizes:
        for b in sizes:
            if all(x <= y for x, y in zip(a, b)):
                assert need[a] <= need[b], (a, b)


def test_refusals(bfp8, cuda_device):
    rng = np.random.default_rng(33)
    s = _setup(cuda_device, rng, [(70, 1), (20, 2)], 2, 2, 32)
    ws = torch.empty(bfp8.bfp8_kv_attention_workspace(2, 3, 2, 4, 2), dtype=torch.uint8, device=cuda_device)
    out = torch.empty_like(s["q"])

    def call(err, match=None, **kw):
        a = dict(q=s["q"], k=s["k"][0], ke=s["k"][1], table=s["table"], off=s["off"], kv=s["kv"], out=out, ws=ws, lse=None)
        a.update(kw)
        with pytest.raises(err, match=match):
            bfp8.bfp8_kv_attention(a["q"], a["k"], s["v"][0], a["ke"], s["v"][1], a["table"], a["off"], a["kv"], a["out"],
                                   2, lse=a["lse"], workspace=a["ws"])

    call(bfp8.Bfp8Error, "INVALID_ARG", ws=None)
    call(bfp8.Bfp8Error, "INVALID_ARG", ws=ws[:-256])
    call(bfp8.Bfp8Error, "INVALID_ARG", ws=torch.empty(ws.numel() + 256, dtype=torch.uint8, device=cuda_device)[8:])
    call(bfp8.Bfp8Error, "INVALID_ARG", q=s["q"][:, :3], out=out[:, :3])      # 3 heads on 2 KV heads
    call(ValueError, "bfloat16", q=s["q"].float())
    call(ValueError, "shape", out=out[:2])
    call(ValueError, "int32", table=s["table"].long())
    call(ValueError, "shape", off=s["off"][:2])
    call(ValueError, "shape", kv=s["kv"][:1])
    call(ValueError, "shape", lse=torch.empty(3, 3, device=cuda_device))
    call(ValueError, "k_exp", ke=s["k"][1][:, :1])
    call(ValueError, "shape|head dim", k=s["k"][0][..., :64])
    pad = torch.empty(3, 4, 132, dtype=torch.bfloat16, device=cuda_device)
    call(bfp8.Bfp8Error, "UNSUPPORTED", q=pad[:, :, 4:])
    # nothing to do
    bfp8.bfp8_kv_attention(s["q"][:0], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"][:0], s["off"][:1], s["kv"][:0],
                           out[:0], 1, workspace=ws)


def test_c_abi_refuses_host_memory(bfp8, cuda_device):
    import ctypes
    d = torch.zeros(32 << 20, dtype=torch.uint8, device=cuda_device).data_ptr()
    h = torch.zeros(1 << 16, dtype=torch.uint8).data_ptr()
    cache = bfp8.bfp8_kv_cache(d, d, d, d, 4, 16, 1, 128, 2048, 2048, 128, 2048, 2048, 128, 1, 1)
    fields = ("q_bf16", "out_bf16", "lse", "block_table", "q_offsets", "kv_len", "workspace")
    for bad in fields:
        a = bfp8.bfp8_kv_attention_args(**{f: (h if f == bad else d) for f in fields}, q_stride_token=128, q_stride_head=128,
                                        out_stride_token=128, out_stride_head=128, lse_stride_token=1, ld_table=4,
                                        max_blocks=4, batch=1, tokens=1, max_q_len=1, n_heads=1, softmax_scale=1.0,
                                        window=-1, ws_bytes=30 << 20)
        rc = bfp8._lib.bfp8_kv_attention(ctypes.byref(a), ctypes.byref(cache), None)
        assert bfp8.bfp8_status_string(rc) == "INVALID_ARG", bad
