"""bfp8_kv_attention at the ends of its range: scores far past what a softmax resolves,
queries that are infinite or nearly so, what lies behind a window, and limits that
meet 32 bits.
"""

import numpy as np
import pytest
import torch

from oracle import kv as KV
from test_gpu_kv_attention import D, _check, _run, _setup

pytestmark = pytest.mark.gpu


def _rows(s):
    """(token, head, keys that it sees, values that it sees) of every row, in float64."""
    q, (kd, vd), G = s["q"].double().cpu().numpy(), s["deq"], s["G"]
    table, off = s["table"].cpu().numpy(), s["off"].cpu().numpy()
    page = kd.shape[2]
    for b, (kv, n) in enumerate(s["lengths"]):
        pages = table[b, :-(-kv // page)]
        for h in range(kd.shape[1]):
            k, v = (x[pages, h].reshape(-1, D)[:kv] for x in (kd, vd))
            for t in range(off[b], off[b + 1]):
                end = kv - n + (t - off[b]) + 1
                for g in range(G):
                    yield t, h * G + g, q[t, h * G + g], k[:end], v[:end]


BIG = [[(300, 1), (64, 2)], [(300, 200)], [(260, 1), (400, 200), (70, 70)]]   # few rows; a prompt; both


@pytest.mark.parametrize("lengths", BIG)
@pytest.mark.parametrize("ek", [12, 16, 18, 19, 20, 21, 22, 24, 28, 34, 40])
def test_large_scores_find_the_largest(bfp8, cuda_device, lengths, ek):
    """Keys with large scales: scores of 2^(8 + ek), whose float32 steps pass the softmax's range. A
    row's score is off by FP32's rounding of its products' sum, less than 2^-16 of the sum of their
    sizes; where the largest score leads by more than twice that and by 30, the output is its value (a
    weight's and BF16's rounding apart) and lse the score."""
    rng = np.random.default_rng(ek)
    s = _setup(cuda_device, rng, lengths, 2, 4, 32)
    s["k"][1].fill_(127 + ek)
    s["deq"] = [KV.dequantize(c[0].cpu().numpy(), c[1].cpu().numpy()) for c in (s["k"], s["v"])]
    out, lse = (x.double().cpu().numpy() for x in _run(bfp8, s))
    assert np.isfinite(out).all() and np.isfinite(lse).all()
    seen = 0
    for t, h, q, k, v in _rows(s):
        z = k @ q * D ** -0.5
        off = 2.0 ** -16 * (np.abs(k) @ np.abs(q)).max() * D ** -0.5
        best = int(z.argmax())
        assert abs(lse[t, h] - z[best]) <= off + np.log(len(z)), (t, h)
        if len(z) > 1 and z[best] - np.partition(z, -2)[-2] < 2 * off + 30:
            continue
        seen += 1
        assert np.all(np.abs(out[t, h] - v[best]) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(v[best])), (t, h)
    assert seen > 0


@pytest.mark.parametrize("lengths", BIG + [[(4100, 1)] * 40])
@pytest.mark.parametrize("ek", [10, 13, 14, 15, 16, 17, 18, 19, 20, 21, 22, 26, 40])
def test_large_scores_a_step_apart(bfp8, cuda_device, lengths, ek):
    """Scores of 2^(8 + ek) in log2 units that go up and down by a float32 step every 128 tokens. All
    tokens hold the same value, so whatever the weights, the output is that value; and lse is the
    score, to its rounding and the number of tokens."""
    rng = np.random.default_rng(ek)
    s = _setup(cuda_device, rng, lengths, 1, 4, 32)
    P, _, page, _ = s["deq"][0].shape
    value = rng.integers(0x20, 0x60, D).astype(np.uint8)
    codes = np.zeros((2, P, 1, page, D), np.uint8)
    codes[0, ..., 0] = 0x78                                  # 256
    codes[1] = value
    table = s["table"].cpu().numpy()
    for b, (kv, _) in enumerate(lengths):
        for j in range(-(-kv // page)):                      # 0.25, then 0.5: one step, then two
            codes[0, table[b, j], 0, :, 1] = 0x30 if j * page // 128 % 2 else 0x28
    for x, c, e in (("k", codes[0], 127 + ek), ("v", codes[1], 127)):
        s[x][0].copy_(torch.from_numpy(c))
        s[x][1].fill_(e)
    s["q"].zero_()
    s["q"][..., 0], s["q"][..., 1] = 1.0, 2.0 ** -13
    out, lse = (x.double().cpu().numpy() for x in _run(bfp8, s, scale=float(np.float32(np.log(2)))))
    want = KV.dequantize(value[None, None, None], np.full((1, 1), 127, np.uint8))[0, 0, 0]
    assert np.all(np.abs(out - want) <= (2.0 ** -8 + 2.0 ** -10) * np.abs(want))
    x = np.log(2) * 2.0 ** (8 + ek)
    assert np.all(np.abs(lse - x) <= 2.0 ** -16 * x + np.log(4100))


@pytest.mark.parametrize("lengths", BIG)
def test_infinite_queries_give_nan(bfp8, cuda_device, lengths):
    """An infinity among a row's queries makes its scores infinite, of either sign or NaN: the row is
    NaN, and no other is."""
    rng = np.random.default_rng(41)
    s = _setup(cuda_device, rng, lengths, 2, 4, 32)
    bad = [(0, 1, 5, np.inf), (0, 6, 127, -np.inf), (s["T"] - 1, 3, 64, np.inf), (s["T"] // 2, 0, 0, -np.inf)]
    want = torch.zeros(s["T"], 8, dtype=torch.bool)
    for t, h, d, x in bad:
        s["q"][t, h, d] = x
        want[t, h] = True
    s["q"][s["T"] - 1, 5] = float("inf")
    want[s["T"] - 1, 5] = True
    out, lse = _run(bfp8, s)
    nan = torch.isnan(out.float()).cpu()
    assert torch.equal(nan.all(2), want) and torch.equal(nan.any(2), want) and torch.equal(torch.isnan(lse).cpu(), want)


@pytest.mark.parametrize("lengths", BIG)
@pytest.mark.parametrize("top", [2.0 ** 126, 3.0e38, 2.0 ** 127, 2.0 ** -90])
def test_queries_near_the_ends_of_their_range(bfp8, cuda_device, lengths, top):
    """The largest finite queries, under a scale that brings their scores back, and very small ones."""
    rng = np.random.default_rng(42)
    s = _setup(cuda_device, rng, lengths, 2, 4, 32)
    q = s["q"].float()
    s["q"] = (q / q.abs().amax(2, keepdim=True) * top).to(torch.bfloat16)
    assert bool(torch.isfinite(s["q"]).all())
    _check(bfp8, s, scale=0.5 / top)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("lengths", [[(500, 1), (700, 3), (131, 2), (1000, 1)], [(900, 200)],
                                     [(600, 200), (500, 1), (333, 64), (90, 90), (777, 130)]])
def test_what_lies_behind_the_window_is_never_used(bfp8, cuda_device, lengths, page):
    """Pages behind the window may have gone to other requests: their rows may hold NaN codes, their
    scale bytes anything, and so may the rows of a page ahead of the first that is seen."""
    rng = np.random.default_rng(page)
    window = 100
    s = _setup(cuda_device, rng, lengths, 2, 4, page)
    table = s["table"].cpu().numpy()
    for b, (kv, n) in enumerate(lengths):
        first = max(kv - n - window, 0)
        for i in range(first):
            for x in ("k", "v"):
                s[x][0][int(table[b, i // page]), :, i % page] = 0x7F
        for j in range(first // page):
            for x, e in (("k", 255), ("v", 0 if j % 2 else 255)):
                s[x][1][int(table[b, j])] = e
    _check(bfp8, s, window)
    assert any(kv - n > window + page for kv, n in lengths)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60, 1000, 15])
def test_windows_of_rows_before_the_first_position(bfp8, cuda_device, window):
    """More new rows than the cache holds, under windows that a position below 0 must not carry past 32
    bits: the rows at positions from 0 on see what they see without a window."""
    rng = np.random.default_rng(43)
    for lengths in ([(20, 100)], [(20, 100), (9, 12), (300, 1)], [(5, 7), (0, 3)]):
        _check(bfp8, _setup(cuda_device, rng, lengths, 1, 4, 16), window)


def test_a_mixed_batch_reads_what_was_written_just_before_it(bfp8, cuda_device):
    """Queries, lengths, table, codes and scale bytes that kernels right ahead of the call write, each
    time others, with nothing between them that waits for the device: single tokens and prompts."""
    rng = np.random.default_rng(45)
    lengths = [(700, 1), (400, 120), (333, 2), (900, 300), (40, 1)]
    sets = [_setup(cuda_device, rng, [lengths[i] for i in rng.permutation(len(lengths))], 2, 4, 32) for _ in range(6)]
    want = [_run(bfp8, s) for s in sets]
    live = {x: torch.empty_like(sets[0][x]) for x in ("q", "off", "kv", "table")}
    live |= {x: tuple(torch.zeros_like(t) for t in sets[0][x]) for x in ("k", "v")}
    n = bfp8.bfp8_kv_attention_workspace(5, sets[0]["T"], 300, 8, 2)
    ws = torch.empty(n, dtype=torch.uint8, device=cuda_device)
    outs = []
    torch.cuda.synchronize()
    for i in [0, 3, 1, 5, 2, 4, 0, 5]:
        for x, to in live.items():
            for dst, src in zip(to, sets[i][x]) if isinstance(to, tuple) else [(to, sets[i][x])]:
                dst.copy_(src)
        out, lse = torch.empty_like(live["q"]), torch.empty(live["q"].shape[:2], device=cuda_device)
        bfp8.bfp8_kv_attention(live["q"], live["k"][0], live["v"][0], live["k"][1], live["v"][1], live["table"], live["off"],
                               live["kv"], out, 300, lse=lse, workspace=ws)
        outs.append((i, out, lse))
    torch.cuda.synchronize()
    for i, out, lse in outs:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i


@pytest.mark.parametrize("lengths,most", [([(5000, 5), (90, 3), (7, 7)], 2), ([(300, 200)], 100), ([(900, 40)], 3),
                                          ([(300, 200), (5000, 30), (70, 1), (64, 64)], 20)])
def test_rows_past_the_most_are_not_written(bfp8, cuda_device, lengths, most):
    """A request with more new rows than max_q_len: its first max_q_len rows, at their places in the
    request, and nothing of the others."""
    rng = np.random.default_rng(most)
    s = dict(_setup(cuda_device, rng, lengths, 2, 4, 32), maxq=most)
    out, lse = _run(bfp8, s)
    off = s["off"].tolist()
    past = [t for b in range(len(lengths)) for t in range(off[b] + most, off[b + 1])]
    assert past and bool(torch.isnan(out[past].float()).all()) and bool(torch.isnan(lse[past]).all())
    _check(bfp8, s, rows=set(range(s["T"])) - set(past), got=(out, lse))


@pytest.mark.parametrize("most", [1000, 2 ** 31, 2 ** 62, 2 ** 63 - 1])
def test_a_most_beyond_the_tokens(bfp8, cuda_device, most):
    """max_q_len is an upper bound: any above the call's tokens is as good as their number."""
    rng = np.random.default_rng(46)
    for lengths in ([(70, 1), (300, 3)], [(400, 150)], [(400, 150), (60, 1)]):
        s = _setup(cuda_device, rng, lengths, 2, 4, 32)
        need = [bfp8.bfp8_kv_attention_workspace(len(lengths), s["T"], q, 8, 2) for q in (s["T"], most)]
        assert need[0] == need[1]
        _check(bfp8, dict(s, maxq=most))


def test_a_workspace_holds_every_smaller_call_of_other_heads(bfp8, cuda_device):
    """Heads vary too: layers with other numbers of query and KV heads share one workspace."""
    heads = [(4, 1), (4, 4), (16, 2), (64, 4), (64, 8), (64, 64), (128, 1), (128, 8)]
    sizes = [(b, t, q, *h) for b in (1, 3) for t in (1, 700) for q in (1, 8, 16, 65, 700) for h in heads]
    need = {x: bfp8.bfp8_kv_attention_workspace(*x) for x in sizes}
    for a in sizes:
        for b in sizes:
            if all(x <= y for x, y in zip(a, b)):
                assert need[a] <= need[b], (a, b)
    # and the call takes it: 8 rows of 8 heads on 2 KV heads, in the workspace of 8 on 8
    rng = np.random.default_rng(44)
    s = _setup(cuda_device, rng, [(70, 20), (100, 1)], 2, 4, 32)
    ws = torch.empty(bfp8.bfp8_kv_attention_workspace(2, s["T"], 20, 8, 8), dtype=torch.uint8, device=cuda_device)
    _check(bfp8, s, got=_run(bfp8, s, ws=ws))


# ---- one prompt with several items of 256 rows an SM, which blocks take whole ------


def _whole(dev, seed, kv, n, page, G=5, H=64):
    """64 KV heads of five: 640 items for 460 rows and more, on 152 SMs."""
    return _setup(dev, np.random.default_rng(seed), [(kv, n)], H, G, page)


def _boundary_rows(n, G=5):
    """Tokens on both sides of every 128th row, the first and the last."""
    return {t for r in range(0, n * G + 1, 128) for t in ((r - 1) // G, r // G, r // G + 1) if 0 <= t < n} | {0, n - 1}


@pytest.mark.parametrize("page,window", [(16, -1), (64, 100), (128, 300), (32, 0)])
def test_whole_items_of_a_prompt(bfp8, cuda_device, page, window):
    s = _whole(cuda_device, page, 900, 470, page)
    _check(bfp8, s, window, rows=_boundary_rows(470))


def test_whole_items_without_tokens_or_pages(bfp8, cuda_device):
    """Items whose rows all sit before the first position, and a prompt with pages missing."""
    _check(bfp8, _whole(cuda_device, 51, 200, 470, 32), rows=_boundary_rows(470))
    s = _whole(cuda_device, 52, 700, 470, 32)
    s["table"][0, [0, 3, 4, 5, 6, 15]] = torch.tensor([-1, -1, -7, 10 ** 6, 2 ** 31 - 1, s["deq"][0].shape[0]],
                                                       dtype=torch.int32, device=cuda_device)
    _check(bfp8, s, rows=_boundary_rows(470))


def test_whole_items_replayed_with_fewer_rows(bfp8, cuda_device):
    """A call captured for 470 rows, replayed for one, a few and a few hundred."""
    s = _whole(cuda_device, 53, 900, 470, 64)
    out, lse = torch.empty_like(s["q"]), torch.empty(470, 320, device=cuda_device)
    ws = torch.empty(bfp8.bfp8_kv_attention_workspace(1, 470, 470, 320, 64), dtype=torch.uint8, device=cuda_device)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bfp8.bfp8_kv_attention(s["q"], s["k"][0], s["v"][0], s["k"][1], s["v"][1], s["table"], s["off"], s["kv"], out, 470,
                               lse=lse, workspace=ws)
    for kv, n in ((900, 470), (899, 1), (12, 9), (640, 300), (77, 0), (0, 4), (470, 470)):
        s["kv"].fill_(kv)
        s["off"].copy_(torch.tensor([0, n], dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert bfp8.bfp8_device_status() == 0
        _check(bfp8, dict(s, lengths=[(kv, n)]), rows=_boundary_rows(n) if n else set(), got=(out, lse))
        assert bool(torch.isnan(out[n:].float()).all())


@pytest.mark.parametrize("lengths", BIG)
def test_codes_of_a_token_side_by_side(bfp8, cuda_device, lengths):
    """A cache whose tokens lie outside of its heads, for prompts too."""
    s = _setup(cuda_device, np.random.default_rng(47), lengths, 3, 4, 64, order="tokens")
    _check(bfp8, s)


def test_a_table_of_no_width_and_rows_of_no_request(bfp8, cuda_device):
    """With no table there is nothing to see; rows behind the last request's are left alone."""
    for lengths in ([(40, 1), (9, 2)], [(100, 90)], [(100, 90), (5, 1)]):
        s = _setup(cuda_device, np.random.default_rng(48), lengths, 2, 4, 32)
        out, lse = _run(bfp8, dict(s, table=s["table"][:, :0]))
        assert bool((out == 0).all()) and bool(torch.isneginf(lse).all())
        more = dict(s, q=torch.cat([s["q"], s["q"][:3]]), T=s["T"] + 3)
        out, lse = _run(bfp8, more)
        assert bool(torch.isnan(out[s["T"]:].float()).all()) and bool(torch.isnan(lse[s["T"]:]).all())
        _check(bfp8, s, got=(out[:s["T"]], lse[:s["T"]]))
