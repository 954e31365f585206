"""bfp8_delta_rule on the GPU against the oracle in float64.

Tolerances. One token adds to a row of the state an error of at most c (1 + |g|) 2^-24 (alpha |S_row| + |v|): the
gate's logarithm is a handful of rounded steps (alpha's error is 8 |g| 2^-24 and the exponential's), key and query
are normed within 16 2^-24, a product with the state sums 128 terms in chains and trees of at most 16 roundings, and
beta, u and the update are 8 more; c = 64 counts each twice. Requests of many tokens go through chunks of 64, whose
sums run over 64 to 128 terms in the tensor cores (each truncated to FP32, 2^-23) with operands split into two F16
parts (2^-22), three such products one behind another, and the decay of a chunk in place of a token's: c = 512 counts
128 terms of 2^-23 twice, and the operands' three times 4 2^-24 within that. The oracle's `grown` carries such errors through the recurrence, which lengthens
none; the output adds the product with the query (|q'| = scale) and half a BF16 step, 2^-8.
"""

import numpy as np
import pytest
import torch

from hybrid_util import delta_inputs, f64, i32, nan_like, offsets
from oracle import hybrid as HY

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "a", "b", "a_log", "dt_bias", "state", "slots_in", "slots_out", "q_offsets", "out")


def _run(bfp8, t, lens, max_q_len=None, ws=None, **kw):
    before = t["state"].clone()
    most = max(lens) if max_q_len is None else max_q_len
    T, hv = t["out"].shape[:2]
    if ws is None:
        n = bfp8.bfp8_delta_rule_workspace(len(lens), T, max(1, most), t["q"].shape[1], hv)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=t["out"].device)
    bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), most, workspace=ws, **kw)
    torch.cuda.synchronize()
    assert bfp8.bfp8_device_status() == 0
    return before


def _check(t, lens, before, scale=128 ** -0.5, eps=1e-6, c=512):
    x = {k: f64(t[k]) for k in ("q", "k", "v", "a", "b", "a_log", "dt_bias")}
    want_state, out, state = f64(before), f64(t["out"]), f64(t["state"])
    tol_state, at = np.zeros(want_state.shape[:3]), 0
    for n, src, dst in zip(lens, t["slots_in"].tolist(), t["slots_out"].tolist()):
        rows = slice(at, at + n)
        S0 = f64(before)[src] if 0 <= src < len(want_state) else np.zeros(want_state.shape[1:])
        want, S, grown, met = HY.delta_rule(*(x[k][rows] for k in ("q", "k", "v", "a", "b")), x["a_log"], x["dt_bias"], S0,
                                            scale, eps)
        tol = c * 2.0 ** -24 * abs(scale) * met
        off = np.abs(out[rows] - want)
        assert np.all(off <= tol + 2.0 ** -8 * (np.abs(want) + tol)), (n, float(np.max(off / (tol + 2.0 ** -8 * np.abs(want) + 1e-30))))
        if n and 0 <= dst < len(want_state):
            want_state[dst], tol_state[dst] = S, c * 2.0 ** -24 * grown
        at += n
    assert np.isnan(out[at:]).all()
    off = np.linalg.norm(state - want_state, axis=3)
    assert np.all(off <= tol_state), float(np.max(off / (tol_state + 1e-30)))


STEPS = [[1], [1] * 9, [3, 3, 3], [2, 0, 1, 4, 7, 0, 5], [28, 5, 27]]
PROMPTS = [[64], [65], [29], [12, 13, 30], [63], [128, 1, 64], [40, 0, 100, 1, 17, 33], [200], [15, 16, 17, 31, 32, 33], [1, 130, 3, 66]]


@pytest.mark.parametrize("lens", STEPS, ids=str)
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (3, 9), (1, 4)])
def test_steps_match_oracle(bfp8, cuda_device, lens, hk, hv):
    t = delta_inputs(cuda_device, lens, hk, hv, 7 * hv + len(lens), extra=2)
    _check(t, lens, _run(bfp8, t, lens), c=64)


@pytest.mark.parametrize("lens", PROMPTS, ids=str)
@pytest.mark.parametrize("hk,hv", [(1, 1), (2, 4), (1, 3)])
def test_prompts_match_oracle(bfp8, cuda_device, lens, hk, hv):
    t = delta_inputs(cuda_device, lens, hk, hv, 11 * hv + sum(lens), extra=3)
    _check(t, lens, _run(bfp8, t, lens))


@pytest.mark.parametrize("lens,c", [([20, 1, 19], 64), ([21, 20, 12, 13], 512), ([20], 64), ([21], 512)], ids=str)
def test_lengths_about_the_limit_of_steps(bfp8, cuda_device, lens, c):
    t = delta_inputs(cuda_device, lens, 2, 6, 41 + sum(lens), extra=1)
    _check(t, lens, _run(bfp8, t, lens), c=c)


@pytest.mark.parametrize("lens,hk,hv", [([3000], 1, 1), ([2049], 1, 2), ([2500, 7, 40, 1300], 2, 2), ([1500, 1501], 1, 4),
                                        ([64 * 27 + 1, 64 * 30, 0, 64 * 9], 1, 1)], ids=str)
@pytest.mark.parametrize("decay", [1e-3, 1.0])
def test_long_prompts_match_oracle(bfp8, cuda_device, lens, hk, hv, decay):
    """Prompts of few heads, whose chunks are walked in segments at once and joined; short ones beside them."""
    t = delta_inputs(cuda_device, lens, hk, hv, 19 * hv + sum(lens), extra=1, decay=decay)
    _check(t, lens, _run(bfp8, t, lens))


@pytest.mark.parametrize("lens,hk,hv", [([64 * 36 - 5], 16, 64), ([64 * 35 + 1], 9, 72), ([64 * 50, 64 * 11 + 3], 2, 20), ([3300], 4, 40)], ids=str)
def test_long_prompts_of_many_heads_match_oracle(bfp8, cuda_device, lens, hk, hv):
    """Segments that come in waves, the first one longer than the others; one request ends inside its first."""
    t = delta_inputs(cuda_device, lens, hk, hv, 29 * hv + sum(lens), extra=1, decay=0.1)
    _check(t, lens, _run(bfp8, t, lens))


def test_many_requests_of_ragged_lengths(bfp8, cuda_device):
    """More heads than SMs: blocks begin with the longest of each 32 requests."""
    lens = [(37 * i * i + 11 * i) % 150 if i % 5 else 0 for i in range(67)]
    t = delta_inputs(cuda_device, lens, 2, 4, 47, extra=2)
    _check(t, lens, _run(bfp8, t, lens))


def test_long_prompts_in_one_slot_and_replayed(bfp8, cuda_device):
    """Read from and left in the same slot; captured, and replayed with lengths that end in other segments."""
    dev = cuda_device
    T = 2400
    t = delta_inputs(dev, [T], 1, 1, 23)
    t["slots_in"] = t["slots_out"]
    ws = torch.empty(bfp8.bfp8_delta_rule_workspace(1, T, T, 1, 1), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), T, workspace=ws)
    for n in (T, 900, 64, 12, 2239, 0):
        t["q_offsets"].copy_(offsets(dev, [n]))
        t["out"].fill_(float("nan"))
        before = t["state"].clone()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        _check(t, [n], before)


@pytest.mark.parametrize("decay", [1e-6, 40.0])
def test_heads_that_keep_all_and_heads_that_forget_at_once(bfp8, cuda_device, decay):
    lens = [150, 70]
    t = delta_inputs(cuda_device, lens, 1, 2, 5, decay=decay)
    _check(t, lens, _run(bfp8, t, lens))


@pytest.mark.parametrize("n", [5, 200])
def test_keys_that_repeat(bfp8, cuda_device, n):
    """One key for every token, beta near 1, hardly any decay: each value replaces the one before it."""
    t = delta_inputs(cuda_device, [n], 1, 2, 6, decay=1e-4)
    t["k"][:] = t["k"][:1].clone()
    t["b"][:] = 9.0
    _check(t, [n], _run(bfp8, t, [n]))


@pytest.mark.parametrize("n", [4, 100])
def test_keys_and_queries_of_nothing(bfp8, cuda_device, n):
    """A key of zeros stores nothing and a query of zeros reads nothing; eps keeps both finite."""
    t = delta_inputs(cuda_device, [n], 2, 2, 7)
    t["k"][1], t["q"][2] = 0, 0
    before = _run(bfp8, t, [n])
    assert not t["out"][2].any()
    _check(t, [n], before)


@pytest.mark.parametrize("n", [4, 100])
def test_large_and_small_inputs(bfp8, cuda_device, n):
    """Keys and queries are normed whatever their size; values are taken as they are."""
    t = delta_inputs(cuda_device, [n], 1, 2, 8)
    size = torch.tensor([2.0 ** e for e in np.linspace(-6, 50, n).round()], device=cuda_device)[:, None, None]
    t["k"].copy_(t["k"].float() * size)
    t["q"].copy_(t["q"].float() * size.flip(0))
    t["v"].copy_(t["v"].float() * 2.0 ** 40)
    t["state"] *= 2.0 ** 40
    _check(t, [n], _run(bfp8, t, [n], eps=1e-12), eps=1e-12)


@pytest.mark.parametrize("a", [-60.0, 30.0, 3.0e38])
@pytest.mark.parametrize("n", [3, 90])
def test_gates_at_their_ends(bfp8, cuda_device, a, n):
    t = delta_inputs(cuda_device, [n], 1, 2, 9)
    t["a"][::2], t["b"][1::2] = a, -200.0
    t["b"][::3] = 200.0
    x = {k: f64(t[k]) for k in ("a", "b", "a_log", "dt_bias")}
    g, _ = HY.delta_gates(x["a"], x["b"], x["a_log"], x["dt_bias"])
    if a < 1e30:
        _check(t, [n], _run(bfp8, t, [n]))
    else:                                            # a decay to nothing: the state is the last tokens' own
        _run(bfp8, t, [n])
        assert torch.isfinite(t["out"][:n]).all() and torch.isfinite(t["state"]).all()


def test_steps_in_one_slot_are_the_whole_prompt(bfp8, cuda_device):
    """The same slot read and written by chunks, drafted tokens and single ones, against one call's bounds."""
    dev = cuda_device
    whole, cuts = 180, [70, 3, 1, 1, 65, 4, 20, 16]
    t = delta_inputs(dev, [whole], 2, 4, 10, slots=3)
    before, at = t["state"].clone(), 0
    slot = t["slots_in"].clone()
    for n in cuts:
        piece = dict(t, **{k: t[k][at:at + n] for k in ("q", "k", "v", "a", "b", "out")}, slots_in=slot, slots_out=slot,
                     q_offsets=offsets(dev, [n]))
        _run(bfp8, piece, [n])
        at += n
    _check(dict(t, slots_out=slot), [whole], before, c=64 * len(cuts))


def test_slots_outside_the_pool_no_state_and_lengths_past_max_q_len(bfp8, cuda_device):
    dev = cuda_device
    lens = [3, 80, 2, 70]
    t = delta_inputs(dev, lens, 1, 2, 11)
    n_slots = t["state"].shape[0]
    t["slots_in"][:] = i32(dev, [n_slots, -9, 0, 2 ** 31 - 1])
    t["slots_out"][:] = i32(dev, [1, n_slots, -1, 2])
    _check(t, lens, _run(bfp8, t, lens))
    # no state at all: what slots of -1 give
    t["slots_in"].fill_(-1)
    _run(bfp8, t, lens)
    want = t["out"].clone()
    bare = dict(t, state=None, slots_in=None, slots_out=None, out=nan_like(want.shape, dev))
    n = bfp8.bfp8_delta_rule_workspace(4, sum(lens), 80, 1, 2)
    bfp8.bfp8_delta_rule(*(bare[k] for k in NAMES), 80, workspace=torch.empty(n, dtype=torch.uint8, device=dev))
    assert torch.equal(bare["out"], want)
    # tokens past max_q_len are left out: their rows are not written, and the state ends ahead of them
    t["out"].fill_(float("nan"))
    before = _run(bfp8, t, lens, max_q_len=66)
    kept = [min(n, 66) for n in lens]
    rows = np.concatenate([np.arange(k) + sum(lens[:i]) for i, k in enumerate(kept)])
    out = t["out"].clone()
    assert torch.isnan(out[[i for i in range(sum(lens)) if i not in set(rows.tolist())]]).all()
    at = torch.tensor(rows, device=dev)
    short = dict(t, **{k: t[k][at] for k in ("q", "k", "v", "a", "b")}, out=out[at])
    _check(short, kept, before)


def test_strides_of_every_tensor(bfp8, cuda_device):
    """Token-major heads, states with room between heads and slots, gates as columns of a wider matrix."""
    dev, lens = cuda_device, [70, 1, 4]
    t = delta_inputs(dev, lens, 2, 4, 12)
    T = sum(lens)
    for k, h in (("q", 2), ("k", 2), ("v", 4)):      # heads first, tokens inside
        t[k] = t[k].transpose(0, 1).contiguous().transpose(0, 1)
    ab = torch.empty(T, 13, dtype=torch.bfloat16, device=dev)
    ab[:, 1:5], ab[:, 8:12] = t["a"], t["b"]
    t["a"], t["b"] = ab[:, 1:5], ab[:, 8:12]
    pool = torch.randn(t["state"].shape[0], 6, 128 * 128 + 4, device=dev)
    pool[:, 1:5, :128 * 128] = t["state"].view(-1, 4, 128 * 128)
    t["state"] = pool[:, 1:5, :128 * 128].unflatten(2, (128, 128))
    t["out"] = nan_like((4, T, 128), dev).transpose(0, 1)
    spare = pool.clone()
    before = _run(bfp8, t, lens)
    _check(t, lens, before)
    assert torch.equal(pool[:, [0, 5]], spare[:, [0, 5]]) and torch.equal(pool[:, :, 128 * 128:], spare[:, :, 128 * 128:])


@pytest.mark.parametrize("lens", [[3, 3, 3], [70, 90, 70]])
def test_nan_reaches_its_own_request_only(bfp8, cuda_device, lens):
    t = delta_inputs(cuda_device, lens, 1, 2, 13)
    _run(bfp8, t, lens)
    clean, clean_state = t["out"].clone(), t["state"].clone()
    t2 = delta_inputs(cuda_device, lens, 1, 2, 13)
    mid = lens[0] + lens[1] // 2
    t2["v"][mid, 1, 5] = float("nan")
    _run(bfp8, t2, lens)
    for a, b in ((0, lens[0]), (lens[0] + lens[1], sum(lens))):
        assert torch.equal(t2["out"][a:b], clean[a:b])
    assert torch.isnan(t2["out"][mid:lens[0] + lens[1], 1, 5]).all()
    assert torch.equal(t2["out"][:, 0], clean[:, 0])
    dst = t["slots_out"].tolist()
    assert torch.isnan(t2["state"][dst[1], 1, 5]).any()
    for d in (dst[0], dst[2]):
        assert torch.equal(t2["state"][d], clean_state[d])


def test_many_readers_of_one_slot(bfp8, cuda_device):
    """Requests that go on from one shared prefix."""
    lens = [2, 70, 1, 9]
    t = delta_inputs(cuda_device, lens, 1, 2, 14)
    used = set(t["slots_out"].tolist())
    t["slots_in"].fill_(next(i for i in range(t["state"].shape[0]) if i not in used))
    _check(t, lens, _run(bfp8, t, lens))


def test_captured_step_follows_its_inputs(bfp8, cuda_device):
    """Captured once and replayed with other lengths: what a call of those lengths gives, bit for bit."""
    dev = cuda_device
    lens = [80, 0, 3, 1]
    t = delta_inputs(dev, lens, 2, 4, 15)
    T, hv = t["out"].shape[:2]
    ws = torch.empty(bfp8.bfp8_delta_rule_workspace(4, T, T, 2, 4), dtype=torch.uint8, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        bfp8.bfp8_delta_rule(*(t[k] for k in NAMES), T, workspace=ws)
    start = t["state"].clone()
    for lens in ([80, 0, 3, 1], [1, 1, 1, 1], [0, 84, 0, 0], [20, 20, 20, 24], [0, 0, 0, 0]):
        t["q_offsets"].copy_(offsets(dev, lens))
        t["state"].copy_(start)
        t["out"].fill_(float("nan"))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        _check(t, lens, start)
        other = dict(t, state=start.clone(), out=nan_like(t["out"].shape, dev))
        _run(bfp8, other, lens, max_q_len=T)
        assert torch.equal(other["state"], t["state"])
        assert torch.equal(torch.nan_to_num(other["out"]), torch.nan_to_num(t["out"]))


def test_results_do_not_depend_on_the_batch_around(bfp8, cuda_device):
    """A request alone, and among others, with the same max_q_len: the same bits."""
    dev = cuda_device
    lens = [5, 100, 17, 64]
    t = delta_inputs(dev, lens, 2, 4, 16)
    start = t["state"].clone()
    _run(bfp8, t, lens)
    at = 0
    for b, n in enumerate(lens):
        one = dict(t, **{k: t[k][at:at + n] for k in ("q", "k", "v", "a", "b")}, state=start.clone(),
                   slots_in=t["slots_in"][b:b + 1], slots_out=t["slots_out"][b:b + 1], q_offsets=offsets(dev, [n]),
                   out=nan_like((n, 4, 128), dev))
        _run(bfp8, one, [n], max_q_len=max(lens))
        d = t["slots_out"][b]
        assert torch.equal(one["out"], t["out"][at:at + n]) and torch.equal(one["state"][d], t["state"][d])
        at += n


def test_refusals(bfp8, cuda_device):
    dev = cuda_device
    t = delta_inputs(dev, [70, 4], 2, 4, 17)
    ws = torch.empty(bfp8.bfp8_delta_rule_workspace(2, 74, 70, 2, 4) + 256, dtype=torch.uint8, device=dev)

    def call(max_q_len=70, workspace=ws, **kw):
        bfp8.bfp8_delta_rule(*((t | kw)[k] for k in NAMES), max_q_len, workspace=workspace)

    call()
    for bad in (dict(q=t["q"].float()), dict(k=t["k"][:-1]), dict(v=t["v"][:, :3]), dict(a=t["a"].float()), dict(a=t["a"][:, :3]),
                dict(a_log=t["a_log"].double()), dict(a_log=t["a_log"].to(torch.bfloat16)), dict(state=t["state"][:, :3]),
                dict(state=t["state"].transpose(2, 3)), dict(state=t["state"].half()), dict(slots_in=t["slots_in"][:1]),
                dict(out=t["out"].float()), dict(state=None), dict(q=t["q"].cpu())):
        with pytest.raises(ValueError):
            call(**bad)
