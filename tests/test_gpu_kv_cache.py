"""bfp8_kv_plan and bfp8_kv_append on the GPU against the oracle: whole numbers
and codes are equal, to the last one.
"""

import numpy as np
import pytest
import torch

from gpu_util import dec_e4m3
from oracle import kv as KV

pytestmark = pytest.mark.gpu

D = 128


# ---- block plan ---------------------------------------------------------------


def _plan(bfp8, dev, ctx, new, free, table, page, capacity, pitch=None):
    B, width = np.asarray(table).shape
    wide = torch.full((B, pitch or width), -7, dtype=torch.int32, device=dev)
    t = wide[:, :width]
    t.copy_(torch.tensor(np.asarray(table), dtype=torch.int32))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)   # noqa: E731
    out = dict(q_offsets=torch.full((B + 1,), -9, dtype=torch.int32, device=dev),
               kv_len=torch.full((B,), -9, dtype=torch.int32, device=dev),
               slots=torch.full((capacity,), -9, dtype=torch.int64, device=dev),
               positions=torch.full((capacity,), -9, dtype=torch.int32, device=dev),
               counts=torch.full((3,), -9, dtype=torch.int32, device=dev))
    args = (i32(ctx), i32(new), i32(free), t, page, *out.values())
    for _ in range(2):   # a repeated call changes nothing
        bfp8.bfp8_kv_plan(*args)
    torch.cuda.synchronize()
    assert bool((wide[:, width:] == -7).all())
    return [t.cpu().numpy()] + [v.cpu().numpy() for v in out.values()]


def _check_plan(bfp8, dev, ctx, new, free, table, page, capacity, pitch=None):
    got = _plan(bfp8, dev, ctx, new, free, table, page, capacity, pitch)
    want = KV.block_plan(ctx, new, free, table, page, capacity)
    for name, g, w in zip(("table", "q_offsets", "kv_len", "slots", "positions", "counts"), got, want):
        assert np.array_equal(g, np.asarray(w)), name


def _random_plan(rng, B, page, q_hi, ctx_hi, width=None):
    ctx, new = rng.integers(0, ctx_hi + 1, B), rng.integers(0, q_hi + 1, B)
    before, after = -(-ctx // page), -(-(ctx + new) // page)
    perm = rng.permutation(int(after.sum()) + 5)
    table = np.full((B, width or max(1, int(after.max()))), -1)
    k = 0
    for b in range(B):
        n = min(before[b], table.shape[1])
        table[b, :n] = perm[k:k + n]
        k += before[b]
    return ctx, new, perm[k:], table


@pytest.mark.parametrize("B,page,q_hi,ctx_hi", [(1, 16, 1, 0), (1, 64, 949, 300), (64, 64, 1, 5000), (33, 128, 300, 7),
                                                (511, 16, 40, 200), (513, 32, 3, 1000), (2050, 16, 9, 90)])
def test_plan_matches_oracle(bfp8, cuda_device, B, page, q_hi, ctx_hi):
    rng = np.random.default_rng(B * page)
    ctx, new, free, table = _random_plan(rng, B, page, q_hi, ctx_hi)
    total = int(new.sum())
    _check_plan(bfp8, cuda_device, ctx, new, free, table, page, total + 37, pitch=table.shape[1] + 3)
    _check_plan(bfp8, cuda_device, ctx, new, free, table, page, max(1, total // 2))   # capacity below the tokens


def test_plan_edges(bfp8, cuda_device):
    dev = cuda_device
    rng = np.random.default_rng(7)
    ctx, new, free, table = _random_plan(rng, 40, 32, 200, 300)
    _check_plan(bfp8, dev, ctx, new, free[:60], table, 32, int(new.sum()))            # the free list runs out
    _check_plan(bfp8, dev, ctx, new, free, table[:, :5], 32, int(new.sum()))          # the table is too narrow
    _check_plan(bfp8, dev, ctx, new, free[:0], table, 32, int(new.sum()))             # no free page at all
    _check_plan(bfp8, dev, ctx, 0 * new, free, table, 32, 4)                          # nothing new
    _check_plan(bfp8, dev, [-3, 5], [4, -2], [1, 2], [[-1, -1], [6, -1]], 16, 8)      # negative lengths count as 0
    _check_plan(bfp8, dev, [5], [3], [1], [[-1, -1]], 16, 8)                          # a held page that is not there
    # slots past 32 bits
    big = 2 ** 31 - 2
    _check_plan(bfp8, dev, [0, 100], [300, 5], [big, big - 1, big - 2, 3], [[-1] * 4, [big - 5, -1, -1, -1]], 128, 310)


def test_plan_of_the_most_requests(bfp8, cuda_device):
    """16,384 requests, whose prefixes take 128 KB of a block's shared memory; one more is refused."""
    rng = np.random.default_rng(13)
    ctx, new, free, table = _random_plan(rng, 16384, 16, 3, 40)
    _check_plan(bfp8, cuda_device, ctx, new, free, table, 16, int(new.sum()) + 5)
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):
        _plan(bfp8, cuda_device, [0] * 16385, [0] * 16385, [1], [[-1]] * 16385, 16, 4)


def test_plan_of_no_requests(bfp8, cuda_device):
    dev = cuda_device
    e = lambda *s: torch.empty(*s, dtype=torch.int32, device=dev)   # noqa: E731
    off, counts, slots = e(1), e(3), torch.zeros(5, dtype=torch.int64, device=dev)
    pos = e(5)
    bfp8.bfp8_kv_plan(e(0), e(0), e(0), e(0, 4), 16, off, e(0), slots, pos, counts)
    assert off.tolist() == [0] and counts.tolist() == [0, 0, 0] and slots.tolist() == [-1] * 5 and pos.tolist() == [-1] * 5


def test_plan_counts_tokens_of_missing_held_pages(bfp8, cuda_device):
    """Tokens that continue a page whose table entry is -1 have no page, and are counted: after a step
    that ran out of pages, the next one says how many tokens it loses."""
    for page, ctx, new, free, table, lost in [
            (16, [5], [3], [1], [[-1, -1]], 3),                       # all of them
            (16, [5], [20], [1], [[-1, -1]], 11),                     # the rest of that page; the next is new
            (16, [5, 16, 0, 31], [1, 2, 4, 9], [7, 8, 9], [[-1, -1, -1]] * 4, 2),   # requests 0 and 3, one each
            (32, [40, 64, 33], [5, 0, 1], [3], [[2, -1, -1], [4, -1, -1], [6, 5, -1]], 5),
            (16, [5], [3], [], [[4]], 0)]:
        got = _plan(bfp8, cuda_device, ctx, new, free, table, page, sum(new) + 3)
        assert got[-1][2] == lost, (page, ctx, got[-1])
        assert int((got[3][:sum(new)] < 0).sum()) == lost
        _check_plan(bfp8, cuda_device, ctx, new, free, table, page, sum(new) + 3)
    rng = np.random.default_rng(12)
    ctx, new, free, table = _random_plan(rng, 700, 16, 30, 100)
    table[rng.random(table.shape) < 0.3] = -1
    _check_plan(bfp8, cuda_device, ctx, new, free[:200], table, 16, int(new.sum()))
    got = _plan(bfp8, cuda_device, ctx, new, free[:200], table, 16, int(new.sum()))
    assert int((got[3] < 0).sum()) == got[-1][2]


# ---- append ------------------------------------------------------------------


def _cache(dev, P, H, page, rng, order="heads"):
    """Random codes (finite) and scale bytes; `order`: which of heads and tokens is outer in memory."""
    def codes():
        c = rng.integers(0, 256, (P, H, page, D)).astype(np.uint8)
        c[(c & 127) == 127] = 0x30
        t = torch.from_numpy(c).to(dev)
        return t if order == "heads" else t.transpose(1, 2).contiguous().transpose(1, 2)

    def exps():
        return torch.from_numpy(rng.integers(115, 126, (P, H)).astype(np.uint8)).to(dev)

    return codes(), codes(), exps(), exps()


def _kv(dev, T, H, rng, spread=1.0):
    x = rng.normal(size=(T, 2, H, D)) * np.exp2(rng.uniform(-spread, spread, (T, 2, H, 1)) * 3)
    kv = torch.from_numpy(x.astype(np.float32)).to(dev).to(torch.bfloat16)
    return kv[:, 0], kv[:, 1]


def _check_append(bfp8, dev, k, v, slots, cache):
    kc, vc, ke, ve = cache
    want = [KV.append(x.double().cpu().numpy(), slots, c.cpu().numpy(), e.cpu().numpy())
            for x, c, e in ((k, kc, ke), (v, vc, ve))]
    bfp8.bfp8_kv_append(k, v, torch.tensor(np.asarray(slots), dtype=torch.int64, device=dev), kc, vc, ke, ve)
    torch.cuda.synchronize()
    for name, (wc, we), c, e in (("k", want[0], kc, ke), ("v", want[1], vc, ve)):
        assert np.array_equal(e.cpu().numpy(), we), name + " scales"
        got = c.cpu().numpy()
        nan = np.isnan(dec_e4m3(wc))
        assert np.array_equal(np.isnan(dec_e4m3(got)), nan), name + " NaN codes"
        assert np.array_equal(got[~nan], wc[~nan]), name + " codes"


def _slots(rng, page, lengths, P):
    """Runs of (held, new) tokens in pages of their own, in order."""
    pages, out = rng.permutation(P), []
    k = 0
    for held, new in lengths:
        for i in range(held, held + new):
            out.append(int(pages[k + i // page]) * page + i % page)
        k += -(-(held + new) // page)
    return out, k


@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("H", [1, 8])
def test_append_matches_oracle(bfp8, cuda_device, page, H, order):
    rng = np.random.default_rng(page + H)
    lengths = [(0, 1), (3, 1), (page - 1, 1), (page - 1, 2), (5, page), (0, page), (0, 2 * page + 3), (page, 1),
               (7, 3 * page + 1), (0, 0), (1, page - 1)]
    slots, used = _slots(rng, page, lengths, 40)
    k, v = _kv(cuda_device, len(slots), H, rng)
    _check_append(bfp8, cuda_device, k, v, slots, _cache(cuda_device, 40, H, page, rng, order))


def test_append_many_tokens(bfp8, cuda_device):
    """Enough rows that a warp takes a window of several, runs crossing the windows' ends."""
    rng = np.random.default_rng(11)
    lengths = [(int(rng.integers(0, 70)), int(rng.integers(1, 400))) for _ in range(24)]
    slots, used = _slots(rng, 64, lengths, 300)
    k, v = _kv(cuda_device, len(slots), 4, rng)
    _check_append(bfp8, cuda_device, k, v, slots, _cache(cuda_device, 300, 4, 64, rng))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_many_short_runs(bfp8, cuda_device, page):
    """More (token, head) pairs than warps: runs of one row, of a few and of a page, dealt out and shared."""
    rng = np.random.default_rng(page)
    lengths = [(int(rng.integers(0, page)), 1) for _ in range(500)]
    lengths += [(int(rng.integers(0, page)), int(rng.integers(2, 2 * page))) for _ in range(20)]
    lengths = [lengths[i] for i in rng.permutation(len(lengths))]
    slots, used = _slots(rng, page, lengths, 700)
    k, v = _kv(cuda_device, len(slots), 6, rng)
    _check_append(bfp8, cuda_device, k, v, slots, _cache(cuda_device, 700, 6, page, rng))


def test_append_skips_rows_and_repeats(bfp8, cuda_device):
    rng = np.random.default_rng(3)
    dev, cache = cuda_device, _cache(cuda_device, 6, 2, 16, rng)
    slots = [-1, 5, 6, -1, 96, 2 ** 40, 17, 18, -1]     # 96 = the first slot past the cache
    k, v = _kv(dev, len(slots), 2, rng)
    _check_append(bfp8, dev, k, v, slots, cache)
    before = [t.clone() for t in cache]
    bfp8.bfp8_kv_append(k, v, torch.tensor(slots, device=dev), *cache)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))
    bfp8.bfp8_kv_append(k[:0], v[:0], torch.empty(0, dtype=torch.int64, device=dev), *cache)
    assert all(torch.equal(a, b) for a, b in zip(before, cache))


def test_append_extremes(bfp8, cuda_device):
    """Zeros, values past both ends of the scales' range, infinities and NaN; scales that grow far."""
    rng = np.random.default_rng(4)
    T, H = 12, 2
    k, v = _kv(cuda_device, T, H, rng)
    k, v = k.contiguous(), v.contiguous()
    k[0] = 0
    v[0] = 1e-38
    k[1] *= 1e36
    k[2, 0, 5] = float("inf")
    k[2, 1, 6] = float("nan")
    v[3, 0] = float("nan")
    v[4, 1, :3] = torch.tensor([448.0, -449.0, 3.0e38], device=cuda_device)
    v[5] = -0.0
    k[6] *= 2.0 ** -30
    slots = [16 * i + (0 if i < 6 else 3) for i in range(T)]
    _check_append(bfp8, cuda_device, k, v, slots, _cache(cuda_device, T, H, 16, rng))


def test_append_reads_strided_rows(bfp8, cuda_device):
    """Columns of a wider projection's rows, every second token, heads apart."""
    rng = np.random.default_rng(5)
    wide = torch.from_numpy(rng.normal(size=(20, 9, 136)).astype(np.float32)).to(cuda_device).to(torch.bfloat16)
    k, v = wide[::2, 0:6:2, 8:], wide[1::2, 1:7:2, :128]
    _check_append(bfp8, cuda_device, k, v, list(range(100, 110)), _cache(cuda_device, 9, 3, 32, rng))


def test_append_in_a_cache_past_32_bits(bfp8, cuda_device):
    """Pages whose byte offsets need more than 32 bits."""
    P, H, page = 140000, 8, 32                       # 4.6 GB of codes
    rng = np.random.default_rng(6)
    kc = torch.zeros(P, H, page, D, dtype=torch.uint8, device=cuda_device)
    vc = torch.zeros_like(kc)
    ke = torch.full((P, H), 120, dtype=torch.uint8, device=cuda_device)
    ve = ke.clone()
    pages = [0, 65536, 131072, P - 1]
    slots = [p * page + i for p in pages for i in range(3)]
    k, v = _kv(cuda_device, len(slots), H, rng)
    bfp8.bfp8_kv_append(k, v, torch.tensor(slots, device=cuda_device), kc, vc, ke, ve)
    small = [s % page + i // 3 * page for i, s in enumerate(slots)]
    zeros, e0 = np.zeros((4, H, page, D), np.uint8), np.full((4, H), 120, np.uint8)
    for x, c, e in ((k, kc, ke), (v, vc, ve)):
        wc, we = KV.append(x.double().cpu().numpy(), small, zeros, e0)
        assert np.array_equal(c[pages].cpu().numpy(), wc) and np.array_equal(e[pages].cpu().numpy(), we)


def test_refusals(bfp8, cuda_device):
    dev, rng = cuda_device, np.random.default_rng(8)
    kc, vc, ke, ve = _cache(dev, 4, 2, 16, rng)
    k, v = _kv(dev, 3, 2, rng)
    slots = torch.tensor([0, 1, 2], device=dev)
    with pytest.raises(ValueError, match="shape"):
        bfp8.bfp8_kv_append(k[:, :1], v, slots, kc, vc, ke, ve)
    with pytest.raises(ValueError, match="bfloat16"):
        bfp8.bfp8_kv_append(k.float(), v, slots, kc, vc, ke, ve)
    with pytest.raises(ValueError, match="int64"):
        bfp8.bfp8_kv_append(k, v, slots.int(), kc, vc, ke, ve)
    with pytest.raises(ValueError, match="k_exp"):
        bfp8.bfp8_kv_append(k, v, slots, kc, vc, ke[:2], ve)
    with pytest.raises(ValueError, match="same strides"):
        bfp8.bfp8_kv_append(k, v, slots, kc, vc, ke, ve.t().contiguous().t())
    with pytest.raises(ValueError, match="contiguous codes"):
        bfp8.bfp8_kv_append(k, v, slots, kc.transpose(2, 3).contiguous().transpose(2, 3), vc, ke, ve)
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):      # page size 8
        bfp8.bfp8_kv_append(k, v, slots, kc[:, :, :8], vc[:, :, :8], ke, ve)
    odd = torch.zeros(3, 2, 132, dtype=torch.bfloat16, device=dev)[:, :, 4:]
    with pytest.raises(bfp8.Bfp8Error, match="UNSUPPORTED"):      # rows not 16-byte aligned
        bfp8.bfp8_kv_append(odd, v, slots, kc, vc, ke, ve)
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=dev)   # noqa: E731
    table = torch.zeros(2, 3, dtype=torch.int32, device=dev)
    good = (i32(2), i32(2), i32(4), table, 16, i32(3), i32(2), slots, i32(3), i32(3))
    bfp8.bfp8_kv_plan(*good)
    for at, bad, err in [(4, 24, bfp8.Bfp8Error), (5, i32(2), ValueError), (0, i32(3), ValueError),
                         (7, slots.int(), ValueError), (9, i32(2), ValueError), (3, table.t(), ValueError)]:
        with pytest.raises(err):
            bfp8.bfp8_kv_plan(*good[:at], bad, *good[at + 1:])


def test_entry_points_refuse_host_memory(bfp8, cuda_device):
    import ctypes
    lib, d = bfp8._lib, torch.zeros(1 << 16, dtype=torch.uint8, device=cuda_device).data_ptr()
    h = torch.zeros(1 << 16, dtype=torch.uint8).data_ptr()
    cache = lambda k: ctypes.byref(bfp8.bfp8_kv_cache(k, d, d, d, 1, 16, 1, 128, 2048, 2048, 128, 2048, 2048, 128, 1, 1))  # noqa: E731
    for args in [(h, 128, 128, d, 128, 128, d, 1, cache(d), None), (d, 128, 128, d, 128, 128, h, 1, cache(d), None),
                 (d, 128, 128, d, 128, 128, d, 1, cache(h), None)]:
        assert bfp8.bfp8_status_string(lib.bfp8_kv_append(*args)) == "INVALID_ARG"
    assert bfp8.bfp8_status_string(lib.bfp8_kv_plan(d, d, 1, d, 4, h, 4, 4, 16, d, d, d, d, 4, d, None)) == "INVALID_ARG"


def test_append_on_another_stream_and_in_a_graph(bfp8, cuda_device):
    rng = np.random.default_rng(9)
    slots, _ = _slots(rng, 32, [(3, 40), (0, 5)], 8)
    k, v = _kv(cuda_device, len(slots), 2, rng)
    cache = _cache(cuda_device, 8, 2, 32, rng)
    twin = [t.clone() for t in cache]
    s = torch.tensor(slots, device=cuda_device)
    bfp8.bfp8_kv_append(k, v, s, *twin)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bfp8.bfp8_kv_append(k, v, s, *cache)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(cache, twin))
