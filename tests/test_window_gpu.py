"""Paged decode under a sliding window with sinks (fa_decode_paged_window) against the 64-bit reference of the
paged decode (tests/paged_ref.py, which derives the tolerances) over each row's visible entries.  All that no row
sees holds NaN, and the table entries of pages that no row sees are out of range."""
import numpy as np
import pytest
import torch

import paged_ref as R
from gpu_util import to64
from test_cache_gpu import entries, gen, make_cache, randn, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def visible(n, Tq, t, left, sinks):
    """Slots that row t sees."""
    p = n - Tq + t
    return [j for j in range(p + 1) if left < 0 or j >= p - left or j < sinks]


def attend(q, k, v, scale, group, codes, left, sinks):
    """paged_ref.attend, row by row."""
    Hq, Tq, d = q.shape
    n = k.shape[1]
    o, lse, to, tl = np.zeros_like(q), np.full((Hq, Tq), -np.inf), np.zeros_like(q), np.zeros((Hq, Tq))
    for t in range(Tq):
        at = visible(n, Tq, t, left, sinks)
        if at:
            o[:, t:t + 1], lse[:, t:t + 1], _, to[:, t:t + 1], tl[:, t:t + 1], _ = R.attend(q[:, t:t + 1], k[:, at], v[:, at], scale,
                                                                                       False, group, codes)
    return o, lse, to, tl


def hide(cache, Tq, left, sinks):
    """Puts NaN where no row looks, and gives back (out of range) the pages that no row sees."""
    ps = cache.page_size
    for b in range(cache.B):
        n = int(cache.lens[b])
        seen = np.zeros(-(-n // ps) * ps, dtype=bool)
        for t in range(Tq):
            seen[visible(n, Tq, t, left, sinks)] = True
        for i in range(len(seen) // ps):
            page, mine = int(cache.block_table[b, i]), torch.from_numpy(~seen[i * ps:(i + 1) * ps]).to(DEV)
            for pool in (cache.k, cache.v):
                pool[page, :, mine] = 0x7F if pool.dtype == torch.uint8 else float("nan")
            if mine.all():
                cache.block_table[b, i] = -1 if i % 2 else 1 << 30


CASES = [
    # lens, Hq, Hkv, d, ps, Tq, left, sinks, fp8
    ([1], 1, 1, 64, 16, 1, 0, 0, False),
    ([17, 0, 1, 300], 8, 2, 128, 16, 1, 0, 1, False),
    ([5, 64, 65, 128, 129, 1000, 0], 8, 4, 128, 16, 1, 63, 4, False),
    ([5, 64, 65, 128, 129, 1000, 1], 4, 4, 64, 32, 1, 100, 0, False),
    ([700, 3, 513], 5, 1, 128, 64, 3, 127, 16, False),
    ([700, 3, 513, 2], 16, 1, 256, 128, 16, 40, 5, False),
    ([300, 64, 2000], 7, 7, 256, 256, 2, 255, 300, False),
    ([5000, 40], 48, 3, 128, 64, 7, 1000, 4, False),
    ([100, 2000, 31, 0], 16, 2, 64, 16, 1, 500, 4, True),
    ([100, 2049, 33, 1], 8, 8, 128, 32, 2, 64, 130, True),
    ([700, 19], 12, 3, 256, 16, 5, 30, 1, True),
    ([9001, 1], 64, 1, 128, 256, 1, 4095, 4, False),
    ([40000, 12, 20000], 8, 2, 128, 64, 1, 8191, 4, False),
    ([33000, 700], 8, 1, 64, 16, 4, 20000, 200, True),
    ([600, 601, 17], 80, 1, 128, 32, 1, 400, 33, False),
    ([900, 40], 4, 2, 128, 16, 1, 10 ** 9, 10 ** 9, False),
    ([900, 40], 4, 2, 128, 16, 2, 2 ** 31 - 1, 2 ** 31 - 1, False),
]


@pytest.mark.parametrize("case", CASES)
def test_window(fa, case):
    lens, Hq, Hkv, d, ps, Tq, left, sinks, fp8 = case
    cache = make_cache(fa, 3, lens, Hkv, d, ps, fp8)
    ref = [entries(cache, b) for b in range(cache.B)]
    hide(cache, Tq, left, sinks)
    q = randn(gen(4), cache.B, Hq, Tq, d)
    o, lse = fa.attention_decode_paged(cache, q, d ** -0.5, window=(left, 0), sinks=sinks)
    assert fa.fa_sync_status() == fa.FA_OK
    for b in range(cache.B):
        ro, rl, to, tl = attend(to64(q[b]), *ref[b], d ** -0.5, Hq // Hkv, fp8, left, sinks)
        dead = np.isneginf(rl)
        assert np.array_equal(np.isneginf(to64(lse[b])), dead)
        within(to64(lse[b])[~dead], rl[~dead], tl[~dead])
        within(to64(o[b]), ro, to, 2.0 ** -8)


@pytest.mark.parametrize("seed", range(12))
def test_many_lengths(fa, seed):
    """Batches of drawn lengths and windows: whole units and shares."""
    rng = np.random.default_rng(seed)
    d, ps, Hkv = int(rng.choice([64, 128])), int(rng.choice([16, 64])), int(rng.choice([1, 3]))
    G, Tq, fp8 = int(rng.choice([1, 4, 9])), int(rng.choice([1, 2])), bool(rng.random() < 0.4)
    B, left, sinks = int(rng.integers(1, 40)), int(rng.integers(0, 3000)), int(rng.choice([0, 4, 70]))
    lens = [int(x) for x in rng.integers(0, 6000, B)]
    test_window(fa, (lens, Hkv * G, Hkv, d, ps, Tq, left, sinks, fp8))


@pytest.mark.parametrize("B,Hkv,d,fp8,lens", [
    (64, 8, 128, False, "ragged"), (50, 8, 128, False, "ragged"), (33, 10, 128, True, "equal"), (20, 12, 256, False, "ragged"),
    (64, 8, 64, True, "one"), (63, 6, 64, False, "few"), (110, 4, 128, False, "ragged"), (128, 3, 128, False, "few"),
    (140, 3, 128, False, "ragged"),
])
def test_more_units_than_start_at_once(fa, B, Hkv, d, fp8, lens):
    """They are taken in order of length, each of them once."""
    rng = np.random.default_rng(B)
    lens = {"ragged": rng.integers(0, 1500, B), "equal": np.repeat([1, 400], B)[:B], "one": np.where(np.arange(B) == 40, 1200, 3),
            "few": np.where(rng.random(B) < 0.3, 700, rng.integers(0, 40, B))}[lens]
    test_window(fa, ([int(x) for x in lens], Hkv, Hkv, d, 16, 1, 900, 4, fp8))


def test_no_left_bound_is_the_whole_cache(fa):
    cache = make_cache(fa, 5, [900, 33], 2, 128, 16)
    q = randn(gen(6), 2, 8, 2, 128)
    want = fa.attention_decode_paged(cache, q, 0.1)
    got = fa.attention_decode_paged(cache, q, 0.1, window=(-1, 0), sinks=3)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    got = fa.attention_decode_paged(cache, q, 0.1, sinks=3)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_far_sequences(fa):
    """Slots up to 2^30 in the table, of which the window's few pages exist."""
    ps, n = 256, (1 << 30) - 300
    table = torch.full((1, 1 << 22), -1, dtype=I32, device=DEV)
    pages = 7
    k, v = (randn(gen(7 + i), pages, 1, ps, 64) for i in range(2))
    table[0, 0] = 6
    last = (n - 1) // ps
    table[0, last - 5:last + 1] = torch.arange(6, dtype=I32, device=DEV)
    cache = fa.KVCache(k, v, table, torch.tensor([n], dtype=I32, device=DEV))
    q = randn(gen(9), 1, 2, 3, 64)
    o, lse = fa.attention_decode_paged(cache, q, 0.125, window=(900, 0), sinks=4)
    assert fa.fa_sync_status() == fa.FA_OK
    first = (last - 5) * ps
    kk, vv = (np.concatenate([to64(x[6, :, :4]), to64(x[:6]).transpose(1, 0, 2, 3).reshape(1, -1, 64)[:, :n - first]], 1) for x in (k, v))
    qq = to64(q[0])
    for t in range(3):
        p = n - 3 + t
        at = [0, 1, 2, 3] + [4 + j - first for j in range(p - 900, p + 1)]
        ro, rl, _, to, tl, _ = R.attend(qq[:, t:t + 1], kk[:, at], vv[:, at], 0.125, False, 2)
        within(to64(o[0, :, t:t + 1]), ro, to, 2.0 ** -8)
        within(to64(lse[0, :, t:t + 1]), rl, tl)


def test_both_ways_captured_and_shared_workspace(fa):
    """The compiled checks and the others; two captured graphs that share a workspace, replayed with other lengths."""
    cache = make_cache(fa, 10, [3000, 700, 40], 2, 128, 16, width=200, garbage=False)
    q = randn(gen(11), 3, 8, 1, 128)
    o, o2, lse, lse2 = torch.empty_like(q), torch.empty_like(q), torch.empty((3, 8, 1), device=DEV), torch.empty((3, 8, 1), device=DEV)
    ws = torch.empty(fa.fa_decode_paged_window_workspace_bytes(cache, 8), dtype=torch.uint8, device=DEV)
    fa.fa_decode_paged_window(cache, q, o, lse, 600, 4, 0.1, ws)
    fa._decode_window(cache, q, o2, lse2, 600, 4, 0.1, ws, None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if fa._fa_py is not None:
        call = fa._fa_py.decode_window
        assert call(cache._ref, cache._index, q, o, lse, 600, 4, 0.1, ws, None) == fa.FA_OK
        assert call(cache._ref, cache._index, q, o, lse.half(), 600, 4, 0.1, ws, None) is None
        assert call(cache._ref, cache._index, q, o, lse, 600.5, 4, 0.1, ws, None) is None
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for left, out in ((600, (o, lse)), (90, (o2, lse2))):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.fa_decode_paged_window(cache, q, *out, left, 4, 0.1, ws)
        graphs.append(graph)
    full = [3000, 700, 40]
    for cut in (0, 13, 39):
        cache.lens.copy_(torch.tensor([n - cut for n in full], dtype=I32))
        for graph in graphs:
            graph.replay()
        for left, out in ((600, (o, lse)), (90, (o2, lse2))):
            want = fa.attention_decode_paged(cache, q, 0.1, window=(left, 0), sinks=4)
            assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])
    assert fa.fa_sync_status() == fa.FA_OK


def test_without_slots_pages_or_entries(fa):
    """Tables without a slot, pools without a page, batches without an entry or a sequence: zeros, whatever the
    workspace held."""
    for pages, width, lens in ((0, 0, [0, 0]), (0, 3, [0, 0]), (4, 0, [0]), (4, 2, [0, 0, 0]), (4, 700, [0] * 70), (4, 2, [])):
        k = torch.zeros((pages, 2, 16, 64), dtype=BF16, device=DEV)
        cache = fa.KVCache(k, k.clone(), torch.zeros((len(lens), width), dtype=I32, device=DEV), torch.tensor(lens, dtype=I32, device=DEV))
        q = randn(gen(1), len(lens), 4, 2, 64)
        o, lse = torch.full_like(q, 7), torch.full(q.shape[:3], 7.0, device=DEV)
        for fill in (0, 255):
            ws = torch.full((max(fa.fa_decode_paged_window_workspace_bytes(cache, 4, 2), 256),), fill, dtype=torch.uint8, device=DEV)
            fa.fa_decode_paged_window(cache, q, o.fill_(7), lse.fill_(7), 3, 4, 0.1, ws)
            assert fa.fa_sync_status() == fa.FA_OK and torch.all(o == 0) and torch.all(lse == -np.inf)
        none = torch.zeros(0, dtype=I32, device=DEV)
        ws = torch.zeros(max(fa.fa_decode_paged_shared_workspace_bytes(cache, 4, 2, none), 256), dtype=torch.uint8, device=DEV)
        fa.fa_decode_paged_shared(cache, q, o.fill_(7), lse.fill_(7), none, 0.1, ws)
        assert fa.fa_sync_status() == fa.FA_OK and torch.all(o == 0) and torch.all(lse == -np.inf)


def test_bad_lengths_and_pages(fa):
    cache = make_cache(fa, 12, [500, 500, 500, 500], 2, 64, 16)
    q = randn(gen(13), 4, 4, 1, 64)
    want = fa.attention_decode_paged(cache, q, 0.1, window=(99, 0), sinks=4)
    cache.lens[0] = -1
    cache.lens[1] = cache.max_pages * 16 + 1
    cache.block_table[2, 5] = -7                 # not seen
    cache.block_table[3, 30] = cache.num_pages   # slots 480 .. 495
    got = fa.attention_decode_paged(cache, q, 0.1, window=(99, 0), sinks=4)
    assert fa.fa_sync_status() == fa.FA_ERR_BAD_INDEX
    assert torch.all(got[0][:2] == 0) and torch.all(got[1][:2] == -np.inf)
    assert torch.equal(got[0][2], want[0][2]) and torch.isfinite(got[0][3].float()).all() and not torch.equal(got[0][3], want[0][3])
    assert fa.fa_sync_status() == fa.FA_OK


def test_refusals(fa):
    cache = make_cache(fa, 14, [50], 1, 64, 16)
    q = randn(gen(15), 1, 2, 1, 64)
    o, lse = torch.empty_like(q), torch.empty((1, 2, 1), device=DEV)
    ws = torch.empty(fa.fa_decode_paged_window_workspace_bytes(cache, 2), dtype=torch.uint8, device=DEV)
    for left, sinks in ((-2, 0), (5, -1)):
        with pytest.raises(fa.FAError):
            fa.fa_decode_paged_window(cache, q, o, lse, left, sinks, 0.1, ws)
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged_window(cache, q, o, lse, 5, 0, 0.1, ws[:-256])
    with pytest.raises(TypeError):
        fa.fa_decode_paged_window(cache, q.float(), o, lse, 5, 0, 0.1, ws)
    for bad in (dict(window=(5, 1)), dict(window=(5, 0), causal=False), dict(window=(5, 0), accumulate=True), dict(sinks=2, causal=False)):
        with pytest.raises(ValueError):
            fa.attention_decode_paged(cache, q, 0.1, **bad)
    assert fa.fa_sync_status() == fa.FA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_outside_the_buffers(fa, fp8):
    """Guard bands around o, lse and the workspace."""
    lens, Hq, Hkv, d = [3000, 70, 0], 10, 2, 128
    cache = make_cache(fa, 16, lens, Hkv, d, 16, fp8)
    q = randn(gen(17), 3, Hq, 1, d)
    n, nb = q.numel(), fa.fa_decode_paged_window_workspace_bytes(cache, Hq)
    ob, lb, wb = torch.full((n + 512,), 7.0, dtype=BF16, device=DEV), torch.full((3 * Hq + 128,), 7.0, device=DEV), \
        torch.full((nb + 512,), 7, dtype=torch.uint8, device=DEV)
    o, lse = ob[256:256 + n].view(q.shape), lb[64:64 + 3 * Hq].view(3, Hq, 1)
    fa.fa_decode_paged_window(cache, q, o, lse, 900, 4, 0.1, wb[256:256 + nb])
    want = fa.attention_decode_paged(cache, q, 0.1, window=(900, 0), sinks=4)
    assert fa.fa_sync_status() == fa.FA_OK and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for t, a, b in ((ob, 256, n), (lb, 64, 3 * Hq), (wb, 256, nb)):
        assert torch.all(t[:a] == 7) and torch.all(t[a + b:] == 7)
