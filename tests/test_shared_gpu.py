"""Paged decode of a batch that shares a prefix (fa_decode_paged_shared) against the 64-bit reference of the paged
decode.  The library computes the prefix by itself where its estimate says that this is faster; the test library
(built with FA_TEST_WITHHOLD) always does, and small cases run through it.  Tolerances as in tests/paged_ref.py, and 2^-8 of each probability of a prefix's entry, which meets
its v as bf16: 2^-8 sum p |v| over the prefix."""
import ctypes

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


@pytest.fixture(scope="module")
def always(fa):
    from exact_io_aware_05_gb300 import build
    build.build(test_variant=True)
    lib = ctypes.CDLL(build.TEST_SO)
    for name in ("fa_decode_paged_shared", "fa_sync_status"):
        getattr(lib, name).argtypes = getattr(fa.lib(), name).argtypes
    return lib


def call(fa, lib, cache, q, pages, scale, causal=True, ws=None):
    """o, lse and the workspace of a call; lib None: through the package."""
    B, Hq, Tq, _ = q.shape
    if ws is None:
        ws = torch.full((fa.fa_decode_paged_shared_workspace_bytes(cache, Hq, Tq, pages),), 255, dtype=torch.uint8, device=DEV)
    if lib is None:
        o, lse = fa.attention_decode_paged(cache, q, scale, causal=causal, prefix_pages=pages, workspace=ws)
        return o, lse, ws
    o, lse = torch.empty_like(q), torch.empty(q.shape[:3], device=DEV)
    assert lib.fa_decode_paged_shared(cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, Tq, int(causal), pages.data_ptr(),
                                      pages.numel(), scale, ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream) == 0
    return o, lse, ws


def status(fa, lib):
    return fa.fa_sync_status() if lib is None else lib.fa_sync_status(torch.cuda.current_stream().cuda_stream)


def shared_cache(fa, seed, P, tails, Hkv, d, ps, fp8=False, **kw):
    """A cache whose sequences share P entries; tails: entries behind them, or, negative, the whole length (< P) as
    -1 - length.  Table entries of pages that a sequence does not reach stay out of range."""
    lens = [P + x if x >= 0 else -1 - x for x in tails]
    cache = make_cache(fa, seed, lens + [P], Hkv, d, ps, fp8, **kw)   # one more sequence, that owns the prefix
    pages = cache.block_table[-1, :P // ps].clone()
    for b, n in enumerate(lens):
        m = min(P, -(-n // ps) * ps) // ps
        cache.block_table[b, :m] = pages[:m]
    c = fa.KVCache(cache.k, cache.v, cache.block_table[:-1].contiguous(), cache.lens[:-1].contiguous(), cache.k_scale, cache.v_scale)
    return c, pages


def check(fa, lib, cache, pages, P, Hq, Tq, causal=True, seed=2, scale=None, sequences=None, q_scale=1.0, joined=True):
    """joined: the prefix is to be computed by itself, and so its states lie in the workspace behind the paged
    decode's part."""
    d = cache.d
    scale = d ** -0.5 if scale is None else scale
    q = (randn(gen(seed), cache.B, Hq, Tq, d, dtype=F32) * q_scale).to(BF16)
    o, lse, ws = call(fa, lib, cache, q, pages, scale, causal)
    assert status(fa, lib) == fa.FA_OK
    assert joined == bool((ws[fa.fa_decode_paged_workspace_bytes(cache, Hq, Tq) + 256:] != 255).any())
    G = Hq // cache.Hkv
    for b in (range(cache.B) if sequences is None else sequences):
        k, v = entries(cache, b)
        qq = to64(q[b])
        ro, rl, _, to, tl, _ = R.attend(qq, k, v, scale, causal, G, cache.k_scale is not None)
        n = k.shape[1]
        for h in range(Hq):   # the prefix's probabilities in bf16
            for t in range(Tq):
                m = min(P, max(0, n - Tq + t + 1) if causal else n)
                if m and np.isfinite(rl[h, t]):
                    p = np.exp(scale * (k[h // G, :m] @ qq[h, t]) - rl[h, t])
                    to[h, t] += 2.0 ** -8 * (p @ np.abs(v[h // G, :m]))
        dead = np.isneginf(rl)
        assert np.array_equal(np.isneginf(to64(lse[b])), dead)
        within(to64(lse[b])[~dead], rl[~dead], tl[~dead])
        within(to64(o[b]), ro, to, 2.0 ** -8)
    return q, o, lse


SMALL = [
    # P, tails, Hq, Hkv, d, ps, Tq, causal, fp8
    (16, [1], 1, 1, 64, 16, 1, True, False),
    (128, [1, 2, 17], 4, 1, 128, 16, 1, True, False),
    (256, [5, 0, 300, -1, -101], 8, 2, 128, 16, 1, True, False),         # one at its end, one empty, one of 100
    (208, [5, 3, 40], 6, 2, 64, 16, 3, True, False),                     # a tile that ends in the prefix's last page
    (512, [5, 3, 40, 1], 16, 2, 256, 256, 1, True, False),
    (96, [1, 7], 32, 1, 256, 32, 16, True, False),
    (1024, list(range(1, 41)), 8, 1, 128, 64, 1, True, False),           # 320 rows: two blocks, the second with one tile
    (640, list(range(1, 10)), 16, 1, 64, 128, 2, True, False),
    (384, [0, 1, 2, 3, -384, -383], 4, 2, 128, 128, 4, True, False),     # rows that end inside the prefix
    (384, [0, 1, 2, 3, -384, -383], 4, 2, 128, 128, 4, False, False),
    (4096, [100, 3], 5, 5, 128, 16, 1, True, False),
    (256, [5, 0, 300, -1, -101], 8, 2, 128, 16, 1, True, True),
    (208, [5, 3, 40], 6, 2, 64, 16, 3, True, True),
    (512, [5, 3, 40, 1], 16, 2, 256, 256, 1, False, True),
    (1024, list(range(1, 41)), 8, 1, 128, 64, 1, True, True),
    (3008, [20, 500], 64, 2, 64, 16, 2, True, True),
    (8192, [77], 4, 1, 256, 64, 1, True, True),
    (64, [1] * 130, 1, 1, 64, 64, 1, True, False),
    (96, [700, 20, 1500], 80, 1, 128, 32, 2, True, False),               # own entries in several row blocks, split over CTAs
    (160, [3000, 9, 0, 4000], 4, 2, 64, 32, 1, True, True),
]
LARGE = [   # sizes at which the library computes the prefix by itself
    (208, [5, 3, 40, 0] * 20, 6, 6, 128, 16, 1, True, False),
    (20000 // 32 * 32, [900, 31, 0, 1, 1], 12, 3, 64, 32, 1, True, False),
    (192, [1] * 130, 8, 8, 64, 64, 1, True, False),
    (4096, [5, 0, 9, 1, 1, 1, 1, 1], 4, 4, 256, 32, 1, True, False),
    (4096, [5, 0, 9, 100, -7, 1, 1, 1, 1, 1, 1, 1] * 2, 8, 4, 128, 64, 1, True, True),
    (8192, [5, 0, 9, 100, -7, 1, 1, 1, 1, 1, 1, 1] * 2, 4, 4, 64, 16, 1, False, True),
    (4096, [3, 0, 0, 1, 1, 1, 1, 1], 4, 4, 256, 256, 1, True, True),
    (2048, [3], 24, 3, 128, 16, 7, True, False),                         # many rows of one sequence
    (2048, [3, 900], 32, 2, 64, 32, 4, True, True),
]


@pytest.mark.parametrize("case", SMALL)
def test_shared_small(fa, always, case):
    P, tails, Hq, Hkv, d, ps, Tq, causal, fp8 = case
    cache, pages = shared_cache(fa, 3, P, tails, Hkv, d, ps, fp8)
    check(fa, always, cache, pages, P, Hq, Tq, causal)


@pytest.mark.parametrize("case", LARGE)
def test_shared(fa, case):
    P, tails, Hq, Hkv, d, ps, Tq, causal, fp8 = case
    cache, pages = shared_cache(fa, 3, P, tails, Hkv, d, ps, fp8)
    check(fa, None, cache, pages, P, Hq, Tq, causal, sequences=range(min(len(tails), 12)))


@pytest.mark.parametrize("d,fp8", [(64, False), (128, False), (256, False), (128, True)])
def test_large_scores(fa, always, d, fp8):
    """Maxima that grow along the prefix by far more than the rescale's threshold."""
    cache, pages = shared_cache(fa, 4, 2048, [40, 3, 0], 2, d, 16, fp8)
    if not fp8:
        cache.k[pages.long()] *= torch.linspace(0.05, 8, len(pages), device=DEV).to(BF16)[:, None, None, None]
    check(fa, always, cache, pages, 2048, 8, 1, q_scale=6.0)


@pytest.mark.parametrize("P,tails,Hq,Hkv,d,fp8", [(16, [1], 1, 1, 64, False), (512, [5, 0, 300, -1, -101], 8, 2, 128, False),
                                                  (1024, [9, 70], 8, 2, 128, True), (64, [1] * 130, 1, 1, 256, False)])
def test_small_ones_are_read_by_every_sequence(fa, P, tails, Hq, Hkv, d, fp8):
    cache, pages = shared_cache(fa, 3, P, tails, Hkv, d, 16, fp8)
    q, o, lse = check(fa, None, cache, pages, P, Hq, 1, joined=False)
    want = fa.attention_decode_paged(cache, q, d ** -0.5)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_no_prefix_and_a_part_of_one(fa, always):
    cache, pages = shared_cache(fa, 5, 512, [40, 3, 700], 2, 128, 16)
    q = randn(gen(6), 3, 8, 2, 128)
    want = fa.attention_decode_paged(cache, q, 0.1)
    got = fa.attention_decode_paged(cache, q, 0.1, prefix_pages=pages[:0])
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    check(fa, always, cache, pages[:7], 7 * 16, 8, 2)      # the rest of it as the sequences' own
    got, again = (call(fa, always, cache, q, pages, 0.1) for _ in range(2))
    assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])
    assert status(fa, always) == fa.FA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_pages_and_lengths(fa, always, fp8):
    """A page of the prefix out of range is masked for all; a length out of range counts as empty."""
    P = 400
    cache, pages = shared_cache(fa, 7, P, [40, 3, 70], 2, 128, 16, fp8)
    k, v = zip(*(entries(cache, b) for b in range(3)))
    pages[3], pages[24] = cache.num_pages, -1
    cache.block_table[:, 3], cache.block_table[:, 24] = cache.num_pages, -1
    q = randn(gen(8), 3, 8, 1, 128)
    for lib in (None, always):      # the one reads the table
        call(fa, lib, cache, q, pages, 0.1)
        assert status(fa, lib) == fa.FA_ERR_BAD_INDEX
    cache.lens[1] = -5
    for lib in (None, always):
        o, lse, _ = call(fa, lib, cache, q, pages, 0.1)
        assert status(fa, lib) == fa.FA_ERR_BAD_INDEX
        assert torch.all(o[1] == 0) and torch.all(lse[1] == -np.inf)
        for b in (0, 2):
            keep = [j for j in range(k[b].shape[1]) if j // 16 not in (3, 24)]
            ro, rl, _, to, tl, _ = R.attend(to64(q[b]), k[b][:, keep], v[b][:, keep], 0.1, False, 4, fp8)
            within(to64(lse[b]), rl, tl)
            A = np.stack([[np.exp(0.1 * (k[b][h // 4][keep] @ to64(q[b])[h, 0]) - rl[h, 0]) @ np.abs(v[b][h // 4][keep])] for h in range(8)])
            within(to64(o[b]), ro, to + 2.0 ** -8 * A, 2.0 ** -8)
        assert status(fa, lib) == fa.FA_OK


def test_far_pages(fa, always):
    """Pages beyond 2^32 bytes of the pool."""
    n = (5 << 30) // (2 * 16 * 64 * 2) // 2 * 2
    k, v = (torch.zeros((n, 2, 16, 64), dtype=BF16, device=DEV) for _ in range(2))
    P = 320
    ids = torch.randperm(n // 8, generator=gen(9), device=DEV)[:22].to(I32) + (n - n // 8)
    for i, pool in enumerate((k, v)):
        pool[ids.long()] = randn(gen(10 + i), 22, 2, 16, 64)
    table = torch.cat((ids[:20].expand(2, 20), ids[20:].view(2, 1)), 1).contiguous()
    cache = fa.KVCache(k, v, table, torch.tensor([P + 5, P + 16], dtype=I32, device=DEV))
    check(fa, always, cache, ids[:20].clone(), P, 4, 1)


def test_both_ways_captured_and_two_streams(fa):
    cache, pages = shared_cache(fa, 11, 8192, [500, 3, 70], 4, 128, 16)
    q = randn(gen(12), 3, 64, 1, 128)
    check(fa, None, cache, pages, 8192, 64, 1, sequences=[1])
    o, o2, lse, lse2 = torch.empty_like(q), torch.empty_like(q), torch.empty((3, 64, 1), device=DEV), torch.empty((3, 64, 1), device=DEV)
    n = fa.fa_decode_paged_shared_workspace_bytes(cache, 64, 1, pages)
    ws, ws2 = (torch.full((n,), 255, dtype=torch.uint8, device=DEV) for _ in range(2))
    fa.fa_decode_paged_shared(cache, q, o, lse, pages, 0.1, ws)
    fa._decode_shared(cache, q, o2, lse2, pages, 0.1, ws, True, None)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    if fa._fa_py is not None:
        call = fa._fa_py.decode_shared
        assert call(cache._ref, cache._index, q, o, lse, pages, 0.1, ws, True, None) == fa.FA_OK
        assert call(cache._ref, cache._index, q, o, lse, pages.long(), 0.1, ws, True, None) is None
        assert call(cache._ref, cache._index, q, o, lse, pages[::2], 0.1, ws, True, None) is None
    # two captured graphs that share a workspace, on one stream, with lengths that change between replays
    graphs = []
    for out in ((o, lse), (o2, lse2)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            fa.fa_decode_paged_shared(cache, q, *out, pages, 0.1, ws, causal=out[0] is o)
        graphs.append(graph)
    for cut in (0, 3):
        cache.lens.copy_(torch.tensor([8692 - cut, 8195 - cut, 8262 - cut], dtype=I32))
        for t in (o, o2):
            t.fill_(7)
        for graph in graphs:
            graph.replay()
        for causal, out in ((True, (o, lse)), (False, (o2, lse2))):
            want = fa.attention_decode_paged(cache, q, 0.1, causal=causal, prefix_pages=pages)
            assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])
    # two streams at once, a workspace each
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        fa.fa_decode_paged_shared(cache, q, o, lse, pages, 0.1, ws, stream=side[0])
        fa.fa_decode_paged_shared(cache, q, o2, lse2, pages, 0.1, ws2, stream=side[1])
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(o2, want[0]) and torch.equal(lse, lse2)
    assert fa.fa_sync_status() == fa.FA_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_outside_the_buffers(fa, always, fp8):
    cache, pages = shared_cache(fa, 13, 320, [500, 3, -1, 70, 9], 2, 128, 16, fp8)
    Hq, B = 14, 5
    q = randn(gen(14), B, Hq, 1, 128)
    n, nb = q.numel(), fa.fa_decode_paged_shared_workspace_bytes(cache, Hq, 1, pages)
    ob, lb = torch.full((n + 512,), 7.0, dtype=BF16, device=DEV), torch.full((B * Hq + 128,), 7.0, device=DEV)
    wb = torch.full((nb + 512,), 7, dtype=torch.uint8, device=DEV)
    o, lse = ob[256:256 + n].view(q.shape), lb[64:64 + B * Hq].view(B, Hq, 1)
    ws = wb[256:256 + nb]
    assert always.fa_decode_paged_shared(cache._ref, q.data_ptr(), o.data_ptr(), lse.data_ptr(), Hq, 1, 1, pages.data_ptr(), pages.numel(), 0.1,
                                         ws.data_ptr(), nb, torch.cuda.current_stream().cuda_stream) == 0
    want = call(fa, always, cache, q, pages, 0.1)
    assert status(fa, always) == fa.FA_OK and torch.equal(o, want[0]) and torch.equal(lse, want[1])
    for t, a, b in ((ob, 256, n), (lb, 64, B * Hq), (wb, 256, nb)):
        assert torch.all(t[:a] == 7) and torch.all(t[a + b:] == 7)


def test_refusals(fa):
    cache, pages = shared_cache(fa, 15, 64, [5], 1, 64, 16)
    q = randn(gen(16), 1, 2, 1, 64)
    o, lse = torch.empty_like(q), torch.empty((1, 2, 1), device=DEV)
    n = fa.fa_decode_paged_shared_workspace_bytes(cache, 2, 1, pages)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged_shared(cache, q, o, lse, pages, 0.1, ws[:-256])
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged_shared(cache, q, o, lse, torch.zeros(cache.max_pages + 1, dtype=I32, device=DEV), 0.1, torch.empty(1 << 24, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        fa.fa_decode_paged_shared(cache, q, o, lse, pages[None], 0.1, ws)
    with pytest.raises(TypeError):
        fa.fa_decode_paged_shared(cache, q, o, lse, pages.long(), 0.1, ws)
    with pytest.raises(ValueError):
        fa.attention_decode_paged(cache, q, 0.1, prefix_pages=pages, window=(5, 0))
    assert fa.fa_sync_status() == fa.FA_OK
