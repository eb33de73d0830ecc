"""fa_decode_paged_shared takes the prefix's pages from prefix_pages alone, whether the prefix is computed by itself
(the test library always does) or read by every sequence (the library at these sizes): entries of the block table that
stand for them may hold anything, and a page of prefix_pages out of range is masked for all.  Tolerances as in
tests/test_shared_gpu.py."""
import numpy as np
import pytest
import torch

import paged_ref as R
from gpu_util import to64
from test_cache_gpu import entries, gen, randn, within
from test_shared_gpu import always, call, fa, shared_cache, status  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def expect(cache, q, o, lse, k, v, keep, fp8, b):
    G = q.shape[1] // cache.Hkv
    ro, rl, _, to, tl, _ = R.attend(to64(q[b]), k[:, keep], v[:, keep], 0.1, False, G, fp8)
    within(to64(lse[b]), rl, tl)
    for h in range(q.shape[1]):   # the prefix's probabilities in bf16 (of all entries: the larger bound)
        for t in range(q.shape[2]):
            p = np.exp(0.1 * (k[h // G][keep] @ to64(q[b])[h, t]) - rl[h, t])
            to[h, t] += 2.0 ** -8 * (p @ np.abs(v[h // G][keep]))
    within(to64(o[b]), ro, to, 2.0 ** -8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [False, True])
@pytest.mark.parametrize("P,tails,ps,causal", [(400, [40, 3, 70], 16, False), (64, [1, 0], 64, True)])
def test_the_tables_entries_of_the_prefix_are_not_read(fa, always, fp8, bad, P, tails, ps, causal):
    """bad: out of range; else the page of the first sequence's own entries."""
    cache, pages = shared_cache(fa, 21, P, tails, 2, 128, ps, fp8)
    kv = [entries(cache, b) for b in range(len(tails))]
    cache.block_table[:, :P // ps] = cache.num_pages + 5 if bad else cache.block_table[0, P // ps].clone()
    q = randn(gen(22), len(tails), 8, 1, 128)
    for lib in (None, always):
        o, lse, _ = call(fa, lib, cache, q, pages, 0.1, causal)
        assert status(fa, lib) == fa.FA_OK
        for b, (k, v) in enumerate(kv):
            expect(cache, q, o, lse, k, v, np.arange(k.shape[1]), fp8, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_out_of_range_are_masked_though_the_table_is_good(fa, always, fp8):
    cache, pages = shared_cache(fa, 23, 400, [40, 3, 70], 2, 128, 16, fp8)
    kv = [entries(cache, b) for b in range(3)]
    pages[3], pages[24] = cache.num_pages, -1
    q = randn(gen(24), 3, 8, 1, 128)
    for lib in (None, always):
        o, lse, _ = call(fa, lib, cache, q, pages, 0.1)
        assert status(fa, lib) == fa.FA_ERR_BAD_INDEX
        for b, (k, v) in enumerate(kv):
            expect(cache, q, o, lse, k, v, [j for j in range(k.shape[1]) if j // 16 not in (3, 24)], fp8, b)
    pages[0] = -1                                       # and a prefix of which nothing is left but one page
    pages[2:] = -1
    for lib in (None, always):
        o, lse, _ = call(fa, lib, cache, q, pages, 0.1)
        assert status(fa, lib) == fa.FA_ERR_BAD_INDEX
        for b, (k, v) in enumerate(kv):
            expect(cache, q, o, lse, k, v, [j for j in range(k.shape[1]) if j // 16 == 1 or j >= 400], fp8, b)


def test_lengths_inside_the_prefix(fa, always):
    """Sequences that end inside the prefix, with several rows: the same pages."""
    cache, pages = shared_cache(fa, 25, 384, [0, 9, -384, -200], 2, 64, 128)
    kv = [entries(cache, b) for b in range(4)]
    cache.block_table[:, :3] = -7
    q = randn(gen(26), 4, 4, 1, 64)
    for lib in (None, always):
        o, lse, _ = call(fa, lib, cache, q, pages, 0.1)
        assert status(fa, lib) == fa.FA_OK
        for b, (k, v) in enumerate(kv):
            expect(cache, q, o, lse, k, v, np.arange(k.shape[1]), False, b)
