"""Sizes at the ends of the cache calls' ranges, on the host: what is refused and what is an empty call.
The addresses are made up (see test_cache_host.py), so the file runs only where there is no GPU."""
import ctypes

import pytest
import torch

from test_cache_host import INVALID, MB, NO_GPU, P, UNSUPPORTED, cache, vp  # noqa: F401

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import build
    build.build()
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def evict(fa, budget, **kw):
    c = cache(fa, **kw)
    far = 1 << 46     # `kept` is as long as the budget says
    return fa.lib().fa_cache_evict(ctypes.byref(c), budget, 0, 0, P + 8 * MB, P + 9 * MB, P + 10 * MB, far, None)


def test_evict_budgets(fa):
    """A budget beyond the most slots of a sequence is refused: the kernels count entries of `kept` in steps
    of thousands, which would pass 2^31."""
    assert evict(fa, 1 << 30) in NO_GPU
    for budget in ((1 << 30) + 1, 2 ** 31 - 1):
        assert evict(fa, budget) == INVALID


def test_workspace_sizes_of_refused_calls(fa):
    """0 for every size that fa_decode_paged refuses: page sizes, and products beyond 31 and 63 bits."""
    size = fa.lib().fa_decode_paged_workspace_bytes
    for ps in (16, 32, 64, 128, 256):
        assert size(2, 4, 2, 1, 4, ps, 64, 0) > 0
    for ps in (1, 8, 17, 48, 512):
        assert size(2, 4, 2, 1, 4, ps, 64, 0) == 0
        c = cache(fa, page_size=ps)
        assert fa.lib().fa_decode_paged(ctypes.byref(c), P + 8 * MB, P + 9 * MB, P + 10 * MB, 4, 1, 1, 0.1, 0, P + 16 * MB,
                                        64 * MB, None) == UNSUPPORTED
    assert size(1 << 30, 1 << 30, 1, 16, 4, 16, 64, 0) == 0      # 2^64 rows
    assert size(1 << 30, 1 << 29, 1, 16, 4, 16, 64, 1) == 0      # 2^63
    assert size(1 << 27, 1, 1, 16, 4, 16, 64, 0) == 0            # 2^31


def test_binding_workspace_of_a_refused_page_size(fa):
    z = torch.zeros((4, 2, 48, 64), dtype=torch.bfloat16)
    c = fa.KVCache(z, z.clone(), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    assert fa.fa_decode_paged_workspace_bytes(c, 4) == 0


def test_empty_caches_are_empty_calls(fa):
    """No sequences, or no slots: arrays without an element have no address (torch gives 0), and the calls are
    those of a cache that has some, with nothing to do."""
    lib = fa.lib()

    def decode(acc, **kw):
        c = cache(fa, **kw)
        return lib.fa_decode_paged(ctypes.byref(c), P + 8 * MB, P + 9 * MB, P + 10 * MB, 4, 1, 1, 0.1, acc, P + 16 * MB, 64 * MB, None)

    for acc in (0, 1):
        assert decode(acc, B=0, weight=None, order=None, lens=None, block_table=None) == 0
        assert decode(acc, max_pages=0, weight=None, order=None, block_table=None) in NO_GPU
    assert decode(1, weight=None) == INVALID                                  # slots without weights

    def evict(w, o, n_recent=2, **kw):
        c = cache(fa, **kw)
        return lib.fa_cache_evict(ctypes.byref(c), 8, 1, n_recent, w, o, P + 10 * MB, P + 11 * MB, None)

    assert evict(None, None, B=0, weight=None, order=None, lens=None, block_table=None) == 0
    assert evict(None, None, max_pages=0, weight=None, order=None, block_table=None) in NO_GPU
    assert evict(P + 8 * MB, None, order=None) == INVALID                     # slots, and recent without an order
    assert evict(None, P + 9 * MB) == INVALID


def test_binding_of_empty_caches(fa):
    """The same through the handle: weights and an order of no element are there."""
    for B, pages in ((0, 3), (2, 0)):
        c = fa.alloc_kv_cache(B, 2, 64, 16 * pages, 16, weight=True, device="cpu")
        assert c.weight.numel() == 0 and c.order.numel() == 0
        assert fa.fa_decode_paged_workspace_bytes(c, 4, accumulate=True) > 0
