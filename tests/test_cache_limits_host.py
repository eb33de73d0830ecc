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
