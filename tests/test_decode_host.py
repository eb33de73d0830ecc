"""Refusals of the paged decodes under a window and over a shared prefix on the host, before any CUDA call, and the
size of their workspaces.  The addresses are made up: the file runs only where there is no GPU."""
import ctypes

import pytest
import torch

from test_cache_host import INVALID, MB, NO_GPU, P, UNSUPPORTED, cache, fa  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")
Q, O, LSE, WS, PAGES = (P + i * MB for i in (20, 21, 22, 23, 40))


def test_window_refusals(fa):
    f = fa.lib().fa_decode_paged_window

    def call(q=Q, o=O, lse=LSE, Hq=4, Tq=1, left=5, sinks=2, scale=0.1, ws=WS, n=16 * MB, **kw):
        return f(ctypes.byref(cache(fa, **kw)), q, o, lse, Hq, Tq, left, sinks, scale, ws, n, None)
    assert call() in NO_GPU and call(left=-1) in NO_GPU and call(left=2 ** 31 - 1, sinks=2 ** 31 - 1) in NO_GPU
    assert call(B=0) == 0
    assert call(left=-2) == INVALID and call(sinks=-1) == INVALID and call(left=-2, B=0) == INVALID
    assert call(scale=0.0) == INVALID and call(scale=float("nan")) == INVALID
    assert call(Tq=17) == UNSUPPORTED and call(Tq=0) == INVALID and call(Hq=3) == INVALID
    assert call(d=96) == UNSUPPORTED and call(page_size=8) == UNSUPPORTED
    assert call(q=None) == INVALID and call(o=O + 8) == INVALID and call(o=Q) == INVALID and call(lse=O) == INVALID
    assert call(o=P) == INVALID and call(ws=None) == INVALID and call(ws=WS + 128) == INVALID and call(n=255) == INVALID
    assert call(ws=P + 4 * MB) == INVALID       # the cache's state


def test_shared_refusals(fa):
    f = fa.lib().fa_decode_paged_shared

    def call(q=Q, o=O, lse=LSE, Hq=4, Tq=1, causal=1, pages=PAGES, np=2, scale=0.1, ws=WS, n=16 * MB, **kw):
        return f(ctypes.byref(cache(fa, **kw)), q, o, lse, Hq, Tq, causal, pages, np, scale, ws, n, None)
    assert call() in NO_GPU and call(causal=0) in NO_GPU and call(np=4) in NO_GPU and call(np=0, pages=None) in NO_GPU
    assert call(B=0) == 0
    assert call(np=5) == INVALID and call(np=-1) == INVALID and call(causal=2) == INVALID
    assert call(pages=None) == INVALID and call(pages=PAGES + 2) == INVALID
    assert call(pages=O) == INVALID and call(pages=LSE + 4) == INVALID and call(pages=WS + 64) == INVALID
    assert call(Tq=17) == UNSUPPORTED and call(Hq=3) == INVALID and call(scale=-1.0) == INVALID
    assert call(o=Q) == INVALID and call(ws=WS + 16) == INVALID and call(n=255) == INVALID


def test_shared_workspace(fa):
    """The paged decode's part, the own entries' o and lse, and a state of d + 2 floats for each row and run."""
    size, paged = fa.lib().fa_decode_paged_shared_workspace_bytes, fa.lib().fa_decode_paged_workspace_bytes
    for d, dtype, rows in ((64, fa.FA_BF16, 256), (128, fa.FA_E4M3, 256), (256, fa.FA_BF16, 128)):
        B, Hq, Hkv, Tq, pages, ps = 5, 8, 2, 3, 100, 16
        args = (B, Hq, Hkv, Tq, pages, ps, d)

        def up(x):
            return (x + 255) // 256 * 256
        base = up(paged(*args, 0)) + up(B * Hq * Tq * d * 4) + up(B * Hq * Tq * 4)
        assert size(*args, dtype, 0) == base
        state, tiles = Hkv * rows * (d + 2) * 4, -(-pages * ps // (64 if d == 256 else 128))
        runs = (size(*args, dtype, pages) - base) / state
        assert runs == int(runs) and 1 <= runs <= tiles
        assert size(*args, dtype, pages + 1) == 0 and size(*args, dtype, -1) == 0 and size(*args, fa.FA_F32, 1) == 0
    assert size(5, 8, 3, 1, 100, 16, 64, 0, 1) == 0 and size(5, 8, 2, 17, 100, 16, 64, 0, 1) == 0
    assert size(5, 8, 2, 1, 100, 16, 96, 0, 1) == 0


def test_sinks_that_are_no_count(fa):
    """Without a window they do not reach the library, and are checked all the same."""
    cache = fa.alloc_kv_cache(1, 1, 64, 16, device="cpu")
    q = torch.empty((1, 1, 1, 64), dtype=torch.bfloat16)
    for kw in (dict(), dict(window=(5, 0)), dict(prefix_pages=torch.zeros(1, dtype=torch.int32))):
        for bad in (-3, 2 ** 32):
            with pytest.raises(ValueError, match="sinks"):
                fa.attention_decode_paged(cache, q, 0.1, sinks=bad, **kw)
        with pytest.raises(TypeError):
            fa.attention_decode_paged(cache, q, 0.1, sinks=1.5, **kw)
