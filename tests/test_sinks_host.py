"""Refusals of the attention under a window with sinks on the host, before any CUDA call, and the size of its
workspace.  The addresses are made up: the refusals run only where there is no GPU."""
import pytest
import torch

from test_cache_host import INVALID, MB, NO_GPU, P, UNSUPPORTED, fa  # noqa: F401  (fa: a fixture)

made_up = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")


@made_up
def test_refusals(fa):
    f, g = fa.lib().fa_fwd_sinks, fa.lib().fa_bwd_sinks
    t = [P + i * MB for i in range(10)]

    def fwd(left=5, sinks=2, d=64, scale=0.1, o=t[3]):
        return f(t[0], t[1], t[2], o, t[4], 1, 1, 100, 100, d, left, sinks, scale, None)

    def bwd(left=5, sinks=2, d=64, det=0, ws=t[9], dq=t[6], nbytes=None):
        need = fa.fa_bwd_sinks_workspace_bytes(1, 1, 100, 100, d, left, sinks)
        return g(t[0], t[1], t[2], t[3], t[4], t[5], dq, t[7], t[8], 1, 1, 100, 100, d, left, sinks, det, 0.1, ws,
                 need if nbytes is None else nbytes, None)
    assert fwd() in NO_GPU and fwd(left=-1) in NO_GPU and fwd(left=2 ** 31 - 1, sinks=2 ** 31 - 1) in NO_GPU
    assert fwd(left=-2) == INVALID and fwd(sinks=-1) == INVALID and fwd(scale=0.0) == INVALID and fwd(o=t[0]) == INVALID
    assert fwd(d=96) == UNSUPPORTED
    assert bwd() in NO_GPU and bwd(left=2 ** 31 - 1, sinks=2 ** 31 - 1) in NO_GPU
    assert bwd(left=-2) == INVALID and bwd(sinks=-1) == INVALID and bwd(det=2) == INVALID and bwd(ws=None) == INVALID
    assert bwd(dq=t[0]) == INVALID and bwd(d=256) == UNSUPPORTED and bwd(ws=P + 9 * MB + 16) == INVALID
    assert bwd(nbytes=fa.fa_bwd_sinks_workspace_bytes(1, 1, 100, 100, 64, 5, 2) - 1) == INVALID


def test_bounds_beyond_32_bits(fa):
    t = torch.empty((1, 1, 4, 64), dtype=torch.bfloat16)
    for left, sinks in ((2 ** 32, 0), (5, 2 ** 32 + 1), (-2 ** 40, 0)):
        with pytest.raises(ValueError):
            fa.fa_fwd_sinks(t, t, t, t, torch.empty((1, 1, 4)), left, sinks, 1.0)
        with pytest.raises(ValueError):
            fa.fa_bwd_sinks(t, t, t, t, torch.empty((1, 1, 4)), t, t, t, t, left, sinks, 1.0, t)
        with pytest.raises(ValueError):
            fa.fa_bwd_sinks_workspace_bytes(1, 1, 4, 4, 64, left, sinks)


def test_workspace(fa):
    """The partial sums: per head and key block with sinks, parts x (dV and dK) x 128 rows of d floats; none without
    a left bound or sinks."""
    size, base = fa.fa_bwd_sinks_workspace_bytes, fa.fa_bwd_workspace_bytes
    for args in ((1, 1, 3000, 3000, 128), (2, 3, 777, 5000, 64), (8, 32, 4096, 4096, 128)):
        assert size(*args, -1, 4) == size(*args, 100, 0) == base(*args)
        for left, sinks in ((0, 1), (100, 4), (100, 300), (10 ** 9, 10 ** 9)):
            extra, unit = size(*args, left, sinks) - base(*args), args[0] * args[1] * -(-min(sinks, args[3]) // 128) * 2 * 128 * args[4] * 4
            assert extra % unit == 0 and extra // unit in (0, *range(2, 65))
    assert size(1, 1, 3000, 3000, 128, 255, 4) - base(1, 1, 3000, 3000, 128) == 3 * 2 * 128 * 128 * 4   # 24 query blocks, 8 a part
    for sinks in (128, 2000, 65536):       # up to eight parts for each of the 152 SMs
        assert size(1, 32, 65536, 65536, 64, 100, sinks) - base(1, 32, 65536, 65536, 64) <= 8 * 152 * 2 * 128 * 64 * 4
    assert size(0, 3, 100, 100, 64, 5, 1) == base(0, 3, 100, 100, 64)
    assert size(1, 1, 100, 100, 64, -2, 0) == 0 and size(1, 1, 100, 100, 64, 0, -1) == 0 and size(1, 1, 100, 100, 96, 0, 1) == 0


def test_no_parts_where_the_left_bound_hides_nothing(fa):
    size, base = fa.fa_bwd_sinks_workspace_bytes, fa.fa_bwd_workspace_bytes
    for args in ((1, 1, 3000, 3000, 128), (2, 3, 777, 5000, 64)):
        for left, sinks in ((100, args[3]), (0, 10 ** 9), (args[3] - 1, 4), (2 ** 31 - 1, 4)):
            assert size(*args, left, sinks) == base(*args), (left, sinks)
        assert size(*args, 100, args[3] - 1) >= base(*args)


def test_bounds_are_whole_numbers(fa):
    t = torch.empty((1, 1, 4, 64), dtype=torch.bfloat16)
    for left, sinks in ((600.5, 4), (600.0, 4), (600, 4.5), (None, 4), ("600", 4)):
        with pytest.raises(TypeError):
            fa.fa_fwd_sinks(t, t, t, t, torch.empty((1, 1, 4)), left, sinks, 1.0)
        with pytest.raises(TypeError):
            fa.fa_bwd_sinks(t, t, t, t, torch.empty((1, 1, 4)), t, t, t, t, left, sinks, 1.0, t)
        with pytest.raises(TypeError):
            fa.fa_bwd_sinks_workspace_bytes(1, 1, 4, 4, 64, left, sinks)
        cache = fa.alloc_kv_cache(1, 1, 64, 16, device="cpu")
        q, o, lse = torch.empty((1, 1, 1, 64), dtype=torch.bfloat16), torch.empty((1, 1, 1, 64), dtype=torch.bfloat16), torch.empty((1, 1, 1))
        with pytest.raises(TypeError):
            fa.fa_decode_paged_window(cache, q, o, lse, left, sinks, 1.0, torch.empty(256, dtype=torch.uint8))
    for left, sinks in ((torch.tensor(100), 4), (True, torch.tensor(4))):
        assert fa.fa_bwd_sinks_workspace_bytes(1, 1, 3000, 3000, 64, left, sinks) == fa.fa_bwd_sinks_workspace_bytes(1, 1, 3000, 3000, 64, int(left), 4)
