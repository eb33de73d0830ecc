"""The probabilities of a bf16 cache's paged decode enter their product with 16 bits.

An output's own rounding, 2^-8 |o|, hides any error of the probabilities unless |o| is far below
A = sum p |v|.  Here the values of the last three entries cancel the sum of the others to about 2^-24 A, and
queries have one feature that is not 0, so that scores are exact products.

Tolerance, relative to A.  The probabilities' two bf16 halves leave 2^-17 (the first is off by at most 2^-8 p and
what is left has 8 bits again).  A score of up to 8.1 in log2 units carries the roundings of its factor (two) and of
the difference: 8.1 * 3 * 2^-24 * ln 2 < 2^-19.9; exp2 twice, of the entry and of its warp's maximum, 2 * 2^-22.
Sums: four products of 16 entries into an fp32 accumulator, at most 17 roundings of 2^-24 each, are 2^-17.9; the
factor and the sum over four warps 4 * 2^-24.  Together below 2^-17 (1 + 0.14 + 0.07 + 0.54 + 0.04) < 2^-16.
"""
import numpy as np
import pytest
import torch

from gpu_util import to64
from test_cache_gpu import BF16, DEV, entries, gen, make_cache, randn

pytestmark = pytest.mark.gpu
N = 32      # two groups of 16 entries, two halves of the probabilities: at most four products in one accumulator


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def bf16(x):
    return to64(torch.from_numpy(np.asarray(x, dtype=np.float64)).to(BF16))


@pytest.mark.parametrize("rows", [1, 8, 16, 32, 64])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_probabilities_have_16_bits(fa, d, rows):
    cache = make_cache(fa, 7, [N], 1, d, 16)
    g = gen(8)
    s = bf16(torch.rand(N, generator=g, device=DEV).cpu().numpy() * 4 - 2)
    s[-3:] = bf16([2.0, -1.5, -5.625])          # 1, 2^-5 and 2^-11 of the largest
    p = np.exp(s - s.max())
    p /= p.sum()
    v = to64(randn(g, N, d))
    for i in (N - 3, N - 2, N - 1):
        v[i] = bf16(-(p[:i] @ v[:i]) / p[i])
    pages = cache.block_table[0, :N // 16].long()
    k = torch.zeros((N, d))
    k[:, 0] = torch.from_numpy(s)
    for pool, x in ((cache.k, k), (cache.v, torch.from_numpy(v))):
        pool[pages] = x.to(DEV, BF16).view(N // 16, 1, 16, d)
    k64, v64 = entries(cache, 0)
    assert np.array_equal(k64[0, :, 0], s) and np.array_equal(v64[0], v)

    ref, A = p @ v, p @ np.abs(v)
    assert (np.abs(ref) <= 2.0 ** -20 * A).all()
    tol = 2.0 ** -16 * A + 2.0 ** -8 * np.abs(ref)
    # the bound sees what it is there for: probabilities of 11 bits are outside
    e, m = np.frexp(p)
    assert (np.abs(np.ldexp(np.round(e * 2.0 ** 11) / 2.0 ** 11, m) @ v - ref) > tol).any()

    q = torch.zeros((1, rows, 1, d), device=DEV, dtype=BF16)
    q[..., 0] = 1.0
    o, _ = fa.attention_decode_paged(cache, q, 1.0)
    assert fa.fa_sync_status() == fa.FA_OK
    excess = np.abs(to64(o[0, :, 0]) - ref) - tol
    assert excess.max() <= 0, float((np.abs(to64(o[0, :, 0]) - ref) / A).max())
