"""Queries of a wide range over an e4m3 cache (fa_decode_paged): features far below the row's
largest.

Tolerances are those of tests/paged_ref.py, with one term more.  A query row enters its products as
f16 after a power of two that brings its largest value to [2^14, 2^15).  A bf16 value has 8
significant bits, so it is exact there from 2^-17 on, which is 2^-31 of the largest or more; below it
goes in f16's steps of 2^-24, so that it is off by at most 2^-25, 2^-39 of the row's largest.  A score
is then off by at most r = c 2^-39 max|q| sum|k| more, an output by 2 r A and lse by r.
"""
import numpy as np
import pytest
import torch

import paged_ref as R
from gpu_util import to64
from test_cache_gpu import entries, gen, make_cache, randn, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def check(fa, cache, q, scale, Hkv):
    o, lse = fa.attention_decode_paged(cache, q, scale, accumulate=True)
    assert fa.fa_sync_status() == fa.FA_OK
    Hq = q.shape[1]
    for b in range(cache.B):
        k, v = entries(cache, b)
        q64 = to64(q[b])
        ro, rl, _, to, tl, _ = R.attend(q64, k, v, scale, True, Hq // Hkv, True)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            r = scale * 2.0 ** -39 * np.abs(q64[h]).max() * np.abs(k[kv]).sum(-1).max(initial=0.0)
            to[h] += 2 * r * np.abs(v[kv]).max(initial=0.0)
            tl[h] += r
        within(to64(lse[b]), rl, tl)
        within(to64(o[b]), ro, to, 2.0 ** -8)


@pytest.mark.parametrize("below", [0, 8, 13, 17, 24, 30])
@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_one_large_feature_against_zero_keys(fa, d, rows, below):
    """A feature 2^below times the others, whose keys are 0: the scores are the others' alone."""
    cache = make_cache(fa, 90 + below, [150, 700], 2, d, 16, fp8=True, weight=True)
    cache.k[..., 0] = 0
    q = randn(gen(91), 2, 2 * rows, 1, d, dtype=F32).abs().clamp(0.25, 1.9) * 2.0 ** (12 - below)
    q = torch.where(torch.rand(q.shape, generator=gen(92), device=DEV) < 0.5, -q, q)
    q[..., 0] = 4096.0
    # scores of a few units: keys are about 40 k_scale
    check(fa, cache, q.to(BF16), 2.0 ** (below - 12) / (40 * float(cache.k_scale.max()) * d ** 0.5), 2)
