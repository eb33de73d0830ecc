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


@pytest.mark.parametrize("rows", [1, 16, 40])
@pytest.mark.parametrize("q_exp,k_exp", [(-100, -64), (-126, 0), (-130, -30), (-60, -64), (0, -64), (60, -60), (-70, 64)])
def test_scores_of_small_and_large_scales(fa, rows, q_exp, k_exp):
    """Queries and key scales from end to end of their ranges, entries masked by length and by row: what
    underflows is 0, and masked entries stay masked."""
    cache = make_cache(fa, 95, [37, 100, 5], 1, 64, 16, fp8=True, weight=True)
    cache.k_scale.fill_(2.0 ** k_exp)
    q = (randn(gen(96), 3, rows, 3, 64, dtype=F32).double() * 2.0 ** q_exp).to(BF16)
    c = 1.0 if q_exp + k_exp < -20 else 2.0 ** -10
    check(fa, cache, q, c, 1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 16, 40])
def test_zero_scores_of_the_largest_scales(fa, rows, fp8):
    """Keys of 0 under the largest query, key scale and softmax scale: every entry counts alike."""
    cache = make_cache(fa, 97, [37, 100, 5], 1, 64, 16, fp8=fp8, weight=True)
    for b in range(3):
        cache.k[cache.block_table[b, :-(-int(cache.lens[b]) // 16)].long()] = 0
    if fp8:
        cache.k_scale.fill_(2.0 ** 64)
    q = (randn(gen(98), 3, rows, 1, 64, dtype=F32).clamp(-2, 2) * 2.0 ** 100).to(BF16)
    check(fa, cache, q, 3.0e38, 1)
    q.zero_()
    check(fa, cache, q, 1e-44, 1)


@pytest.mark.parametrize("rows", [1, 16, 40])
def test_subnormal_queries_count(fa, rows):
    """Queries below bf16's normal range under a softmax scale that makes scores of a few units of them."""
    cache = make_cache(fa, 99, [37, 100, 5], 1, 64, 16, fp8=True, weight=True)
    cache.k_scale.fill_(1.0)
    q = (randn(gen(100), 3, rows, 1, 64, dtype=F32).double() * 2.0 ** -129).to(BF16)
    assert float(q.double().abs().max()) < 2.0 ** -126 and bool((q != 0).any())
    check(fa, cache, q, 2.0 ** 122, 1)


def test_an_undefined_key_scale_shows(fa):
    """A NaN among the key scales makes NaN of its head's rows, and of no others."""
    cache = make_cache(fa, 101, [37, 100], 2, 64, 16, fp8=True)
    q = randn(gen(102), 2, 4, 1, 64)
    want, _ = fa.attention_decode_paged(cache, q, 0.1)
    cache.k_scale[1] = float("nan")
    o, lse = fa.attention_decode_paged(cache, q, 0.1)
    assert fa.fa_sync_status() == fa.FA_OK
    assert torch.isnan(o[:, 2:]).all() and torch.isnan(lse[:, 2:]).all() and torch.equal(o[:, :2], want[:, :2])
