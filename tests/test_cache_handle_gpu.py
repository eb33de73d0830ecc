"""A KVCache whose tensors are assigned between calls: the calls read and write the new ones."""
import pytest
import torch

from test_cache_gpu import BF16, DEV, check_decode, gen, make_cache, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def test_assigned_tensors_are_read_and_written(fa):
    """A step of append, decode with weights and evict in which every tensor of the handle is replaced by a
    copy, the one before filled with values that would show."""
    cache = make_cache(fa, 21, [40, 7, 64], 2, 64, 16, weight=True, seen=torch.tensor([40, 7, 64], device=DEV, dtype=torch.int32))
    old = {}
    for name in cache._TENSORS:
        t = getattr(cache, name)
        if t is not None:
            setattr(cache, name, t.clone())
            old[name] = t.fill_(1 if t.dtype != BF16 else float("nan"))
    marks = {n: t.clone() for n, t in old.items()}
    cache.lens = cache.lens + 1
    cache.seen = cache.seen + 1
    k, v = randn(gen(22), 3, 2, 1, 64), randn(gen(23), 3, 2, 1, 64)
    fa.fa_cache_append(cache, k, v)
    for b, n in enumerate((40, 7, 64)):
        page = int(cache.block_table[b, n // 16]) if n // 16 < cache.max_pages else None
        if 0 <= page < cache.num_pages:
            assert torch.equal(cache.k[page, :, n % 16], k[b, :, 0]) and torch.equal(cache.v[page, :, n % 16], v[b, :, 0])
            assert cache.order[b, :, n].tolist() == [n, n] and cache.weight[b, :, n].tolist() == [0, 0]
    fa.fa_sync_status()
    cache.lens = torch.tensor([41, 8, 64], device=DEV, dtype=torch.int32)    # the third's page is out of range
    check_decode(fa, cache, 4, 1, accumulate=True)
    cache.weight = torch.rand_like(cache.weight)
    kept = fa.fa_cache_evict(cache, 10)
    assert fa.fa_sync_status() == fa.FA_OK and cache.lens.tolist() == [10, 8, 10]
    assert int(kept[0].max()) <= 40 and int(kept[0].min()) >= 0
    check_decode(fa, cache, 4, 1, accumulate=True)
    for n, t in old.items():
        assert torch.equal(t.view(torch.uint8), marks[n].view(torch.uint8)), n


def test_empty_caches_with_weights(fa):
    """No sequences, and sequences without a slot: nothing to attend to, to add up or to evict."""
    for B, pages in ((0, 3), (2, 0)):
        cache = fa.alloc_kv_cache(B, 2, 64, 16 * pages, 16, weight=True)
        q = torch.ones((B, 4, 1, 64), device=DEV, dtype=BF16)
        o, lse = fa.attention_decode_paged(cache, q, 0.1, accumulate=True)
        kept = fa.fa_cache_evict(cache, 5, n_first=1, n_recent=2)
        assert fa.fa_sync_status() == fa.FA_OK
        assert torch.all(o == 0) and torch.all(torch.isneginf(lse)) and torch.all(kept == -1) and cache.lens.tolist() == [0] * B
        no = torch.zeros((B, 2, 0, 64), device=DEV, dtype=BF16)
        fa.fa_cache_append(cache, no, no)
        assert fa.fa_sync_status() == fa.FA_OK
