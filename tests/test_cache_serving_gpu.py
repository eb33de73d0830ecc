"""What a serving loop of append, decode with weights and evict leaves in lens and seen."""
import pytest
import torch

from test_cache_gpu import BF16, DEV, I32, gen, randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


@pytest.mark.parametrize("captured", [False, True])
def test_lengths_at_the_end_of_a_serving_loop(fa, captured):
    """Prompts below, at and above the budget: each sequence grows to it and stays there; seen counts on."""
    B, Hq, Hkv, d, budget, steps, prompt = 4, 8, 2, 64, 48, 40, [30, 7, 60, 48]
    g = gen(61)
    cache = fa.alloc_kv_cache(B, Hkv, d, budget + 16, 16, weight=True)
    new = torch.tensor(prompt, device=DEV, dtype=I32)
    cache.lens.add_(new)
    cache.seen.add_(new)
    fa.fa_cache_append(cache, randn(g, B, Hkv, 60, d), randn(g, B, Hkv, 60, d), new_lens=new)
    q, k, v = randn(g, B, Hq, 1, d), randn(g, B, Hkv, 1, d), randn(g, B, Hkv, 1, d)
    o, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, Hq, 1, True), dtype=torch.uint8, device=DEV)
    kept = torch.empty((B, Hkv, budget), dtype=I32, device=DEV)

    def step():
        cache.lens.add_(1)
        cache.seen.add_(1)
        fa.fa_cache_append(cache, k, v)
        fa.fa_decode_paged(cache, q, o, lse, d ** -0.5, ws, accumulate=True)
        fa.fa_cache_evict(cache, budget, kept=kept, n_first=2, n_recent=8)

    run = step
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay
    for _ in range(steps):
        run()
    assert fa.fa_sync_status() == fa.FA_OK
    lens = [min(budget, p + steps) for p in prompt]
    assert lens == [48, 47, 48, 48] and cache.lens.tolist() == lens
    assert cache.seen.tolist() == [p + steps for p in prompt]
    for b in range(B):
        for h in range(Hkv):      # the first two and the last eight are there, and none twice
            order = cache.order[b, h, :lens[b]].tolist()
            assert len(set(order)) == lens[b] and {0, 1} <= set(order)
            assert set(range(prompt[b] + steps - 8, prompt[b] + steps)) <= set(order)


def test_a_captured_step_behind_copies(fa):
    """Copies and fills, which are no kernels, between the calls of a captured step: each call waits for them."""
    B, Hq, Hkv, d = 3, 4, 2, 128
    g = gen(62)
    cache = fa.alloc_kv_cache(B, Hkv, d, 4096, 32, weight=True)
    start = [t.copy_(randn(g, *t.shape)) for t in (cache.k, cache.v)]
    start = [t.clone() for t in start]
    q, k, v = randn(g, B, Hq, 1, d), randn(g, B, Hkv, 1, d), randn(g, B, Hkv, 1, d)
    spec = fa.rope_spec(d)
    lens, pos = torch.zeros(B, device=DEV, dtype=I32), torch.zeros((1, B, 1), device=DEV, dtype=I32)
    o, lse = torch.empty_like(q), torch.empty((B, Hq, 1), device=DEV)
    qr, out = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, Hq, 1, True), dtype=torch.uint8, device=DEV)
    kept = torch.empty((B, Hkv, 500), dtype=I32, device=DEV)

    def step():
        cache.lens.copy_(lens)
        cache.seen.copy_(lens)
        fa.fa_cache_append(cache, k, v, pos, spec, q=q, q_out=qr)
        cache.weight.zero_()
        fa.fa_decode_paged(cache, qr, o, lse, 0.1, ws, accumulate=True)
        out.copy_(o)
        fa.fa_cache_evict(cache, 500, kept=kept, n_recent=3)
        cache.lens.add_(0)

    def result(run, n):
        cache.k.copy_(start[0])
        cache.v.copy_(start[1])
        cache.order.copy_(torch.arange(4096, device=DEV, dtype=I32).expand(B, Hkv, -1))
        lens.copy_(torch.tensor(n, dtype=I32))
        pos.copy_(lens.view(1, B, 1))
        run()
        assert fa.fa_sync_status() == fa.FA_OK
        return [t.clone() for t in (out, lse, kept, cache.lens, cache.weight, cache.order, cache.k, cache.v)]

    result(step, [5, 6, 7])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n in ([1, 700, 4096], [2000, 2, 501], [500, 499, 1], [4000, 3000, 2000]):
        eager = result(step, n)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(result(graph.replay, n), eager))
