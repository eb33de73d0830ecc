"""Rotary positions and the paged key/value cache (fa_rope, fa_cache_append, fa_decode_paged,
fa_cache_evict) against 64-bit references (tests/paged_ref.py, which derives the tolerances):
every element, at tile, page and split edges, ragged and empty sequences, garbage behind the
lengths, grouped heads, both cache types, captured graphs and other streams."""
import numpy as np
import pytest
import torch

import paged_ref as R
from gpu_util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def gen(seed):
    return torch.Generator(DEV).manual_seed(seed)


def randn(g, *shape, dtype=BF16):
    return torch.randn(shape, generator=g, device=DEV, dtype=F32).to(dtype)


def within(got, ref, tol, half=0.0):
    """Every element within tol plus `half` of |ref| (the output's rounding)."""
    excess = np.abs(got - ref) - tol - half * np.abs(ref)
    assert not np.isnan(got).any()
    assert excess.max(initial=-1.0) <= 0, (float(excess.max()), float(np.abs(got - ref).max()))


def freqs_of(rot, base=10000.0):
    return [base ** (-2.0 * i / rot) for i in range(rot // 2)]


# ---------------------------------------------------------------- rotation
ROPE = [
    # B, Hq, Hk, T, d, rot, axes, interleaved, packed, dtype, inverse, far
    (1, 1, 1, 1, 64, 64, 1, False, False, BF16, False, 0),
    (2, 3, 1, 33, 128, 128, 3, False, True, BF16, False, 0),
    (2, 3, 1, 33, 128, 128, 3, False, True, BF16, True, 70000),
    (1, 5, 2, 129, 256, 256, 4, True, False, BF16, False, 1000000),
    (3, 2, 2, 65, 64, 32, 2, True, True, F32, True, 1000000),
    (1, 17, 3, 257, 128, 48, 3, False, False, F32, False, 2000000000),
    (2, 1, 0, 70, 256, 16, 1, False, False, F32, False, -2000000000),
    (1, 40, 8, 1500, 128, 128, 8, True, True, BF16, False, 10),
]


def rope_case(c, seed):
    B, Hq, Hk, T, d, rot, axes, inter, packed, dt, inv, far = c
    g = gen(seed)
    freqs = freqs_of(rot)
    axis = [i * axes // (rot // 2) for i in range(rot // 2)]
    pos = (torch.randint(-50, 5000, (axes, B, T), generator=g, device=DEV) + far).to(I32)
    if packed:
        x = randn(g, B, T, Hq + Hk, d, dtype=dt).transpose(1, 2)
        q, k = x[:, :Hq], x[:, Hq:]
    else:
        q, k = randn(g, B, Hq, T, d, dtype=dt), randn(g, B, Hk, T, d, dtype=dt)
    return q, k, pos, freqs, axis


@pytest.mark.parametrize("c", ROPE)
def test_rope(fa, c):
    B, Hq, Hk, T, d, rot, axes, inter, packed, dt, inv, far = c
    q, k, pos, freqs, axis = rope_case(c, 5)
    spec = fa.RopeSpec(d, freqs, axis, inter)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    (fa.fa_rope_bwd if inv else fa.fa_rope)(q, qo, pos, spec, k=k, k_out=ko)
    assert fa.fa_sync_status() == fa.FA_OK
    half = 2.0 ** -8 if dt == BF16 else 0.0
    for x, y in ((q, qo), (k, ko)):
        for b in range(B):
            ref, tol = R.rotate(to64(x[b]), pos[:, b].cpu().numpy(), freqs, axis, inter, inv)
            within(to64(y[b]), ref, tol, half)
            assert torch.equal(y[b, ..., rot:], x[b, ..., rot:])   # behind the pairs: as it was


@pytest.mark.parametrize("inter", [False, True])
def test_rope_in_place_alone_and_other_outputs(fa, inter):
    """In place, one tensor alone and strided outputs give the bits of the plain call."""
    c = (2, 4, 4, 37, 128, 96, 2, inter, True, BF16, False, 0)
    q, k, pos, freqs, axis = rope_case(c, 7)
    spec = fa.RopeSpec(128, freqs, axis, inter)
    qo, ko = fa.rope_forward(q, k, pos, spec)
    q1 = torch.empty_like(qo)
    fa.fa_rope(q, q1, pos, spec)
    assert torch.equal(q1, qo)
    packed = torch.zeros((2, 37, 8, 128), device=DEV, dtype=BF16).transpose(1, 2)
    fa.fa_rope(q, packed[:, :4], pos, spec, k=k, k_out=packed[:, 4:])
    assert torch.equal(packed[:, :4], qo) and torch.equal(packed[:, 4:], ko)
    fa.fa_rope(q, q, pos, spec, k=k, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_rope_gradient(fa):
    """Against differences of the forward pass, and against its adjoint: the rotation is linear,
    so a difference over any step is a derivative, and <R x, g> = <x, R' g>."""
    c = (2, 2, 1, 19, 64, 48, 3, False, False, F32, False, 300)
    q, k, pos, freqs, axis = rope_case(c, 9)
    spec = fa.RopeSpec(64, freqs, axis)
    g = gen(10)
    gq, gk = randn(g, *q.shape, dtype=F32), randn(g, *k.shape, dtype=F32)
    qo, ko = fa.rope_forward(q, k, pos, spec)
    dq, dk = fa.rope_backward(gq, gk, pos, spec)
    for x, y, go, dx in ((q, qo, gq, dq), (k, ko, gk, dk)):
        lhs, rhs = (to64(y) * to64(go)).sum(), (to64(x) * to64(dx)).sum()
        # each output is off by (|a| + |b|) 2^-21
        room = 2.0 ** -20 * 2 * np.sqrt((to64(x) ** 2).sum() * (to64(go) ** 2).sum())
        assert abs(lhs - rhs) <= room
    e = torch.zeros_like(q)
    for at in ((0, 0, 3, 5), (1, 1, 18, 31), (0, 1, 7, 50)):
        e.zero_()
        e[at] = 1.0
        plus, minus = torch.empty_like(q), torch.empty_like(q)
        fa.fa_rope(q + e, plus, pos, spec)
        fa.fa_rope(q - e, minus, pos, spec)
        num = ((to64(plus) - to64(minus)) / 2 * to64(gq)).sum()
        b, h, t, _ = at
        # both outputs off by (|a| + |b|) 2^-21 and the inputs q +- e by half a step; only this row differs
        room = 2.0 ** -19 * (np.abs(to64(q[b, h, t])).max() + 2) * np.abs(to64(gq[b, h, t])).sum()
        assert abs(num - float(dq[at])) <= room


def test_rope_empty(fa):
    spec = fa.rope_spec(64, (8, 12, 12))
    for B, H, T in ((0, 2, 5), (2, 0, 5), (2, 2, 0)):
        q = torch.zeros((B, H, T, 64), device=DEV, dtype=BF16)
        fa.fa_rope(q, torch.empty_like(q), torch.zeros((3, B, T), device=DEV, dtype=I32), spec)
    assert fa.fa_sync_status() == fa.FA_OK


# ---------------------------------------------------------------- a cache with known contents
def make_cache(fa, seed, lens, Hkv, d, ps, fp8=False, weight=False, extra_pages=3, garbage=True, seen=None, width=None,
               pool=None):
    """A cache of random entries on scattered pages; everything behind the lengths is NaN
    (bf16 and e4m3 alike), the table behind them out of range."""
    g = gen(seed)
    B = len(lens)
    pages = [-(-n // ps) for n in lens]
    width = (max(pages) + 1 if B else 1) if width is None else width
    n = sum(pages) + extra_pages if pool is None else pool
    perm = torch.randperm(n, generator=g, device=DEV).to(I32)
    table = torch.full((B, width), 1 << 30 if garbage else 0, device=DEV, dtype=I32)
    if fp8:
        k, v = (torch.full((n, Hkv, ps, d), 0x7F, device=DEV, dtype=torch.uint8) for _ in range(2))
        ks, vs = (0.25 + torch.rand(Hkv, generator=g, device=DEV) for _ in range(2))
        vs = vs / 64
    else:
        k, v = (torch.full((n, Hkv, ps, d), float("nan"), device=DEV, dtype=BF16) for _ in range(2))
        ks = vs = None
    at = 0
    for b, m in enumerate(lens):
        mine = perm[at:at + pages[b]]
        at += pages[b]
        table[b, :pages[b]] = mine
        for pool_t in (k, v):
            x = randn(g, pages[b], ps, Hkv, d, dtype=F32)
            if fp8:
                x = (x * 40).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            x = x.to(pool_t.dtype).reshape(pages[b] * ps, Hkv, d)
            x[m:] = 0x7F if fp8 else float("nan")
            pool_t[mine.long()] = x.view(pages[b], ps, Hkv, d).transpose(1, 2)
    w = o = None
    if weight:
        w = torch.rand((B, Hkv, width * ps), generator=g, device=DEV)
        o = torch.arange(width * ps, device=DEV, dtype=I32).expand(B, Hkv, -1).contiguous()
    lens_t = torch.tensor(lens, device=DEV, dtype=I32)
    return fa.KVCache(k, v, table, lens_t, ks, vs, w, o, seen)


def entries(cache, b, n=None):
    """K and V of sequence b as float64 [Hkv][n][d]."""
    n = int(cache.lens[b]) if n is None else n
    ps = cache.page_size
    pages = cache.block_table[b, :-(-n // ps)].long()
    out = []
    for pool, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        x = pool[pages]
        x = to64(x.view(torch.float8_e4m3fn).float()) * to64(scale)[None, :, None, None] if scale is not None else to64(x)
        out.append(x.transpose(1, 0, 2, 3).reshape(cache.Hkv, -1, cache.d)[:, :n])
    return out


def check_decode(fa, cache, Hq, Tq, causal=True, accumulate=False, seed=1, sequences=None, scale=None, q_scale=1.0):
    g = gen(seed)
    d = cache.d
    scale = d ** -0.5 if scale is None else scale
    q = (randn(g, cache.B, Hq, Tq, d, dtype=F32) * q_scale).to(BF16)
    w0 = cache.weight.clone() if accumulate else None
    o, lse = fa.attention_decode_paged(cache, q, scale, causal=causal, accumulate=accumulate)
    assert fa.fa_sync_status() == fa.FA_OK
    G = Hq // cache.Hkv
    for b in (range(cache.B) if sequences is None else sequences):
        k, v = entries(cache, b)
        ro, rl, rw, to, tl, tw = R.attend(to64(q[b]), k, v, scale, causal, G, cache.k_scale is not None)
        dead = np.isneginf(rl)
        assert np.array_equal(np.isneginf(to64(lse[b])), dead)
        within(to64(lse[b])[~dead], rl[~dead], tl[~dead])
        within(to64(o[b]), ro, to, 2.0 ** -8)
        if accumulate:
            n = k.shape[1]
            w = to64(cache.weight[b])
            w_ref = to64(w0[b])
            w_ref[:, :n] += rw
            pad = np.zeros_like(w_ref)
            pad[:, :n] = tw + R.U * (G * Tq + 1) * np.abs(w_ref[:, :n])
            within(w, w_ref, pad)
            assert torch.equal(cache.weight[b][:, n:], w0[b][:, n:])
    return q, o, lse


DECODE = [
    # lens, Hq, Hkv, d, ps, Tq, causal, fp8, accumulate
    ([1], 1, 1, 64, 16, 1, True, False, False),
    ([17], 32, 8, 128, 16, 1, True, False, False),
    ([0, 1, 15, 16, 17, 63, 64, 65, 0, 127, 128, 129], 8, 4, 128, 16, 1, True, False, True),
    ([255, 256, 257, 511, 513], 6, 2, 64, 32, 1, True, False, True),
    ([1000, 3, 777], 5, 1, 128, 64, 3, True, False, True),
    ([2, 1, 5, 130], 4, 4, 128, 16, 4, True, False, True),
    ([300, 64], 16, 1, 256, 128, 16, True, False, False),
    ([300, 64], 7, 7, 256, 256, 2, False, False, True),
    ([5000], 48, 3, 128, 64, 7, True, False, True),
    ([100, 2000, 31, 0], 16, 2, 64, 16, 1, True, True, True),
    ([100, 2049, 33, 1], 8, 8, 128, 32, 2, True, True, False),
    ([700, 19], 12, 3, 256, 16, 5, False, True, True),
    ([9001, 1], 64, 1, 128, 256, 1, True, False, False),
    ([40000, 12], 8, 2, 128, 64, 1, True, False, True),
]


@pytest.mark.parametrize("case", DECODE)
def test_decode_paged(fa, case):
    lens, Hq, Hkv, d, ps, Tq, causal, fp8, acc = case
    cache = make_cache(fa, sum(lens) + d, lens, Hkv, d, ps, fp8, weight=acc)
    check_decode(fa, cache, Hq, Tq, causal, acc)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_decode_rows_of_a_head_group(fa, d, fp8):
    """Every instance by rows (up to 8, 16, 32 and 64 at a time, and more), at both ends of each; units whole
    and in shares, with weights."""
    for M in (1, 7, 8, 9, 16, 17, 32, 33, 64, 70):
        cache = make_cache(fa, 300 + M, [350, 0, 1, 2900], 2, d, 32, fp8, weight=True)
        check_decode(fa, cache, 2 * M, 1, accumulate=True, seed=M)
        cache = make_cache(fa, 400 + M, [130, 75, 16], 1, d, 16, fp8, weight=True)
        check_decode(fa, cache, M, 1, accumulate=True, seed=M)


@pytest.mark.parametrize("d,fp8,ps", [(64, False, 16), (128, False, 64), (128, True, 16), (64, True, 64)])
def test_decode_even_lengths_in_a_long_table(fa, d, fp8, ps):
    """Units as even as shares: taken whole by the lengths, though the table allows more."""
    lens = [700, 650, 0, 720] + [690] * 24
    cache = make_cache(fa, 33, lens, 8, d, ps, fp8, weight=True, width=4096 // ps)
    check_decode(fa, cache, 24, 1, accumulate=True, sequences=[0, 1, 2, 3, 27])


def test_decode_batch_of_many_lengths(fa):
    """More sequences than one warp reads at a time, most of them short, some empty."""
    rng = np.random.default_rng(3)
    lens = [int(x) for x in rng.integers(0, 90, 700)] + [4000, 0, 1]
    cache = make_cache(fa, 4, lens, 2, 64, 16)
    check_decode(fa, cache, 6, 1, sequences=list(range(0, 703, 29)) + [699, 700, 701, 702])


def test_decode_large_scores(fa):
    """One key far above all others: the statistics keep their range."""
    cache = make_cache(fa, 5, [3000, 70], 2, 128, 16, weight=True)
    check_decode(fa, cache, 4, 1, accumulate=True, scale=1.0, q_scale=4.0)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_small_probabilities_add_up(fa, fp8):
    """20000 equal keys beside one that outweighs each by 2^20: their share is still there."""
    n = 20001
    cache = make_cache(fa, 6, [n], 1, 64, 64, fp8)
    one = 1.0 if not fp8 else 1.0 / float(cache.k_scale[0])
    k = torch.zeros((n, 64), device=DEV)
    k[777, 0] = 1.0
    pages = cache.block_table[0, :-(-n // 64)].long()
    flat = torch.zeros((len(pages) * 64, 64), device=DEV)
    flat[:n] = k * (8.0 if fp8 else 1.0)
    codes = flat.to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else flat.to(BF16)
    cache.k[pages] = codes.view(len(pages), 1, 64, 64)
    q = torch.zeros((1, 1, 1, 64), device=DEV, dtype=BF16)
    q[..., 0] = 1.0
    kv, _ = entries(cache, 0)
    scale = 20 * np.log(2.0) / kv[0, 777, 0]
    o, lse = fa.attention_decode_paged(cache, q, scale)
    assert fa.fa_sync_status() == fa.FA_OK and one > 0
    k64, v64 = entries(cache, 0)
    ro, rl, _, to, tl, _ = R.attend(to64(q[0]), k64, v64, scale, True, 1)
    within(to64(o[0]), ro, to, 2.0 ** -8)
    within(to64(lse[0]), rl, tl)


def test_decode_far_pages(fa):
    """Pages whose elements lie beyond 2^32: only the ones in use are written."""
    Hkv, ps, d, pool = 8, 64, 128, 70000            # 4.6e9 elements of K
    k, v = (torch.empty((pool, Hkv, ps, d), device=DEV, dtype=BF16) for _ in range(2))
    g = gen(8)
    table = torch.tensor([[pool - 1, 3, pool - 70, 33000, 65999]], device=DEV, dtype=I32)
    for t in (k, v):
        t[table[0].long()] = randn(g, 5, Hkv, ps, d)
    cache = fa.KVCache(k, v, table, torch.tensor([5 * ps - 7], device=DEV, dtype=I32))
    check_decode(fa, cache, 16, 1)
    # and written there: a token appended behind them
    kn, vn = randn(g, 1, Hkv, 1, d), randn(g, 1, Hkv, 1, d)
    cache.lens.add_(1)
    fa.fa_cache_append(cache, kn, vn)
    assert fa.fa_sync_status() == fa.FA_OK
    at = 5 * ps - 7
    assert torch.equal(k[65999, :, at % ps], kn[0, :, 0]) and torch.equal(v[65999, :, at % ps], vn[0, :, 0])


def test_decode_matches_contiguous(fa):
    """The contiguous decode of the same keys: equal up to the rounding of both."""
    B, H, T, d = 2, 4, 900, 128
    cache = make_cache(fa, 11, [T, T], H, d, 64)
    k, v = (torch.stack([torch.from_numpy(entries(cache, b)[i]) for b in range(B)]).to(DEV, BF16) for i in (0, 1))
    q = randn(gen(12), B, H, 3, d)
    o1, l1 = fa.attention_decode_paged(cache, q, 0.1)
    o2, l2 = fa.attention_decode(q, k, v, True, 0.1)
    assert float((o1.float() - o2.float()).abs().max()) <= 2 * 2.0 ** -8 * float(o1.abs().max()) + 1e-3
    assert float((l1 - l2).abs().max()) <= 1e-4


def test_decode_same_bits_and_shared_workspace(fa):
    """The same call gives the same bits; a workspace used by another call in between changes nothing."""
    a = make_cache(fa, 13, [3000, 1, 900, 64], 4, 128, 16, weight=True)
    b = make_cache(fa, 14, [10000], 2, 128, 16, weight=True)
    qa, qb = randn(gen(15), 4, 16, 1, 128), randn(gen(16), 1, 4, 2, 128)
    n = max(fa.fa_decode_paged_workspace_bytes(a, 16, 1, True), fa.fa_decode_paged_workspace_bytes(b, 4, 2, True))
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV)    # NaN patterns on entry
    w0 = a.weight.clone()
    o1, l1 = fa.attention_decode_paged(a, qa, 0.1, accumulate=True, workspace=ws)
    w1 = a.weight.clone()
    fa.attention_decode_paged(b, qb, 0.1, accumulate=True, workspace=ws)
    a.weight.copy_(w0)
    o2, l2 = fa.attention_decode_paged(a, qa, 0.1, accumulate=True, workspace=ws)
    assert torch.equal(o1, o2) and torch.equal(l1, l2) and torch.equal(w1, a.weight)


def test_decode_captured_with_changing_lengths(fa):
    """Two graphs over one workspace, replayed in turn while lengths, pages and queries change."""
    cache = make_cache(fa, 17, [500, 20, 64], 2, 128, 16, weight=True, garbage=False)
    q = randn(gen(18), 3, 8, 1, 128)
    o, lse = torch.empty_like(q), torch.empty((3, 8, 1), device=DEV)
    q2 = randn(gen(19), 3, 8, 1, 128)
    o2, lse2 = torch.empty_like(q), torch.empty((3, 8, 1), device=DEV)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, 8, 1, True), dtype=torch.uint8, device=DEV)
    graphs = []
    for qq, oo, ll in ((q, o, lse), (q2, o2, lse2)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            fa.fa_decode_paged(cache, qq, oo, ll, 0.09, ws, accumulate=True)
        graphs.append(gr)
    for lens in ([500, 20, 64], [1, 0, 63], [331, 17, 2]):
        cache.lens.copy_(torch.tensor(lens, dtype=I32))
        cache.weight.zero_()
        for gr in graphs:
            gr.replay()
        assert fa.fa_sync_status() == fa.FA_OK
        for qq, oo, ll in ((q, o, lse), (q2, o2, lse2)):
            for b in range(3):
                k, v = entries(cache, b)
                ro, rl, rw, to, tl, tw = R.attend(to64(qq[b]), k, v, 0.09, True, 4)
                within(to64(oo[b]), ro, to, 2.0 ** -8)
                if lens[b]:
                    within(to64(ll[b]), rl, tl)
        for b in range(3):
            k, v = entries(cache, b)
            w = sum(R.attend(to64(qq[b]), k, v, 0.09, True, 4)[2] for qq in (q, q2))
            within(to64(cache.weight[b])[:, :lens[b]], w, 1e-4 * w + 1e-12)


def test_decode_two_streams(fa):
    """Two calls at once on two streams, each with its own workspace."""
    a = make_cache(fa, 20, [7000, 300], 4, 128, 16)
    b = make_cache(fa, 21, [40, 9000, 1], 2, 64, 32, fp8=True)
    qa, qb = randn(gen(22), 2, 8, 1, 128), randn(gen(23), 3, 16, 1, 64)
    ref_a, ref_b = fa.attention_decode_paged(a, qa, 0.1), fa.attention_decode_paged(b, qb, 0.1)
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((fa.attention_decode_paged(a, qa, 0.1, stream=sa), fa.attention_decode_paged(b, qb, 0.1, stream=sb)))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert all(torch.equal(x, y) for x, y in zip(ga + gb, ref_a + ref_b))


@pytest.mark.parametrize("raw", [False, True])
def test_allocating_calls_on_another_stream(fa, raw):
    """The current stream still works on blocks that it has freed: what a call on another stream
    allocates must not be one of them."""
    cache = make_cache(fa, 5, [70, 33], 2, 64, 16, weight=True)
    q = randn(gen(6), 2, 8, 1, 64)
    k = randn(gen(7), 2, 2, 1, 64)
    spec = fa.rope_spec(64)
    pos = torch.arange(2, dtype=torch.int32, device="cuda").view(1, 2, 1)
    want = [*fa.attention_decode_paged(cache, q, 0.1), *fa.rope_forward(q, k, pos, spec), *fa.rope_backward(q, k, pos, spec)]
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    for run in (lambda s: fa.attention_decode_paged(cache, q, 0.1, stream=s),
                lambda s: fa.rope_forward(q, k, pos, spec, stream=s), lambda s: fa.rope_backward(q, k, pos, spec, stream=s)):
        torch.cuda._sleep(20_000_000)
        junk = [torch.full((n,), 0x55, dtype=torch.uint8, device="cuda") for n in (128, 512, 2048) for _ in range(20)]
        del junk   # the blocks are free again, and the fills still wait
        got = run(other.cuda_stream if raw else other)
        torch.cuda.current_stream().wait_stream(other)
        torch.cuda.synchronize()
        for x in got:
            assert torch.equal(x, want.pop(0))
    torch.cuda._sleep(20_000_000)
    junk = [torch.full((64,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(20)]
    del junk
    kept = fa.fa_cache_evict(cache, 3, stream=other.cuda_stream if raw else other)
    torch.cuda.synchronize()
    assert int(kept.min()) >= 0 and int(kept.max()) < 70 and cache.lens.tolist() == [3, 3]


def test_decode_bad_lengths_and_pages(fa):
    """A length outside the table counts as empty, a page outside the pool as masked; both are
    reported and never read."""
    cache = make_cache(fa, 24, [100, 200, 50], 2, 64, 16, weight=True)
    cache.lens[0] = -3
    cache.lens[2] = cache.max_pages * 16 + 1
    cache.block_table[1, 4] = cache.num_pages
    cache.block_table[1, 7] = -1
    q = randn(gen(25), 3, 4, 1, 64)
    w0 = cache.weight.clone()
    o, lse = fa.attention_decode_paged(cache, q, 0.125, accumulate=True)
    assert fa.fa_sync_status() == fa.FA_ERR_BAD_INDEX
    assert fa.fa_sync_status() == fa.FA_OK          # read once
    for b in (0, 2):
        assert torch.all(o[b] == 0) and torch.all(torch.isneginf(lse[b])) and torch.equal(cache.weight[b], w0[b])
    good = torch.ones(200, dtype=torch.bool)
    good[64:80] = False
    good[112:128] = False
    cache.block_table[1, 4] = cache.block_table[1, 7] = 0
    k, v = (torch.from_numpy(x)[:, good].numpy() for x in entries(cache, 1))
    ro, rl, rw, to, tl, tw = R.attend(to64(q[1]), k, v, 0.125, True, 2)
    within(to64(o[1]), ro, to, 2.0 ** -8)
    within(to64(lse[1]), rl, tl)
    grown = (to64(cache.weight[1]) - to64(w0[1]))[:, :200]
    within(grown[:, good.numpy()], rw, 1e-4 * rw + 1e-6)
    assert np.all(grown[:, ~good.numpy()] == 0)


def test_decode_no_sequences(fa):
    z = torch.zeros((4, 2, 16, 64), device=DEV, dtype=BF16)
    cache = fa.KVCache(z, z.clone(), torch.zeros((0, 3), device=DEV, dtype=I32), torch.zeros(0, device=DEV, dtype=I32))
    q = torch.zeros((0, 4, 1, 64), device=DEV, dtype=BF16)
    fa.attention_decode_paged(cache, q, 0.1)
    empty = fa.KVCache(z, z.clone(), torch.zeros((2, 0), device=DEV, dtype=I32), torch.zeros(2, device=DEV, dtype=I32))
    o, lse = fa.attention_decode_paged(empty, torch.ones((2, 4, 1, 64), device=DEV, dtype=BF16), 0.1)
    assert fa.fa_sync_status() == fa.FA_OK
    assert torch.all(o == 0) and torch.all(torch.isneginf(lse))


# ---------------------------------------------------------------- append
APPEND = [
    # lens after, new tokens, T, Hq, Hkv, d, ps, rot (0: no rotation), interleaved, fp8, packed, seen
    ([1], [1], 1, 1, 1, 64, 16, 64, False, False, False, False),
    ([17, 300, 16], [1, 1, 1], 1, 32, 8, 128, 16, 128, False, False, True, True),
    ([40, 5, 129, 0], [40, 3, 0, 0], 40, 6, 2, 128, 32, 64, True, False, True, False),
    ([700, 257], [333, 256], 333, 4, 4, 256, 64, 256, False, False, False, True),
    ([90, 64, 65], [64, 17, 1], 64, 8, 2, 128, 16, 128, False, True, True, False),
    ([33, 2], [33, 2], 33, 2, 1, 64, 256, 32, True, True, False, True),
    ([100, 100], [20, 7], 20, 0, 3, 256, 128, 0, False, True, False, False),
    ([100, 100], [20, 7], 20, 0, 3, 64, 16, 0, False, False, True, False),
]


@pytest.mark.parametrize("case", APPEND)
def test_append(fa, case):
    lens, new, T, Hq, Hkv, d, ps, rot, inter, fp8, packed, with_seen = case
    B, g = len(lens), gen(31 + d)
    seen = torch.tensor([n + 1000 for n in lens], device=DEV, dtype=I32) if with_seen else None
    cache = make_cache(fa, 30, lens, Hkv, d, ps, fp8, weight=True, seen=seen)
    if packed:
        x = randn(g, B, T, Hq + 2 * Hkv, d).transpose(1, 2)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (randn(g, B, h, T, d) for h in (Hq, Hkv, Hkv))
    for b in range(B):      # rows behind the new ones: garbage that must not show up
        for x in (q, k, v):
            x[b, :, new[b]:] = float("nan")
    before = [t.clone() for t in (cache.k, cache.v, cache.weight, cache.order)]
    qo = torch.full((B, Hq, T, d), 7.0, device=DEV, dtype=BF16)
    kw = {}
    if rot:
        axis = [i * 3 // (rot // 2) for i in range(rot // 2)]
        pos = torch.randint(0, 9000, (3, B, T), generator=g, device=DEV).to(I32)
        kw = dict(positions=pos, spec=fa.RopeSpec(d, freqs_of(rot), axis, inter))
        if Hq:
            kw.update(q=q, q_out=qo)
    new_t = None if all(n == T for n in new) else torch.tensor(new, device=DEV, dtype=I32)
    fa.fa_cache_append(cache, k, v, new_lens=new_t, **kw)
    assert fa.fa_sync_status() == fa.FA_OK
    expect = [t.clone() for t in before]
    for b in range(B):
        n, first = new[b], lens[b] - new[b]
        slots = torch.arange(first, lens[b], device=DEV)
        pages = cache.block_table[b].long()[slots // ps]
        for i, (x, scale) in enumerate(((k, cache.k_scale), (v, cache.v_scale))):
            got = (cache.k, cache.v)[i][pages, :, slots % ps].transpose(0, 1)      # [Hkv][n][d]
            ref, tol = to64(x[b, :, :n]), 0.0
            if rot and i == 0:
                ref, tol = R.rotate(ref, pos[:, b, :n].cpu().numpy(), freqs_of(rot), axis, inter)
            if fp8:
                s = to64(scale)[:, None, None]
                ref, tol = np.clip(ref / s, -448, 448), tol / s
                got64 = to64(got.view(torch.float8_e4m3fn).float())
                within(got64, ref, tol * 1.0001 + 2.0 ** -10 + np.abs(ref) * 2.0 ** -22, 2.0 ** -4)
            else:
                within(to64(got), ref, tol, 2.0 ** -8)
            expect[i][pages, :, slots % ps] = got.transpose(0, 1)
        if rot and Hq and n:
            ref, tol = R.rotate(to64(q[b, :, :n]), pos[:, b, :n].cpu().numpy(), freqs_of(rot), axis, inter)
            within(to64(qo[b, :, :n]), ref, tol, 2.0 ** -8)
        assert torch.all(qo[b, :, n if rot and Hq else 0:] == 7.0)
        expect[2][b, :, first:lens[b]] = 0
        expect[3][b, :, first:lens[b]] = (slots + (1000 if with_seen else 0)).to(I32)
    # nothing else was written (NaN patterns compared as bits)
    for got, ref in zip((cache.k, cache.v, cache.weight, cache.order), expect):
        same = got.view(torch.uint8) == ref.view(torch.uint8)
        assert bool(same.all())


def test_append_rounds_like_the_type(fa):
    """Special values reach the cache as the type has them: infinities, NaN, saturation, ties."""
    k = torch.zeros((1, 1, 1, 64), device=DEV, dtype=BF16)
    vals = torch.tensor([float("inf"), -float("inf"), float("nan"), 1e30, 0.0625, 17.0, 19.0, -0.0, 2.0 ** -10, 2.0 ** -9],
                        device=DEV)
    k[0, 0, 0, :10] = vals.to(BF16)
    cache = make_cache(fa, 40, [1], 1, 64, 16, fp8=True)
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(0.5)
    fa.fa_cache_append(cache, k, k)
    page = int(cache.block_table[0, 0])
    kc = cache.k[page, 0, 0, :10].view(torch.float8_e4m3fn).float().cpu()
    vc = cache.v[page, 0, 0, :10].view(torch.float8_e4m3fn).float().cpu()
    expect_k = [448, -448, float("nan"), 448, 0.0625, 16.0, 20.0, -0.0, 0.0, 2.0 ** -9]      # ties to even
    expect_v = [448, -448, float("nan"), 448, 0.125, 32.0, 40.0, -0.0, 2.0 ** -9, 2.0 ** -8]
    for got, ref in ((kc, expect_k), (vc, expect_v)):
        ref = torch.tensor(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref))
        assert torch.equal(got[~torch.isnan(ref)], ref[~torch.isnan(ref)])
    b = make_cache(fa, 41, [1], 1, 64, 16)
    fa.fa_cache_append(b, k, k)
    got = b.k[int(b.block_table[0, 0]), 0, 0]
    assert torch.equal(got[~torch.isnan(got)], k[0, 0, 0][~torch.isnan(got)]) and int(torch.isnan(got).sum()) == 1


def test_append_codes_are_the_quotients(fa):
    """Every code is the e4m3 value nearest to the fp32 quotient x / scale, whatever the scale."""
    g = gen(43)
    Hkv, T = 64, 256
    cache = make_cache(fa, 44, [T], Hkv, 128, 256, fp8=True)
    for t, lo, hi in ((cache.k_scale, -64, 64), (cache.v_scale, -6, 2)):
        t.copy_(torch.exp2(lo + (hi - lo) * torch.rand(Hkv, generator=g, device=DEV)))
    v = randn(g, 1, Hkv, T, 128)
    # quotients on and next to the borders between codes, as bf16 allows
    k = ((torch.randint(-480, 480, (1, Hkv, T, 128), generator=g, device=DEV) / 16) * cache.k_scale[:, None, None]).to(BF16)
    fa.fa_cache_append(cache, k, v)
    assert fa.fa_sync_status() == fa.FA_OK
    page = int(cache.block_table[0, 0])
    for pool, x, scale in ((cache.k, k, cache.k_scale), (cache.v, v, cache.v_scale)):
        ref = (x[0].float() / scale[:, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        assert torch.equal(pool[page], ref)


def test_append_bad_counts_and_pages(fa):
    cache = make_cache(fa, 42, [40, 40, 40, 40], 1, 64, 16, weight=True)
    cache.lens[0] = cache.max_pages * 16 + 1
    cache.lens[3] = 2                                  # fewer entries than new tokens
    new = torch.tensor([3, -1, 3, 3], device=DEV, dtype=I32)
    cache.block_table[2, 2] = -5
    before = [t.clone().view(torch.uint8) for t in (cache.k, cache.v, cache.weight, cache.order)]
    k = torch.ones((4, 1, 3, 64), device=DEV, dtype=BF16)
    fa.fa_cache_append(cache, k, k, new_lens=new)
    assert fa.fa_sync_status() == fa.FA_ERR_BAD_INDEX
    for t, ref in zip((cache.k, cache.v, cache.weight, cache.order), before):
        assert torch.equal(t.view(torch.uint8), ref)


# ---------------------------------------------------------------- evict
EVICT = [
    # lens, budget, n_first, n_recent, Hkv, d, ps, fp8, kind of weights
    ([1], 1, 0, 0, 1, 64, 16, False, "random"),
    ([2, 1, 0, 5], 1, 0, 1, 2, 64, 16, False, "random"),
    ([100, 33, 17, 64], 33, 4, 8, 2, 128, 16, False, "random"),
    ([1100, 1024, 2049, 2900], 1024, 0, 0, 1, 64, 64, False, "equal"),
    ([9000, 8193, 4097], 5000, 3, 40, 1, 64, 16, False, "equal"),
    ([17000, 9], 8190, 3, 40, 2, 64, 128, True, "few"),
    ([3000, 1500], 1025, 2, 100, 2, 64, 32, True, "few"),
    ([500, 4100], 300, 10, 290, 1, 256, 16, False, "random"),
    ([5000], 4999, 0, 0, 3, 128, 256, False, "special"),
    ([2500, 20], 4, 2, 2, 2, 64, 128, True, "special"),
    ([6000, 7001], 6500, 4, 64, 2, 64, 16, False, "random"),
    ([9000], 2100, 0, 50, 1, 64, 64, False, "rising"),
]


def weights_of(kind, g, shape):
    w = torch.rand(shape, generator=g, device=DEV)
    if kind == "equal":
        w.fill_(0.25)
    elif kind == "few":
        w = (w * 3).floor() / 4
    elif kind == "rising":
        w = torch.arange(shape[-1], device=DEV, dtype=F32).expand(shape).contiguous()
    elif kind == "special":
        w = (w * 4).floor() - 2
        pick = torch.rand(shape, generator=g, device=DEV)
        w = torch.where(pick < 0.1, float("nan"), w)
        w = torch.where((pick > 0.1) & (pick < 0.2), float("inf"), w)
        w = torch.where((pick > 0.2) & (pick < 0.3), -float("inf"), w)
        w = torch.where((pick > 0.3) & (pick < 0.4), -0.0, w)
    return w


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", EVICT)
def test_evict(fa, case, in_place):
    lens, budget, first, recent, Hkv, d, ps, fp8, kind = case
    B, g = len(lens), gen(50)
    seen = torch.tensor([n + 77 for n in lens], device=DEV, dtype=I32)
    cache = make_cache(fa, 51, lens, Hkv, d, ps, fp8, weight=True, seen=seen)
    cap = cache.max_pages * ps
    cache.weight.copy_(weights_of(kind, g, (B, Hkv, cap)))
    cache.order.copy_(torch.rand((B, Hkv, cap + 77), generator=g, device=DEV).argsort(-1)[..., :cap])
    for b in range(B):   # distinct arrival numbers below seen
        n = lens[b]
        for h in range(Hkv):
            cache.order[b, h, :n] = torch.randperm(n + 77, generator=g, device=DEV)[:n].to(I32)
    w0, o0 = cache.weight.clone(), cache.order.clone()
    k0, v0 = cache.k.clone(), cache.v.clone()
    kw = {}
    if not in_place:
        kw = dict(weight_out=torch.full_like(w0, -9), order_out=torch.full_like(o0, -9), lens_out=torch.full_like(cache.lens, -9))
    kept = fa.fa_cache_evict(cache, budget, n_first=first, n_recent=recent, **kw)
    assert fa.fa_sync_status() == fa.FA_OK
    w1, o1, l1 = (cache.weight, cache.order, cache.lens) if in_place else (kw["weight_out"], kw["order_out"], kw["lens_out"])
    ek, ev = k0.clone(), v0.clone()
    for b in range(B):
        n, end = lens[b], min(lens[b], budget)
        assert int(l1[b]) == end
        if not in_place:
            assert int(cache.lens[b]) == n
        table = cache.block_table[b].long()
        for h in range(Hkv):
            src = R.evict(w0[b, h].cpu().numpy(), o0[b, h].cpu().numpy(), n, n + 77, budget, first, recent)
            assert kept[b, h].tolist() == src + [-1] * (budget - end)
            src_t = torch.tensor(src, device=DEV, dtype=torch.int64)
            assert torch.equal(w1[b, h, :end].view(I32), w0[b, h][src_t].view(I32))
            assert torch.equal(o1[b, h, :end], o0[b, h][src_t])
            rest_w, rest_o = (w0, o0) if in_place else (torch.full_like(w0, -9), torch.full_like(o0, -9))
            assert torch.equal(w1[b, h, end:].view(I32), rest_w[b, h, end:].view(I32)) and torch.equal(o1[b, h, end:], rest_o[b, h, end:])
            j = torch.arange(end, device=DEV)
            if end:
                ek[table[j // ps], h, j % ps] = k0[table[src_t // ps], h, src_t % ps]
                ev[table[j // ps], h, j % ps] = v0[table[src_t // ps], h, src_t % ps]
    assert torch.equal(cache.k.view(torch.uint8), ek.view(torch.uint8))
    assert torch.equal(cache.v.view(torch.uint8), ev.view(torch.uint8))


@pytest.mark.parametrize("n,budget", [(261000, 130000), (270000, 100001)])
def test_evict_longest(fa, n, budget):
    """The most entries that fit a cluster's shared memory, and more."""
    cache = make_cache(fa, 54, [n], 1, 64, 256, weight=True)
    cache.weight.copy_(weights_of("few", gen(55), tuple(cache.weight.shape)) + (cache.weight < 0.5))
    w0, k0 = cache.weight.clone(), cache.k.clone()
    kept = fa.fa_cache_evict(cache, budget, n_first=4, n_recent=1000)
    assert fa.fa_sync_status() == fa.FA_OK and int(cache.lens[0]) == budget
    order = np.arange(n)
    src = R.evict(w0[0, 0].cpu().numpy(), order, n, n, budget, 4, 1000)
    assert kept[0, 0].tolist() == src
    src_t, j, table = torch.tensor(src, device=DEV), torch.arange(budget, device=DEV), cache.block_table[0].long()
    assert torch.equal(cache.weight[0, 0, :budget], w0[0, 0][src_t])
    assert torch.equal(cache.k[table[j // 256], 0, j % 256], k0[table[src_t // 256], 0, src_t % 256])


def test_evict_without_order(fa):
    cache = make_cache(fa, 52, [300, 10], 2, 64, 16, weight=True)
    bare = fa.KVCache(cache.k, cache.v, cache.block_table, cache.lens, weight=cache.weight)
    w0 = cache.weight.clone()
    kept = fa.fa_cache_evict(bare, 64)
    assert fa.fa_sync_status() == fa.FA_OK and bare.lens.tolist() == [64, 10]
    for b, n in ((0, 300), (1, 10)):
        for h in range(2):
            src = R.evict(w0[b, h].cpu().numpy(), None, n, n, 64, 0, 0)
            assert kept[b, h, :len(src)].tolist() == src


@pytest.mark.parametrize("budget", [90, 20])
def test_evict_bad_lengths(fa, budget):
    """Few moves (copied by the selection) and many: a length out of range stays as it is."""
    for in_place in (False, True):
        cache = make_cache(fa, 56, [100, 100, 60], 1, 64, 16, weight=True, width=13 if budget == 20 else 8)
        cache.lens[0] = -1
        cache.lens[1] = cache.max_pages * 16 + 5
        out = cache.lens if in_place else torch.zeros_like(cache.lens)
        fa.fa_cache_evict(cache, budget, lens_out=out)
        assert fa.fa_sync_status() == fa.FA_ERR_BAD_INDEX
        assert out.tolist() == [-1, cache.max_pages * 16 + 5, min(60, budget)]


def test_evict_bad_lengths_and_pages(fa):
    cache = make_cache(fa, 53, [100, 100, 100], 1, 64, 16, weight=True)
    cache.lens[0] = -1
    cache.lens[1] = cache.max_pages * 16 + 5
    cache.weight[2, 0] = torch.arange(cache.weight.shape[-1], device=DEV, dtype=F32)   # the last 20 stay
    cache.block_table[2, 5] = cache.num_pages + 3           # slots 80 .. 95
    k0, w0 = cache.k.clone(), cache.weight.clone()
    kept = fa.fa_cache_evict(cache, 20)
    assert fa.fa_sync_status() == fa.FA_ERR_BAD_INDEX
    assert torch.all(kept[:2] == -1) and torch.equal(cache.weight[:2], w0[:2])
    assert kept[2, 0].tolist() == list(range(80, 100))
    p = cache.block_table[2].long()
    moved = cache.k[p[0], 0], cache.k[p[1], 0, :4]
    assert torch.equal(moved[0], k0[p[0], 0])               # from the bad page: left as it was
    assert torch.equal(moved[1], k0[p[6], 0, :4])


# ---------------------------------------------------------------- the binding's two ways
def test_both_ways_of_calling(fa):
    """The compiled checks and the ones that say what is wrong make the same calls."""
    g = gen(80)
    spec = fa.rope_spec(64, (8, 24))
    q, k = randn(g, 2, 4, 3, 64), randn(g, 2, 2, 3, 64)
    pos = torch.randint(0, 99, (2, 2, 3), generator=g, device=DEV).to(I32)
    out = []
    for way in (0, 1):
        cache = make_cache(fa, 81, [200, 77], 2, 64, 16, weight=True)
        qo, ko, q2 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
        o, lse = torch.empty_like(q), torch.empty((2, 4, 3), device=DEV)
        ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, 4, 3, True), dtype=torch.uint8, device=DEV)
        kept = torch.empty((2, 2, 64), dtype=I32, device=DEV)
        if way == 0:
            fa.fa_rope(q, qo, pos, spec, k=k, k_out=ko)
            fa.fa_cache_append(cache, k, k, pos, spec, q=q, q_out=q2)
            fa.fa_decode_paged(cache, q2, o, lse, 0.125, ws, accumulate=True)
            fa.fa_cache_evict(cache, 64, kept=kept, n_recent=3)
        else:
            fa._rope("fa_rope", q, qo, pos, spec, k, ko, 0, None)
            fa._append(cache, k, k, pos, spec, q, q2, None, torch.cuda.current_stream())
            fa._decode(cache, q2, o, lse, 0.125, ws, True, True, torch.cuda.current_stream().cuda_stream)
            fa._evict(cache, 64, cache.weight, cache.order, cache.lens, kept, 0, 3, None)
        assert fa.fa_sync_status() == fa.FA_OK
        out.append([qo, ko, q2, o, lse, kept, cache.k.view(torch.uint8), cache.weight, cache.order, cache.lens])
    assert all(torch.equal(a, b) for a, b in zip(*out))
    # the compiled way refuses by None, not by a wrong call; a status comes back as an error
    assert fa._fa_py.rope(spec._ref, q.half(), q, None, None, pos, 0, None) is None
    assert fa._fa_py.rope(spec._ref, q, q[:, :3], None, None, pos, 0, None) is None
    assert fa._fa_py.rope(spec._ref, q, q, None, None, pos.long(), 0, None) is None
    assert fa._fa_py.rope(spec._ref, q.cpu(), q.cpu(), None, None, pos.cpu(), 0, None) is None
    assert fa._fa_py.append(cache._ref, cache._index, k, q, None, None, None, None, None, None) is None
    assert fa._fa_py.decode(cache._ref, cache._index, q, o, lse.half(), 0.1, ws, True, False, None) is None
    assert fa._fa_py.decode(cache._ref, cache._index, q, o, lse, 0.1, "no", True, False, None) is None
    assert fa._fa_py.evict(cache._ref, cache._index, 63, cache.weight, cache.order, cache.lens, kept, 0, 0, None) is None
    with pytest.raises(fa.FAError):
        fa.fa_decode_paged(cache, q, o, lse, -1.0, ws)
    with pytest.raises(TypeError):
        fa.fa_rope(q.half(), qo, pos, spec)
    with pytest.raises(ValueError):
        fa.fa_cache_append(cache, k, q)


# ---------------------------------------------------------------- nothing outside the buffers
class Guarded:
    """Buffers in the middle of larger ones; `intact()`: nothing around them was written."""

    def __init__(self):
        self.all = []

    def like(self, t, fill=None):
        n, pad = t.numel() * t.element_size(), 1 << 16
        raw = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)
        self.all.append((raw, n, pad))
        view = raw[pad:pad + n].view(t.dtype).view(t.shape)
        if fill is None:
            view.copy_(t)
        return view

    def intact(self):
        return all(bool((raw[:pad] == 0xA5).all()) and bool((raw[pad + n:] == 0xA5).all()) for raw, n, pad in self.all)


@pytest.mark.parametrize("lens,Hq,Hkv,d,ps,Tq,fp8", [
    ([1, 63, 2049, 0], 8, 2, 128, 16, 1, False), ([5000], 16, 1, 64, 64, 7, True), ([130, 700], 4, 4, 256, 32, 3, False),
    ([900] * 40, 32, 8, 128, 16, 1, False), ([9001, 12000, 20000, 32768], 8, 8, 128, 64, 1, False)])
def test_nothing_outside_the_buffers(fa, lens, Hq, Hkv, d, ps, Tq, fp8):
    g, rnd = Guarded(), gen(70)
    base = make_cache(fa, 71, lens, Hkv, d, ps, fp8, weight=True, extra_pages=0)
    B = base.B
    cache = fa.KVCache(g.like(base.k), g.like(base.v), g.like(base.block_table), g.like(base.lens), base.k_scale, base.v_scale,
                       g.like(base.weight), g.like(base.order), g.like(base.lens))
    q = randn(rnd, B, Hq, Tq, d)
    qo, o, lse = g.like(q), g.like(q), g.like(torch.empty((B, Hq, Tq), device=DEV))
    spec = fa.rope_spec(d)
    pos = torch.randint(0, 9999, (1, B, Tq), generator=rnd, device=DEV).to(I32)
    new = torch.minimum(cache.lens, torch.full_like(cache.lens, Tq))
    fa.fa_cache_append(cache, randn(rnd, B, Hkv, Tq, d), randn(rnd, B, Hkv, Tq, d), pos, spec, q=q, q_out=qo, new_lens=new)
    fa.fa_rope(q, g.like(q), pos, spec, k=q, k_out=g.like(q))
    for acc in (False, True):
        ws = g.like(torch.empty(fa.fa_decode_paged_workspace_bytes(cache, Hq, Tq, acc), dtype=torch.uint8, device=DEV), fill=0)
        fa.fa_decode_paged(cache, qo, o, lse, 0.1, ws, accumulate=acc)
    assert fa.fa_sync_status() == fa.FA_OK and g.intact()
    for budget in (max(max(lens) - 16, 1), max(max(lens) // 3, 1)):
        kept = g.like(torch.empty((B, Hkv, budget), dtype=I32, device=DEV))
        fa.fa_cache_evict(cache, budget, g.like(cache.weight), g.like(cache.order), g.like(cache.lens), kept, n_recent=1)
        assert fa.fa_sync_status() == fa.FA_OK and g.intact()
        fa.fa_cache_evict(cache, budget, kept=kept, n_first=1)
        assert fa.fa_sync_status() == fa.FA_OK and g.intact()


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [False, True])
def test_serving_steps(fa, fp8):
    """Prompts of different lengths, then steps of append, decode with weights and evict as a
    serving loop runs them (the step captured once and replayed), followed entry by entry."""
    B, Hq, Hkv, d, ps, budget, steps = 3, 8, 2, 64, 16, 48, 40
    g = gen(60)
    scales = (torch.tensor([0.01, 0.02], device=DEV), torch.tensor([0.015, 0.01], device=DEV)) if fp8 else (None, None)
    cache = fa.alloc_kv_cache(B, Hkv, d, budget + 16, ps, *scales, weight=True)
    spec = fa.rope_spec(d, (8, 12, 12))
    freqs, axis = freqs_of(d), [0] * 8 + [1] * 12 + [2] * 12
    prompt = [30, 7, 60]
    T = max(prompt)
    k, v = randn(g, B, Hkv, T, d), randn(g, B, Hkv, T, d)
    pos = torch.arange(T, device=DEV, dtype=I32).expand(3, B, T).contiguous()
    new = torch.tensor(prompt, device=DEV, dtype=I32)
    cache.lens.add_(new)
    cache.seen.add_(new)
    fa.fa_cache_append(cache, k, v, pos, spec, new_lens=new)
    q1, k1, v1 = (torch.empty((B, h, 1, d), device=DEV, dtype=BF16) for h in (Hq, Hkv, Hkv))
    pos1 = torch.empty((3, B, 1), device=DEV, dtype=I32)
    qr, o, lse = torch.empty_like(q1), torch.empty_like(q1), torch.empty((B, Hq, 1), device=DEV)
    ws = torch.empty(fa.fa_decode_paged_workspace_bytes(cache, Hq, 1, True), dtype=torch.uint8, device=DEV)
    kept = torch.empty((B, Hkv, budget), dtype=I32, device=DEV)

    def step():
        cache.lens.add_(1)
        cache.seen.add_(1)
        fa.fa_cache_append(cache, k1, v1, pos1, spec, q=q1, q_out=qr)
        fa.fa_decode_paged(cache, qr, o, lse, d ** -0.5, ws, accumulate=True)
        fa.fa_cache_evict(cache, budget, kept=kept, n_first=2, n_recent=8)

    state = [t.clone() for t in (cache.lens, cache.seen, cache.k, cache.v, cache.weight, cache.order)]
    for t in (q1, k1, v1, pos1):
        t.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((cache.lens, cache.seen, cache.k, cache.v, cache.weight, cache.order), state):
        t.copy_(s)

    for i in range(steps):
        q1.copy_(randn(g, B, Hq, 1, d) * 3)
        k1.copy_(randn(g, B, Hkv, 1, d))
        v1.copy_(randn(g, B, Hkv, 1, d))
        pos1.copy_((torch.tensor(prompt, device=DEV, dtype=I32) + i)[None, :, None].expand(3, B, 1))
        n0, s0 = cache.lens.tolist(), cache.seen.tolist()
        w0, o0 = cache.weight.clone(), cache.order.clone()
        had = [entries(cache, b, n0[b]) for b in range(B)]
        graph.replay()
        assert fa.fa_sync_status() == fa.FA_OK
        for b in range(B):
            n = n0[b] + 1
            kk, _ = R.rotate(to64(k1[b]), pos1[:, b].cpu().numpy(), freqs, axis)
            qq, tq = R.rotate(to64(q1[b]), pos1[:, b].cpu().numpy(), freqs, axis)
            within(to64(qr[b]), qq, tq, 2.0 ** -8)
            end = min(n, budget)
            for h in range(Hkv):
                src = kept[b, h, :end].tolist()
                # the new token's row as the cache holds it: wherever it ended up, within its type's rounding
                where = src.index(n - 1)
                kb, vb = entries(cache, b, end)
                rows_k = np.concatenate([had[b][0][h], kb[h, where:where + 1]])
                rows_v = np.concatenate([had[b][1][h], vb[h, where:where + 1]])
                half = 2.0 ** -4 if fp8 else 2.0 ** -8
                floor = 2.0 ** -10 * float(scales[0][h]) if fp8 else 1e-6
                within(rows_k[-1], kk[h, 0], np.full(d, floor + 4e-6), half)
                G = Hq // Hkv
                ro, rl, rw, to, tl, tw = R.attend(to64(qr[b, h * G:(h + 1) * G]), rows_k[None], rows_v[None], d ** -0.5, True, G)
                within(to64(o[b, h * G:(h + 1) * G]), ro, to, 2.0 ** -8)
                within(to64(lse[b, h * G:(h + 1) * G]), rl, tl)
                w = to64(w0[b, h, :n]).copy()
                w[-1] = 0
                w += rw[0]
                order = o0[b, h, :n].cpu().numpy().copy()
                order[-1] = s0[b]
                got_w = to64(cache.weight[b, h, :end])
                within(got_w, w[src], tw[0][src] + 8 * R.U * np.abs(w[src]))
                assert cache.order[b, h, :end].tolist() == order[src].tolist()
                # what stays is right up to ties of the weights' tolerance
                gone = sorted(set(range(n)) - set(src))
                prot = (order < 2) | (order >= s0[b] + 1 - 8)
                assert not prot[gone].any()
                free = [s for s in src if not prot[s]]
                if gone and free:
                    assert w[gone].max() <= w[free].min() + 1e-4
                assert np.array_equal(kb[h], rows_k[src]) and np.array_equal(vb[h], rows_v[src])
    assert cache.lens.tolist() == [budget] * B or min(prompt) + steps < budget
