"""Norms of query and key heads with the rotation (fa_norm_rope, its backward, and on the way into the
cache) against 64-bit references (tests/norm_ref.py, which derives the tolerances)."""
import numpy as np
import pytest
import torch

import norm_ref as N
import paged_ref as R
from gpu_util import to64
from test_cache_gpu import freqs_of, gen, make_cache, randn, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-5


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


CASES = [
    # B, Hq, Hk, T, d, rot, axes, interleaved, packed, dtype, weights' dtype (None: no weights), far
    (1, 1, 1, 1, 64, 64, 1, False, False, BF16, BF16, 0),
    (2, 3, 1, 33, 128, 128, 3, False, True, BF16, F32, 70000),
    (1, 5, 2, 129, 256, 256, 4, True, False, BF16, None, 1000000),
    (3, 2, 2, 65, 64, 32, 2, True, True, F32, F32, 0),
    (1, 17, 3, 257, 128, 48, 3, False, False, F32, BF16, 2000000000),
    (2, 1, 0, 70, 256, 16, 1, False, False, F32, F32, -2000000000),
    (1, 40, 8, 1500, 128, 128, 8, True, True, BF16, BF16, 10),
    (4, 0, 3, 31, 64, 64, 1, False, False, BF16, F32, 0),
    (1, 700, 2, 3, 64, 48, 1, False, False, BF16, BF16, 5),
]


def case(c, seed):
    B, Hq, Hk, T, d, rot, axes, inter, packed, dt, wt, far = c
    g = gen(seed)
    freqs = freqs_of(rot)
    axis = [i * axes // (rot // 2) for i in range(rot // 2)]
    pos = (torch.randint(-50, 5000, (axes, B, T), generator=g, device=DEV) + far).to(I32)

    def pair(scale=1.0):
        if packed:
            x = randn(g, B, T, Hq + Hk, d, dtype=dt).mul_(scale).transpose(1, 2)
            return x[:, :Hq], x[:, Hq:]
        return randn(g, B, Hq, T, d, dtype=dt).mul_(scale), randn(g, B, Hk, T, d, dtype=dt).mul_(scale)
    q, k = pair(3.0)
    if B * Hq * T > 4:
        q[0, 0, 0] = 0.0                     # a row of zeros: eps alone
        q[0, 0, -1] = 1e-4
    w = [None if wt is None else (1.0 + 0.5 * randn(g, d, dtype=F32)).to(wt) for _ in range(2)]
    return q, k, pos, freqs, axis, w, pair


def w64(w, d):
    return np.ones(d) if w is None else to64(w)


@pytest.mark.parametrize("c", CASES)
def test_forward(fa, c):
    B, Hq, Hk, T, d, rot, axes, inter, packed, dt, wt, far = c
    q, k, pos, freqs, axis, w, _ = case(c, 5)
    spec, norm = fa.RopeSpec(d, freqs, axis, inter), fa.HeadNorm(d, *w, eps=EPS)
    qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    fa.fa_norm_rope(q, qo, pos, spec, norm, k=k, k_out=ko)
    assert fa.fa_sync_status() == fa.FA_OK
    half = 2.0 ** -8 if dt == BF16 else N.U
    for x, y, ww in ((q, qo, w[0]), (k, ko, w[1])):
        for b in range(B):
            ref, tol = N.forward(to64(x[b]), w64(ww, d), norm._c.eps, pos[:, b].cpu().numpy(), freqs, axis, inter)
            within(to64(y[b]), ref, tol, half)


@pytest.mark.parametrize("c", CASES)
def test_backward(fa, c):
    B, Hq, Hk, T, d, rot, axes, inter, packed, dt, wt, far = c
    q, k, pos, freqs, axis, w, pair = case(c, 6)
    spec, norm = fa.RopeSpec(d, freqs, axis, inter), fa.HeadNorm(d, *w, eps=EPS)
    gq, gk = pair()
    dq, dk = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    dw = [None if x is None else torch.full((d,), float("nan"), device=DEV) for x in w]
    ws = torch.full((fa.fa_norm_rope_bwd_workspace_bytes(d),), 255, dtype=torch.uint8, device=DEV)
    fa.fa_norm_rope_bwd(gq, q, dq, pos, spec, norm, gk, k, dk, *dw, workspace=ws)
    assert fa.fa_sync_status() == fa.FA_OK
    half = 2.0 ** -8 if dt == BF16 else N.U
    for dy, x, dx, ww, dww in ((gq, q, dq, w[0], dw[0]), (gk, k, dk, w[1], dw[1])):
        ref_w, tol_w, mag = np.zeros(d), np.zeros(d), np.zeros(d)
        for b in range(B):
            ref, terms, tol, tw, m = N.backward(to64(dy[b]), to64(x[b]), w64(ww, d), norm._c.eps, pos[:, b].cpu().numpy(), freqs, axis, inter)
            within(to64(dx[b]), ref, tol, half)
            ref_w, tol_w, mag = ref_w + terms.sum((0, 1)), tol_w + tw.sum((0, 1)), mag + m.sum((0, 1))
        if dww is not None:
            within(to64(dww), ref_w, tol_w + x.shape[0] * x.shape[1] * x.shape[2] * N.U * mag, N.U)


def test_gradients_against_differences(fa):
    """sum(dy y(x, w)) changes along random directions as dx and dw say: the 64-bit forward's difference quotient."""
    c = (1, 2, 1, 5, 64, 32, 2, False, False, F32, F32, 3)
    q, k, pos, freqs, axis, w, pair = case(c, 7)
    spec, norm = fa.RopeSpec(64, freqs, axis), fa.HeadNorm(64, *w, eps=EPS)
    q[0, 0, 0] = 0.01      # not the row of zeros, where the curvature is 1 / eps
    q[0, 0, -1] = 0.02
    gq, gk = pair()
    dq, dk, dqw, dkw = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    rng = np.random.default_rng(0)
    p = pos[:, 0].cpu().numpy()
    for dy, x, ww, dx, dw in ((gq, q, w[0], dq, dqw), (gk, k, w[1], dk, dkw)):
        dy, x, ww, dx, dw = (to64(t) for t in (dy, x, ww, dx, dw))
        _, _, tol, tw, mag = N.backward(dy[0], x[0], ww, norm._c.eps, p, freqs, axis, False)
        tw = tw.sum((0, 1)) + x.shape[1] * x.shape[2] * N.U * mag.sum((0, 1)) + N.U * np.abs(dw)

        def f(x, ww):
            return (dy * N.forward(x[0], ww, norm._c.eps, p, freqs, axis, False)[0]).sum()
        for _ in range(4):
            vx, vw, h = rng.standard_normal(x.shape) * np.abs(x).mean(-1, keepdims=True), rng.standard_normal(ww.shape), 1e-5
            # central: off by h^2 times a third derivative and 2^-53 / h of f's terms, below 1e-8 of the terms' sum
            for got, room in ((f(x + h * vx, ww) - f(x - h * vx, ww), (tol[None] + N.U * np.abs(dx)) * np.abs(vx)),
                              (f(x, ww + h * vw) - f(x, ww - h * vw), tw * np.abs(vw))):
                want = dx * vx if room.shape == vx.shape else dw * vw
                terms = np.abs(want).sum() + np.abs(dy * N.forward(x[0], ww, norm._c.eps, p, freqs, axis, False)[0]).sum()
                assert abs(got / (2 * h) - want.sum()) <= room.sum() + 1e-8 * terms


def test_same_bits_in_place_and_without_weights_gradients(fa):
    q, k, pos, freqs, axis, w, pair = case(CASES[6], 8)
    spec, norm = fa.RopeSpec(128, freqs, axis, True), fa.HeadNorm(128, *w, eps=EPS)
    gq, gk = pair()
    first = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    again = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    fa.fa_norm_rope_bwd(gq, q, gq, pos, spec, norm, gk, k, gk)      # over the incoming gradients, no dw
    assert torch.equal(gq, first[0]) and torch.equal(gk, first[1])
    qo, ko = fa.norm_rope_forward(q, k, pos, spec, norm)
    fa.fa_norm_rope(q, q, pos, spec, norm, k, k)                    # over its inputs
    assert torch.equal(q, qo) and torch.equal(k, ko)
    one = fa.HeadNorm(128, w[0], None, eps=EPS)                     # weights of q only
    dq, dk, dqw, dkw = fa.norm_rope_backward(gq, gk, qo, ko, pos, spec, one)
    assert dkw is None and dqw.shape == (128,)
    assert fa.fa_sync_status() == fa.FA_OK


def test_no_rows(fa):
    """Without a token the weights' gradients are zeros."""
    spec, norm = fa.rope_spec(64), fa.HeadNorm(64, torch.ones(64, device=DEV), torch.ones(64, device=DEV))
    q, pos = torch.empty((2, 3, 0, 64), device=DEV), torch.empty((1, 2, 0), dtype=I32, device=DEV)
    dw = torch.full((2, 64), float("nan"), device=DEV)
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_bytes(64), dtype=torch.uint8, device=DEV)
    fa.fa_norm_rope(q, q, pos, spec, norm)
    fa.fa_norm_rope_bwd(q, q, q, pos, spec, norm, q, q, q, dw[0], dw[1], ws)
    assert fa.fa_sync_status() == fa.FA_OK and torch.all(dw == 0)


def test_nothing_else_is_written(fa):
    """Strided outputs: the rest of a packed projection's gradient stays."""
    c = (2, 3, 2, 37, 128, 128, 1, False, False, BF16, BF16, 0)
    q, k, pos, freqs, axis, w, pair = case(c, 9)
    spec, norm = fa.RopeSpec(128, freqs, axis), fa.HeadNorm(128, *w, eps=EPS)
    gq, gk = pair()
    want = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    packed = torch.full((2, 37, 3 + 2 + 2, 128), 7.0, dtype=BF16, device=DEV)
    view = packed.transpose(1, 2)
    dw = torch.full((3, 128), 7.0, device=DEV)
    ws = torch.full((fa.fa_norm_rope_bwd_workspace_bytes(128) + 256,), 7, dtype=torch.uint8, device=DEV)
    fa.fa_norm_rope_bwd(gq, q, view[:, :3], pos, spec, norm, gk, k, view[:, 3:5], dw[0], dw[2], ws[:-256])
    assert torch.equal(view[:, :3], want[0]) and torch.equal(view[:, 3:5], want[1]) and torch.all(view[:, 5:] == 7)
    assert torch.equal(dw[0], want[2]) and torch.equal(dw[2], want[3]) and torch.all(dw[1] == 7) and torch.all(ws[-256:] == 7)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("d,T,new", [(128, 1, None), (64, 5, (5, 0, 3)), (256, 40, (40, 17, 1))])
def test_append(fa, codes, d, T, new):
    """New tokens normed and rotated on the way: q_out, and K as the separate calls would write it; V as it is."""
    g = gen(10)
    lens = [50, 41, 77]
    ref, got = (make_cache(fa, 11, lens, 2, d, 16, codes) for _ in range(2))
    spec = fa.rope_spec(d, (d // 8, d // 4, d // 8))
    w = [1.0 + 0.5 * randn(g, d) for _ in range(2)]
    norm = fa.HeadNorm(d, *w, eps=EPS)
    qkv = (3.0 * randn(g, 3, T, 6 + 2 + 2, d)).transpose(1, 2)
    q, k, v = qkv[:, :6], qkv[:, 6:8], qkv[:, 8:]
    pos = torch.randint(0, 9999, (3, 3, T), generator=g, device=DEV).to(I32)
    nl = None if new is None else torch.tensor(new, dtype=I32, device=DEV)
    qo = torch.full((3, 6, T, d), float("nan"), dtype=BF16, device=DEV)
    before = [t.clone() for t in (got.k, got.v)]
    fa.fa_cache_append(got, k, v, pos, spec, q, qo, nl, norm=norm)
    fa.fa_cache_append(ref, k, v, pos, spec, new_lens=nl)          # V, and which rows change
    assert fa.fa_sync_status() == fa.FA_OK
    assert torch.equal(got.v.view(torch.uint8), ref.v.view(torch.uint8))     # bytes: NaN behind the lengths
    changed = torch.zeros(got.k.shape[0], got.page_size, dtype=torch.bool, device=DEV)
    vals = R.e4m3_values()
    for b in range(3):
        nb = T if new is None else new[b]
        for x, ww, heads in ((q, w[0], 6), (k, w[1], 2)):
            y, tol = N.forward(to64(x[b]), to64(ww), norm._c.eps, pos[:, b].cpu().numpy(), [10000.0 ** (-2 * i / d) for i in range(d // 2)],
                               [0] * (d // 8) + [1] * (d // 4) + [2] * (d // 8), False)
            if heads == 6:
                within(to64(qo[b, :, :nb]), y[:, :nb], tol[:, :nb], 2.0 ** -8)
                assert torch.isnan(qo[b, :, nb:]).all()
                continue
            for t in range(nb):
                slot = lens[b] - nb + t
                page, row = int(got.block_table[b, slot // 16]), slot % 16
                changed[page, row] = True
                if codes:
                    for h in range(2):
                        sc = float(got.k_scale[h])
                        have = vals[got.k[page, h, row].cpu().numpy()] * sc
                        want = np.clip(y[h, t], -448 * sc, 448 * sc)
                        within(have, want, tol[h, t] + 2.0 ** -10 * sc, 2.0 ** -4)
                else:
                    within(to64(got.k[page, :, row]), y[:, t], tol[:, t], 2.0 ** -8)
    keep = ~changed
    assert torch.equal(got.k.view(torch.uint8).transpose(1, 2)[keep], before[0].view(torch.uint8).transpose(1, 2)[keep])


def test_both_ways_of_calling(fa):
    q, k, pos, freqs, axis, w, _ = case(CASES[1], 12)
    spec, norm = fa.RopeSpec(128, freqs, axis), fa.HeadNorm(128, *w)
    out = []
    for way in (0, 1):
        qo, ko = torch.empty_like(q), torch.empty_like(k)
        if way == 0:
            fa.fa_norm_rope(q, qo, pos, spec, norm, k, ko)
        else:
            fa._norm_rope(q, qo, pos, spec, norm, k, ko, None)
        out.append((qo, ko))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    if fa._fa_py is not None:
        call = fa._fa_py.norm_rope
        assert call(spec._ref, norm._ref, norm._index, q, qo, k, ko, pos, None) == fa.FA_OK
        assert call(spec._ref, norm._ref, norm._index + 1, q, qo, k, ko, pos, None) is None
        assert call(spec._ref, norm._ref, norm._index, q, qo.float(), k, ko, pos, None) is None
        assert call(spec._ref, norm._ref, norm._index, q, qo, k, None, pos, None) is None
    g = torch.empty((2, 2, 128), device=DEV)
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device=DEV)
    got = []
    for way, f in enumerate((fa.fa_norm_rope_bwd, fa._norm_rope_bwd)):
        dq, dk = torch.empty_like(q), torch.empty_like(k)
        f(qo, q, dq, pos, spec, norm, ko, k, dk, g[way, 0], g[way, 1], ws, None)
        got.append((dq, dk))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]) and torch.equal(g[0], g[1])
    if fa._fa_py is not None:
        call, args = fa._fa_py.norm_rope_bwd, [spec._ref, norm._ref, norm._index, qo, dq, ko, dk, pos, None, q, k, g[0, 0], g[0, 1], ws]
        assert call(*args) == fa.FA_OK
        for at, bad in ((9, q.float()), (10, None), (11, g[0]), (13, None), (2, norm._index + 1)):
            assert call(*args[:at], bad, *args[at + 1:]) is None
    with pytest.raises(ValueError):
        fa.fa_norm_rope(q, qo, pos, spec, fa.HeadNorm(64), k, ko)
    with pytest.raises(ValueError):
        fa.fa_norm_rope(q, qo, pos, spec, fa.HeadNorm(128, w[0].cpu()), k, ko)
    with pytest.raises(ValueError):
        fa.fa_norm_rope_bwd(q, q, qo, pos, spec, norm, dk_weight=torch.empty(128, device=DEV))
    with pytest.raises(ValueError):
        fa.fa_norm_rope_bwd(q, q, qo, pos, spec, norm, dq_weight=torch.empty(128, device=DEV))      # no workspace


def test_weights_with_other_memory(fa):
    """A weight whose data is replaced, as when a module is converted, is read where it is now."""
    q, k, pos, freqs, axis, w, _ = case(CASES[1], 17)
    spec, p = fa.RopeSpec(128, freqs, axis), torch.nn.Parameter(w[0].clone())
    norm = fa.HeadNorm(128, p, p)
    fa.norm_rope_forward(q, k, pos, spec, norm)
    for t in (w[1], w[1].bfloat16()):
        p.data = t.clone()
        assert all(torch.equal(a, b) for a, b in zip(fa.norm_rope_forward(q, k, pos, spec, norm),
                                                     fa.norm_rope_forward(q, k, pos, spec, fa.HeadNorm(128, t, t))))
    p.data = p.data.cpu()
    with pytest.raises(ValueError):
        fa.norm_rope_forward(q, k, pos, spec, norm)
    assert fa.fa_sync_status() == fa.FA_OK


def test_captured_and_on_another_stream(fa):
    """A training step's calls in a graph, replayed with other inputs, and on a stream of their own."""
    q, k, pos, freqs, axis, w, pair = case(CASES[1], 13)
    spec, norm = fa.RopeSpec(128, freqs, axis), fa.HeadNorm(128, *w)
    gq, gk = pair()
    qo, ko, dq, dk = (torch.empty_like(t) for t in (q, k, q, k))
    dw = torch.empty((2, 128), device=DEV)
    ws = torch.empty(fa.fa_norm_rope_bwd_workspace_bytes(128), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        fa.fa_norm_rope(q, qo, pos, spec, norm, k, ko, stream)
        fa.fa_norm_rope_bwd(gq, q, dq, pos, spec, norm, gk, k, dk, dw[0], dw[1], ws, stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (14, 15):
        q.copy_(case(CASES[1], seed)[0])
        norm.q_weight.mul_(1.25)                 # in place, as an optimizer does
        graph.replay()
        want = (*fa.norm_rope_forward(q, k, pos, spec, norm), *fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm))
        assert all(torch.equal(a, b) for a, b in zip(want, (qo, ko, dq, dk, dw[0], dw[1])))
    assert fa.fa_sync_status() == fa.FA_OK
