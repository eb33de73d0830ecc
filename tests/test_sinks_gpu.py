"""Attention under a causal window with sinks (fa_fwd_sinks, fa_bwd_sinks) against a 64-bit reference
(tests/sinks_ref.py, which derives the tolerances): every element, rows without keys, sinks and windows at and
across tile edges, key blocks with sinks in one piece and in parts."""
import numpy as np
import pytest
import torch

import sinks_ref as S
from gpu_util import to64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def data(B, H, Tq, Tk, d, seed):
    g = torch.Generator(DEV).manual_seed(seed)
    return [torch.randn((B, H, t, d), generator=g, device=DEV).to(BF16) for t in (Tq, Tk, Tk, Tq)]


def within(got, ref, tol, what):
    assert np.isfinite(got).all(), what
    x = np.abs(got - ref) - tol
    assert x.max(initial=-1.0) <= 0, (what, float(x.max()), float(np.abs(got - ref).max()))


SHAPES = [  # B, H, Tq, Tk, d
    (1, 1, 1, 1, 64), (1, 2, 1, 700, 128), (2, 1, 129, 129, 64), (1, 2, 700, 700, 128), (1, 1, 300, 901, 256), (1, 2, 300, 900, 64),
    (1, 1, 900, 300, 128), (1, 1, 1500, 1500, 64), (1, 1, 520, 1031, 256),
]
MASKS = [(0, 1), (0, 0), (100, 4), (127, 128), (128, 129), (300, 3), (1, 400), (640, 64), (5000, 7), (200, 5000), (-1, 9)]


@pytest.mark.parametrize("left,sinks", MASKS)
@pytest.mark.parametrize("B,H,Tq,Tk,d", SHAPES)
def test_forward_and_backward(fa, B, H, Tq, Tk, d, left, sinks):
    q, k, v, do = data(B, H, Tq, Tk, d, Tq + 3 * Tk + d + left)
    scale = d ** -0.5
    o, lse = torch.full_like(q, float("nan")), torch.full((B, H, Tq), float("nan"), device=DEV)
    fa.fa_fwd_sinks(q, k, v, o, lse, left, sinks, scale)
    assert fa.fa_sync_status() == fa.FA_OK
    grads = None
    if d < 256:
        grads = [torch.full_like(t, float("nan")) for t in (q, k, v)]
        n = fa.fa_bwd_sinks_workspace_bytes(B, H, Tq, Tk, d, left, sinks)
        assert n >= fa.fa_bwd_workspace_bytes(B, H, Tq, Tk, d)
        ws = torch.full((n + 256,), 255, dtype=torch.uint8, device=DEV)
        fa.fa_bwd_sinks(q, k, v, o, lse, do, *grads, left, sinks, scale, ws[:n])
        assert fa.fa_sync_status() == fa.FA_OK and torch.all(ws[n:] == 255)
    see = S.visible(Tq, Tk, left, sinks)
    for b in range(B):
        for h in range(H):
            x = [to64(t[b, h]) for t in (q, k, v, do)]
            ro, rl, to, tl, _, _ = S.forward(*x[:3], scale, see)
            within(to64(o[b, h]), ro, to, "o")
            got = to64(lse[b, h])
            dead = ~np.isfinite(rl)
            assert np.all(got[dead] == -np.inf) and np.all(to64(o[b, h])[dead] == 0)
            within(got[~dead], rl[~dead], tl[~dead], "lse")
            if grads:
                ref, tol = S.backward(*x, scale, see)
                for name, g, r, t in zip(("dq", "dk", "dv"), grads, ref, tol):
                    within(to64(g[b, h]), r, t + S.BF * (np.abs(r) + t), name)


def test_gradients_against_differences(fa):
    """The gradients' products with random directions against difference quotients of the 64-bit forward."""
    d, T, left, sinks = 64, 200, 20, 3
    q, k, v, do = data(1, 1, T, T, d, 1)
    o, lse = fa.attention_forward(q, k, v, False, 0.125, window=(left, 0), sinks=sinks)
    grads = fa.attention_backward(q, k, v, o, lse, do, False, 0.125, window=(left, 0), sinks=sinks)
    see = S.visible(T, T, left, sinks)
    x = [to64(t[0, 0]) for t in (q, k, v, do)]
    _, tol = S.backward(*x, 0.125, see)
    rng = np.random.default_rng(0)
    for i in range(3):
        g = to64(grads[i][0, 0])
        for _ in range(3):
            w, h = rng.standard_normal(g.shape), 1e-5

            def f(sign):
                y = list(x[:3])
                y[i] = y[i] + sign * h * w
                return (x[3] * S.forward(*y, 0.125, see)[0]).sum()
            room = ((tol[i] + S.BF * (np.abs(g) + tol[i])) * np.abs(w)).sum()
            # the quotient's own error: h^2 times a third derivative, and 2^-53 / h of f's terms
            assert abs((f(1) - f(-1)) / (2 * h) - (g * w).sum()) <= room + 1e-8 * (np.abs(g * w).sum() + np.abs(x[3]).sum() * 8)


def test_parts_are_used_and_the_sums_repeat(fa):
    """The block with the sinks is cut into parts, unless a window's block is as long.  dK, dV and, in deterministic
    mode, dQ repeat bit for bit."""
    cut = fa.fa_bwd_sinks_workspace_bytes(1, 1, 3000, 3000, 128, 255, 4)
    assert cut > fa.fa_bwd_workspace_bytes(1, 1, 3000, 3000, 128)
    assert fa.fa_bwd_sinks_workspace_bytes(8, 32, 4096, 4096, 128, 4000, 4) == fa.fa_bwd_workspace_bytes(8, 32, 4096, 4096, 128)
    q, k, v, do = data(1, 1, 3000, 3000, 128, 2)
    kw = dict(window=(255, 0), sinks=4)
    o, lse = fa.attention_forward(q, k, v, False, 0.1, **kw)
    first = fa.attention_backward(q, k, v, o, lse, do, False, 0.1, deterministic=True, **kw)
    again = fa.attention_backward(q, k, v, o, lse, do, False, 0.1, deterministic=True, **kw)
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    plain = fa.attention_backward(q, k, v, o, lse, do, False, 0.1, **kw)
    assert torch.equal(first[1], plain[1]) and torch.equal(first[2], plain[2])
    see = S.visible(3000, 3000, 255, 4)
    x = [to64(t[0, 0]) for t in (q, k, v, do)]
    ref, tol = S.backward(*x, 0.1, see)
    for g, r, t in zip(first, ref, tol):
        within(to64(g[0, 0]), r, t + S.BF * (np.abs(r) + t), "deterministic")
    assert fa.fa_sync_status() == fa.FA_OK


def test_no_sinks_is_the_window_and_no_window_is_causal(fa):
    for d in (64, 128, 256):
        q, k, v, do = data(2, 2, 777, 900, d, 3)
        a = fa.attention_forward(q, k, v, False, 0.1, window=(200, 0))
        o, lse = torch.empty_like(q), torch.empty((2, 2, 777), device=DEV)
        fa.fa_fwd_sinks(q, k, v, o, lse, 200, 0, 0.1)
        assert torch.equal(a[0], o) and torch.equal(a[1], lse)
        a = fa.attention_forward(q, k, v, True, 0.1)
        b = fa.attention_forward(q, k, v, True, 0.1, sinks=5)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert fa.fa_sync_status() == fa.FA_OK


def test_keys_outside_of_every_row_are_not_read(fa):
    """Key blocks between the sinks and the window may hold anything."""
    q, k, v, do = data(1, 2, 100, 2000, 128, 4)
    want = fa.attention_forward(q, k, v, False, 0.1, window=(300, 0), sinks=4)
    grads = fa.attention_backward(q, k, v, *want, do, False, 0.1, window=(300, 0), sinks=4, deterministic=True)
    k[:, :, 128:1536] = float("nan")
    v[:, :, 128:1536] = float("inf")
    got = fa.attention_forward(q, k, v, False, 0.1, window=(300, 0), sinks=4)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dq, dk, dv = fa.attention_backward(q, k, v, *want, do, False, 0.1, window=(300, 0), sinks=4)
    assert torch.equal(dk, grads[1]) and torch.equal(dv, grads[2]) and torch.all(dk[:, :, 128:1536] == 0)
    assert fa.fa_sync_status() == fa.FA_OK


def test_captured_and_on_another_stream(fa):
    q, k, v, do = data(1, 1, 1500, 1500, 64, 5)
    o, lse, dq, dk, dv = torch.empty_like(q), torch.empty((1, 1, 1500), device=DEV), *(torch.empty_like(t) for t in (q, k, v))
    ws = torch.empty(fa.fa_bwd_sinks_workspace_bytes(1, 1, 1500, 1500, 64, 100, 4), dtype=torch.uint8, device=DEV)

    def step(stream=None):
        fa.fa_fwd_sinks(q, k, v, o, lse, 100, 4, 0.125, stream)
        fa.fa_bwd_sinks(q, k, v, o, lse, do, dq, dk, dv, 100, 4, 0.125, ws, True, stream)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    torch.cuda.current_stream().wait_stream(side)
    first = [t.clone() for t in (o, lse, dq, dk, dv)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in (o, lse, dq, dk, dv):
        t.zero_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(first, (o, lse, dq, dk, dv)))
    q.neg_()
    graph.replay()
    want = fa.attention_forward(q, k, v, False, 0.125, window=(100, 0), sinks=4)
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    side.wait_stream(torch.cuda.current_stream())
    want = fa.attention_forward(q, k, v, False, 0.125, window=(100, 0), sinks=4, stream=side)
    grads = fa.attention_backward(q, k, v, *want, do, False, 0.125, window=(100, 0), sinks=4, stream=side, deterministic=True)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip((o, lse, dq, dk, dv), (*want, *grads)))
    assert fa.fa_sync_status() == fa.FA_OK


def test_refusals(fa):
    q = torch.randn(1, 1, 64, 64, device=DEV).to(BF16)
    o, lse, ws = torch.empty_like(q), torch.empty(1, 1, 64, device=DEV), torch.empty(1 << 20, dtype=torch.uint8, device=DEV)
    for left, sinks in ((-2, 1), (5, -1)):
        with pytest.raises(fa.FAError) as e:
            fa.fa_fwd_sinks(q, q, q, o, lse, left, sinks, 0.1)
        assert e.value.status == fa.FA_ERR_INVALID_ARG
    with pytest.raises(fa.FAError):
        fa.fa_fwd_sinks(q, q, q, q, lse, 5, 1, 0.1)
    for bad in (dict(causal=False, sinks=2), dict(causal=True, window=(5, 0), sinks=2), dict(causal=False, window=(5, 1), sinks=2)):
        with pytest.raises(ValueError):
            fa.attention_forward(q, q, q, scale=0.1, **bad)
    k = q.clone()
    out = [torch.empty_like(q) for _ in range(3)]
    with pytest.raises(fa.FAError):
        fa.fa_bwd_sinks(q, k, k, o, lse, q, *out, 5, 1, 0.1, ws[:256])
    assert fa.fa_sync_status() == fa.FA_OK
