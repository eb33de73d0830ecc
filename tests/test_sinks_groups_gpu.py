"""Attention under windows, sinks and block masks over many heads, against the 64-bit reference (tests/sinks_ref.py):
more units than SMs, so that a CTA takes several of them in turn (parts of a key block with sinks among them), and more
heads than a group of the launch order, so that there is a second group and a last one with fewer heads.  Every element
of heads of the first, an inner and the last group."""
import numpy as np
import pytest
import torch

import sinks_ref as S
from gpu_util import to64
from test_sinks_gpu import data, fa, within  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attend(fa, x, scale, left, sinks, mask):
    q, k, v, _ = x
    if mask is not None:
        return fa.attention_forward(q, k, v, False, scale, window=(left, 0), block_mask=mask)
    return fa.attention_forward(q, k, v, False, scale, window=(left, 0), sinks=sinks)


def visible(Tq, Tk, left, sinks, mask):
    see = S.visible(Tq, Tk, left, sinks)
    if mask is not None:
        see &= np.kron(mask.cpu().numpy(), np.ones((128, 128)))[:Tq, :Tk] > 0
    return see


def check_forward(x, o, lse, b, h, scale, see):
    q, k, v, _ = (to64(t[b, h]) for t in x)
    ro, rl, to, tl, _, _ = S.forward(q, k, v, scale, see)
    within(to64(o[b, h]), ro, to, ("o", b, h))
    got, dead = to64(lse[b, h]), ~np.isfinite(rl)
    assert np.all(got[dead] == -np.inf) and np.all(to64(o[b, h])[dead] == 0)
    within(got[~dead], rl[~dead], tl[~dead], ("lse", b, h))


# heads: groups of eight and the rest; units of 256 rows (128 at d 256)
@pytest.mark.parametrize("left,sinks", [(255, 4), (255, 130), (0, 1), (700, 0)])
@pytest.mark.parametrize("B,H,Tq,Tk,d", [(1, 11, 4100, 4100, 64), (1, 21, 2000, 2100, 128), (3, 7, 1500, 1300, 256), (2, 9, 2500, 2500, 128)])
def test_forward(fa, B, H, Tq, Tk, d, left, sinks):
    x, scale = data(B, H, Tq, Tk, d, 31 + Tq + left), d ** -0.5
    o, lse = attend(fa, x, scale, left, sinks, None)
    assert fa.fa_sync_status() == fa.FA_OK
    see = visible(Tq, Tk, left, sinks, None)
    for i in (0, 7, 8, B * H - 1):
        check_forward(x, o, lse, i // H, i % H, scale, see)


# 42 heads in groups of four, the last with two; 608 units and more, 152 of them at a time
@pytest.mark.parametrize("deterministic", [False, True])
@pytest.mark.parametrize("left,sinks", [(100, 4), (100, 130), (300, 0)])
@pytest.mark.parametrize("Tq,Tk,d", [(1900, 1900, 64), (1900, 1900, 128), (1700, 2000, 64)])
def test_backward(fa, Tq, Tk, d, left, sinks, deterministic):
    B, H, scale = 2, 21, d ** -0.5
    if sinks:   # the sinks' blocks are cut into parts
        assert fa.fa_bwd_sinks_workspace_bytes(B, H, Tq, Tk, d, left, sinks) > fa.fa_bwd_workspace_bytes(B, H, Tq, Tk, d)
    x = data(B, H, Tq, Tk, d, 32 + Tq + left)
    q, k, v, do = x
    o, lse = attend(fa, x, scale, left, sinks, None)
    grads = fa.attention_backward(q, k, v, o, lse, do, False, scale, deterministic=deterministic, window=(left, 0), sinks=sinks)
    assert fa.fa_sync_status() == fa.FA_OK
    see = visible(Tq, Tk, left, sinks, None)
    for i in (0, 3, 4, 40, 41):
        ref, tol = S.backward(*(to64(t[i // H, i % H]) for t in x), scale, see)
        for name, g, r, t in zip(("dq", "dk", "dv"), grads, ref, tol):
            within(to64(g[i // H, i % H]), r, t + S.BF * (np.abs(r) + t), (name, i))


def test_a_block_mask_over_several_groups(fa):
    """Groups of up to 48 MB: 48 heads forward, 24 backward."""
    B, H, T, d, left = 1, 53, 1900, 128, 5000
    mask = (torch.rand((15, 15), generator=torch.Generator(DEV).manual_seed(33), device=DEV) < 0.5).to(torch.uint8)
    mask[3] = 0
    x, scale = data(B, H, T, T, d, 34), d ** -0.5
    q, k, v, do = x
    o, lse = attend(fa, x, scale, left, 0, mask)
    grads = fa.attention_backward(q, k, v, o, lse, do, False, scale, window=(left, 0), block_mask=mask)
    assert fa.fa_sync_status() == fa.FA_OK
    see = visible(T, T, left, 0, mask)
    for h in (0, 23, 24, 47, 48, 52):
        check_forward(x, o, lse, 0, h, scale, see)
        ref, tol = S.backward(*(to64(t[0, h]) for t in x), scale, see)
        for name, g, r, t in zip(("dq", "dk", "dv"), grads, ref, tol):
            within(to64(g[0, h]), r, t + S.BF * (np.abs(r) + t), (name, h))


def test_one_head_a_group(fa):
    """The widest windows, where a group is one head: some rows, at tiles' and the window's edges."""
    H, T, d, left, sinks, scale = 3, 200000, 64, 195000, 3, 0.125   # 51 MB of K and V a head
    q, k, v, _ = data(1, H, T, T, d, 35)
    o, lse = fa.attention_forward(q, k, v, False, scale, window=(left, 0), sinks=sinks)
    assert fa.fa_sync_status() == fa.FA_OK
    for h in range(H):
        x = [to64(t[0, h]) for t in (q, k, v)]
        for r in (0, 255, 256, 38911, 195003, 195004, 199999):
            see = (np.arange(r + 1) >= r - left) | (np.arange(r + 1) < sinks)
            ro, rl, to, tl, _, _ = S.forward(x[0][r:r + 1], x[1][:r + 1], x[2][:r + 1], scale, see[None])
            within(to64(o[0, h, r]), ro[0], to[0], ("o", h, r))
            within(to64(lse[0, h, r:r + 1]), rl, tl, ("lse", h, r))
