"""Backward of the head norms with the rotation where a CTA runs over several tiles of tokens, with groups of query and key
heads of different sizes, against the 64-bit reference (tests/norm_ref.py): dw is a sum over a CTA's tiles, and its last
tile may be short or empty."""
import numpy as np
import pytest
import torch

import norm_ref as N
from gpu_util import to64
from test_cache_gpu import freqs_of, gen, randn, within
from test_norm_gpu import EPS, fa, w64  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


# B, Hq, Hk, T, d, interleaved, dtype: tiles of 24 tokens (48 at d 64, 12 at 256), 304 CTAs over the head groups
@pytest.mark.parametrize("B,Hq,Hk,T,d,inter,dt", [
    (3, 6, 2, 3500, 128, False, BF16),       # two groups, 438 tiles: three for most CTAs
    (1, 40, 8, 2603, 128, True, BF16),       # groups of 32, 8 and 8 heads, 109 tiles for 101 CTAs
    (1, 32, 8, 4001, 64, False, BF16),       # 84 tiles
    (2, 5, 1, 2047, 256, False, F32),        # 342 tiles, two groups
    (1, 3, 0, 9001, 128, True, F32),         # one group: 376 tiles for 304 CTAs
])
def test_several_tiles(fa, B, Hq, Hk, T, d, inter, dt):
    g = gen(41)
    freqs = freqs_of(d)
    axis = [0] * len(freqs)
    pos = torch.randint(0, 5000, (1, B, T), generator=g, device=DEV).to(I32)
    q, k, gq, gk = (randn(g, B, h, T, d, dtype=dt) for h in (Hq, Hk, Hq, Hk))
    w = [(1.0 + 0.5 * randn(g, d, dtype=F32)) for _ in range(2)]
    spec, norm = fa.RopeSpec(d, freqs, axis, inter), fa.HeadNorm(d, *w, eps=EPS)
    dq, dk, dqw, dkw = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    again = fa.norm_rope_backward(gq, gk, q, k, pos, spec, norm)
    assert fa.fa_sync_status() == fa.FA_OK
    assert all(torch.equal(a, b) for a, b in zip((dq, dk, dqw, dkw), again))
    half = 2.0 ** -8 if dt == BF16 else N.U
    for dy, x, dx, ww, dw in ((gq, q, dq, w[0], dqw), (gk, k, dk, w[1], dkw)):
        ref_w, tol_w, mag = np.zeros(d), np.zeros(d), np.zeros(d)
        for b in range(B):
            p = pos[:, b].cpu().numpy()
            for h in range(x.shape[1]):
                ref, terms, tol, tw, m = N.backward(to64(dy[b, h]), to64(x[b, h]), w64(ww, d), norm._c.eps, p, freqs, axis, inter)
                within(to64(dx[b, h]), ref, tol, half)
                ref_w, tol_w, mag = ref_w + terms.sum(0), tol_w + tw.sum(0), mag + m.sum(0)
        within(to64(dw), ref_w, tol_w + B * x.shape[1] * T * N.U * mag, N.U)
