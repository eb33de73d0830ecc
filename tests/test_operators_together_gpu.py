"""The operators as a model's layer calls them, one after the other: a training step (norms and rotation, attention under
a window with sinks, their gradients) and steps of a decoding batch (norms on the way into the paged cache, a
layer with a window and one over the shared prefix).  Each stage is held against the 64-bit reference of its own
formulas, with what the stage before it gave as the input, at the tolerances of norm_ref, sinks_ref, paged_ref and
test_shared_gpu."""
import numpy as np
import pytest
import torch

import norm_ref as N
import paged_ref as R
import sinks_ref as S
from gpu_util import to64
from test_cache_gpu import entries, freqs_of, gen, randn, within
from test_shared_gpu import shared_cache
from test_window_gpu import attend

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-5


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def step(fa, x, k, v, do, pos, spec, norm, scale, left, sinks):
    """Forward and backward of one layer's attention, by the package's allocating calls."""
    qn, kn = fa.norm_rope_forward(x, k, pos, spec, norm)
    o, lse = fa.attention_forward(qn, kn, v, False, scale, window=(left, 0), sinks=sinks)
    dqn, dkn, dv = fa.attention_backward(qn, kn, v, o, lse, do, False, scale, window=(left, 0), sinks=sinks, deterministic=True)
    dq, dk, dwq, dwk = fa.norm_rope_backward(dqn, dkn, x, k, pos, spec, norm)
    return qn, kn, o, lse, dqn, dkn, dv, dq, dk, dwq, dwk


@pytest.mark.parametrize("d,T,left,sinks", [(64, 300, 50, 4), (128, 700, 200, 3), (128, 129, 0, 1)])
def test_training_step(fa, d, T, left, sinks):
    B, H, scale = 2, 3, d ** -0.5
    g = gen(d + T)
    qkv = randn(g, B, T, 3 * H, d).transpose(1, 2)               # a packed projection
    q, k, v = qkv[:, :H], qkv[:, H:2 * H], qkv[:, 2 * H:].contiguous()
    do = randn(g, B, H, T, d)
    w = [(1.0 + 0.5 * randn(g, d, dtype=F32)) for _ in range(2)]
    freqs, pos = freqs_of(d), torch.arange(T, dtype=I32, device=DEV).expand(1, B, T).contiguous()
    spec, norm = fa.RopeSpec(d, freqs, [0] * (d // 2)), fa.HeadNorm(d, *w, eps=EPS)
    args = (q, k, v, do, pos, spec, norm, scale, left, sinks)
    out = step(fa, *args)
    assert fa.fa_sync_status() == fa.FA_OK
    # captured and replayed with other inputs, and back: the same bits as the eager calls
    graph = torch.cuda.CUDAGraph()
    keep = [t.clone() for t in (q, v, do)]
    with torch.cuda.graph(graph):
        again = step(fa, *args)
    for t in (q, v, do):
        t.copy_(randn(g, *t.shape))
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(step(fa, *args), again))
    for t, s in zip((q, v, do), keep):
        t.copy_(s)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, again))
    assert fa.fa_sync_status() == fa.FA_OK

    qn, kn, o, lse, dqn, dkn, dv, dq, dk, dwq, dwk = out
    see, half = S.visible(T, T, left, sinks), 2.0 ** -8
    sums = {0: [0.0, 0.0, 0.0], 1: [0.0, 0.0, 0.0]}
    for b in range(B):
        at = pos[:, b].cpu().numpy()
        for h in range(H):
            for which, (x, n, dn, dx) in enumerate(((q, qn, dqn, dq), (k, kn, dkn, dk))):
                y, tol = N.forward(to64(x[b, h]), to64(w[which]), norm._c.eps, at, freqs, [0] * (d // 2), False)
                within(to64(n[b, h]), y, tol, half)
                ref, terms, tol, tt, mag = N.backward(to64(dn[b, h]), to64(x[b, h]), to64(w[which]), norm._c.eps, at, freqs, [0] * (d // 2), False)
                within(to64(dx[b, h]), ref, tol, half)
                for i, a in enumerate((terms, tt, mag)):
                    sums[which][i] = sums[which][i] + a.sum(0)
            x = [to64(t[b, h]) for t in (qn, kn, v, do)]
            ro, rl, to, tl, _, _ = S.forward(*x[:3], scale, see)
            within(to64(o[b, h]), ro, to)
            within(to64(lse[b, h]), rl, tl)
            for got, ref, t in zip((dqn, dkn, dv), *S.backward(*x, scale, see)):
                within(to64(got[b, h]), ref, t + S.BF * (np.abs(ref) + t))
    for which, got in enumerate((dwq, dwk)):
        total, tol, mag = sums[which]
        within(to64(got), total, tol + B * H * T * N.U * mag, N.U)


@pytest.mark.parametrize("codes", [False, True])
def test_decoding_steps(fa, codes):
    """A captured step, replayed: lengths grow by one, the token goes normed and turned into the cache, one layer reads a
    window with sinks, one the whole cache over its shared prefix; both share a workspace.  The batch crosses page
    ends, and one sequence stops taking tokens."""
    d, ps, Hq, Hkv, P, steps = 128, 16, 12, 2, 208, 5
    scale, left, sinks = d ** -0.5, 40, 5
    tails, g = [13, 1, 60, 30], gen(9)
    cache, pages = shared_cache(fa, 8, P, [x + steps for x in tails], Hkv, d, ps, codes)    # pages for the steps
    cache.lens.sub_(steps)
    B = cache.B
    w = [1.0 + 0.5 * randn(g, d) for _ in range(2)]
    freqs = freqs_of(d)
    spec, norm = fa.RopeSpec(d, freqs, [0] * (d // 2)), fa.HeadNorm(d, *w, eps=EPS)
    qkv = torch.empty((B, 1, Hq + 2 * Hkv, d), dtype=BF16, device=DEV).transpose(1, 2)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    new = torch.ones(B, dtype=I32, device=DEV)
    pos = torch.empty((1, B, 1), dtype=I32, device=DEV)
    qn = torch.zeros((B, Hq, 1, d), dtype=BF16, device=DEV)
    outs = [(torch.empty_like(qn), torch.empty((B, Hq, 1), device=DEV)) for _ in range(2)]
    ws = torch.empty(max(fa.fa_decode_paged_window_workspace_bytes(cache, Hq, 1),
                         fa.fa_decode_paged_shared_workspace_bytes(cache, Hq, 1, pages)), dtype=torch.uint8, device=DEV)

    def decode():
        pos[0, :, 0] = cache.lens
        cache.lens.add_(new)
        fa.fa_cache_append(cache, k, v, pos, spec, q, qn, new, norm=norm)
        fa.fa_decode_paged_window(cache, qn, *outs[0], left, sinks, scale, ws)
        fa.fa_decode_paged_shared(cache, qn, *outs[1], pages, scale, ws)

    start = [t.clone() for t in (cache.k, cache.v, cache.lens)]
    qkv.copy_(randn(g, *qkv.shape))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        decode()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        decode()
    for t, s in zip((cache.k, cache.v, cache.lens), start):
        t.copy_(s)
    vals = R.e4m3_values()
    for i in range(steps):
        qkv.copy_(randn(g, *qkv.shape) * (1 + i))
        new[1] = int(i < 2)                                       # the second sequence ends after two tokens
        graph.replay()
        assert fa.fa_sync_status() == fa.FA_OK
        for b in range(B):
            n = int(cache.lens[b])
            grown = [x + 1 + i for x in tails]
            assert n == P + (grown[b] if b != 1 else tails[1] + min(i + 1, 2))
            qq, (ke, ve) = to64(qn[b]), entries(cache, b)
            if int(new[b]):
                y, tol = N.forward(to64(q[b]), to64(w[0]), norm._c.eps, np.array([[n - 1]]), freqs, [0] * (d // 2), False)
                within(qq, y, tol, 2.0 ** -8)
                y, tol = N.forward(to64(k[b]), to64(w[1]), norm._c.eps, np.array([[n - 1]]), freqs, [0] * (d // 2), False)
                for h in range(Hkv):
                    if codes:
                        for at, x, t, s in ((ke, y[h, 0], tol[h, 0], cache.k_scale), (ve, to64(v[b, h, 0]), 0.0, cache.v_scale)):
                            s = float(s[h])
                            within(at[h, -1], np.clip(x, vals[0x7E] * -s, vals[0x7E] * s), t + 2.0 ** -10 * s, 2.0 ** -4)
                    else:
                        within(ke[h, -1], y[h, 0], tol[h, 0], 2.0 ** -8)
                        assert np.array_equal(ve[h, -1], to64(v[b, h, 0]))
            G = Hq // Hkv
            ro, rl, to, tl = attend(qq, ke, ve, scale, G, codes, left, sinks)
            within(to64(outs[0][0][b]), ro, to, 2.0 ** -8)
            within(to64(outs[0][1][b]), rl, tl)
            ro, rl, _, to, tl, _ = R.attend(qq, ke, ve, scale, True, G, codes)
            for h in range(Hq):   # the prefix's probabilities in bf16
                p = np.exp(scale * (ke[h // G, :P] @ qq[h, 0]) - rl[h, 0])
                to[h, 0] += 2.0 ** -8 * (p @ np.abs(ve[h // G, :P]))
            within(to64(outs[1][0][b]), ro, to, 2.0 ** -8)
            within(to64(outs[1][1][b]), rl, tl)
