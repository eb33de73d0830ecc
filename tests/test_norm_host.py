"""Refusals of the head norms with the rotation on the host, before any CUDA call, and their handle.  The
addresses are made up: the file runs only where there is no GPU."""
import copy
import ctypes
import math
import pickle

import pytest
import torch

from test_cache_host import INVALID, MB, NO_GPU, P, Heads, cache, fa, heads, spec  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")


def norm(fa, **kw):
    f = dict(q_weight=P + 20 * MB, k_weight=P + 21 * MB, d=64, dtype=fa.FA_BF16, eps=1e-6)
    f.update(kw)
    return fa._HeadNorm(**f)


def test_forward_refusals(fa):
    f = fa.lib().fa_norm_rope
    x, y = (Heads * 2)(heads(fa, 0), heads(fa, 1)), (Heads * 2)(heads(fa, 2), heads(fa, 3))

    def call(x=x, y=y, n=2, m=norm(fa), pos=P + 5 * MB, sp=spec(fa), B=2, T=4, dtype=fa.FA_BF16):
        return f(x, y, n, None if m is None else ctypes.byref(m), pos, None if sp is None else sp._ref, B, T, dtype, None)
    assert call() in NO_GPU
    assert call(y=x) in NO_GPU
    assert call(m=norm(fa, q_weight=None, k_weight=None)) in NO_GPU
    assert call(B=0) == 0 and call(T=0) == 0
    assert call(m=None) == INVALID and call(sp=None) == INVALID
    for bad in (dict(d=128), dict(dtype=fa.FA_E4M3), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
                dict(q_weight=P + 8), dict(k_weight=P + 2), dict(q_weight=P + 2 * MB), dict(k_weight=P + 3 * MB + 64)):
        assert call(m=norm(fa, **bad)) == INVALID, bad
    assert call(n=0) == INVALID and call(n=3) == INVALID and call(pos=None) == INVALID and call(dtype=fa.FA_E4M3) == INVALID
    assert call(y=(Heads * 2)(heads(fa, 2), heads(fa, 2))) == INVALID


def test_backward_refusals(fa):
    f = fa.lib().fa_norm_rope_bwd
    g, x, dx = ((Heads * 2)(heads(fa, i), heads(fa, i + 1)) for i in (0, 2, 4))
    need = fa.lib().fa_norm_rope_bwd_workspace_bytes(64)
    assert need > 0 and fa.lib().fa_norm_rope_bwd_workspace_bytes(96) == 0

    def call(g=g, x=x, dx=dx, n=2, m=norm(fa), pos=P + 7 * MB, sp=spec(fa), B=2, T=4, dtype=fa.FA_BF16, qw=P + 8 * MB, kw=P + 9 * MB,
             ws=P + 10 * MB, nb=need):
        return f(g, x, dx, n, ctypes.byref(m), pos, sp._ref, B, T, dtype, qw, kw, ws, nb, None)
    assert call() in NO_GPU
    assert call(dx=g) in NO_GPU
    assert call(qw=None, kw=None, ws=None, nb=0) in NO_GPU
    assert call(T=0, qw=None, kw=None, ws=None) == 0
    assert call(T=0) in NO_GPU                            # the weights' gradients are still to be set
    many = (Heads * 2)(heads(fa, 0, H=2 ** 30), heads(fa, 1, H=2 ** 30 - 1))
    assert call(g=many, x=many, dx=many, T=0) in NO_GPU
    assert call(x=None) == INVALID and call(dx=x) == INVALID
    assert call(ws=None) == INVALID and call(nb=need - 1) == INVALID and call(ws=P + 10 * MB + 128) == INVALID
    assert call(n=1) == INVALID and call(n=1, kw=None) in NO_GPU
    assert call(m=norm(fa, q_weight=None)) == INVALID and call(m=norm(fa, q_weight=None), qw=None) in NO_GPU
    assert call(m=norm(fa, k_weight=None)) == INVALID
    for at in (P, P + 2 * MB, P + 4 * MB, P + 5 * MB, P + 7 * MB, P + 9 * MB, P + 10 * MB, P + 20 * MB, P + 8 * MB + 4):
        assert call(qw=at) == INVALID, at
    assert call(ws=P + 3 * MB) == INVALID
    assert call(m=norm(fa, q_weight=P + 4 * MB)) == INVALID
    assert call(x=(Heads * 2)(heads(fa, 2, H=3), heads(fa, 3))) == INVALID
    assert call(x=(Heads * 2)(heads(fa, 2, stride_t=65), heads(fa, 3))) == INVALID


def test_append_refusals(fa):
    f = fa.lib().fa_cache_append_norm
    k, v, q, o = (heads(fa, i) for i in (10, 11, 12, 13))

    def call(m=norm(fa), sp=spec(fa), pos=P + 14 * MB, q=q, o=o):
        ref = ctypes.byref
        return f(ref(cache(fa)), ref(k), ref(v), None if q is None else ref(q), None if o is None else ref(o), pos,
                 None if sp is None else sp._ref, None if m is None else ref(m), None, 4, None)
    assert call() in NO_GPU and call(m=None) in NO_GPU
    assert call(q=None, o=None) in NO_GPU
    assert call(sp=None, pos=None, q=None, o=None) == INVALID         # a norm goes with a rotation
    assert call(m=None, sp=None, pos=None, q=None, o=None) in NO_GPU
    assert call(m=norm(fa, d=128)) == INVALID and call(m=norm(fa, eps=0.0)) == INVALID
    assert call(m=norm(fa, q_weight=P)) == INVALID                    # inside the cache
    assert call(m=norm(fa, k_weight=P + 13 * MB)) == INVALID          # inside q_out


def test_handle(fa):
    w = torch.ones(64, dtype=torch.bfloat16)
    n = fa.HeadNorm(64, w, None, eps=1e-5)
    assert n._c.q_weight == w.data_ptr() and n._c.k_weight is None and n._c.dtype == fa.FA_BF16 and n._index == -1
    f32 = torch.ones(64)
    with pytest.raises(TypeError):
        n.k_weight = f32                       # both of one type
    n.q_weight = None
    n.k_weight = f32
    assert n._c.dtype == fa.FA_F32 and n._c.k_weight == f32.data_ptr() and n._c.q_weight is None
    for bad in (torch.ones(63), torch.ones(128)[::2], torch.ones((1, 64))):
        with pytest.raises(ValueError):
            n.k_weight = bad
    with pytest.raises(TypeError):
        n.k_weight = torch.ones(64, dtype=torch.float64)
    with pytest.raises(TypeError):
        n.k_weight = 1.0
    assert n.k_weight is f32
    # other memory for a weight that it holds, of another type too
    p = torch.nn.Parameter(torch.ones(64))
    n.k_weight = p
    p.data = torch.full((64,), 2.0)
    assert n._ref == ctypes.addressof(n._c) and n._c.k_weight == p.data_ptr()
    p.data = p.data.bfloat16()
    assert n._ref and n._c.k_weight == p.data_ptr() and n._c.dtype == fa.FA_BF16
    n.q_weight = w
    p.data = p.data.float()
    with pytest.raises(TypeError):
        n._ref                                 # one of them has become fp32
    p.data = torch.ones(32, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        n._ref
    n.k_weight = f32.bfloat16()
    n.q_weight = None
    n.k_weight = f32
    for name in ("eps", "d", "other"):
        with pytest.raises(AttributeError):
            setattr(n, name, 1)
    with pytest.raises(AttributeError):
        del n.q_weight
    for twin in (copy.copy(n), copy.deepcopy(n), pickle.loads(pickle.dumps(n))):
        assert twin._ref == ctypes.addressof(twin._c) != n._ref and twin._c.k_weight == twin.k_weight.data_ptr() and twin.eps == n.eps
    for bad in (0.0, -1.0, math.nan, math.inf, 1e-60):
        with pytest.raises(ValueError):
            fa.HeadNorm(64, eps=bad)
    with pytest.raises(ValueError):
        fa.HeadNorm(96)
