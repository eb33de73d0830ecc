"""Refusals of the rotary positions and of the paged cache on the host, before any CUDA call,
and the rotation's table of phases.  The addresses are made up, and calls that pass every check
go on to the device: the file runs only where there is none."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses: only without a GPU")

vp, i, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
INVALID, UNSUPPORTED = 1, 2
NO_GPU = (2, 3)      # past every check of the arguments, and no device to launch on


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import build
    build.build()
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


P = 1 << 24        # fake aligned addresses, a megabyte apart: never dereferenced on these paths
MB = 1 << 20


class Heads(ctypes.Structure):
    _fields_ = [("data", vp), ("stride_b", ll), ("stride_h", ll), ("stride_t", ll), ("H", i)]


def heads(fa, at, B=2, H=2, T=4, d=64, **kw):
    f = dict(data=P + at * MB, stride_b=H * T * d, stride_h=T * d, stride_t=d, H=H)
    f.update(kw)
    return Heads(**f)


def test_packed_heads_are_the_structure(fa):
    """The binding packs fa_heads by a format string: the same bytes as the structure's."""
    one = Heads(P, 1 << 40, 2, 3, 4)
    assert fa._HEADS.size == ctypes.sizeof(Heads) and fa._HEADS2.size == 2 * ctypes.sizeof(Heads)
    assert fa._HEADS.pack(P, 1 << 40, 2, 3, 4, 0) == bytes(one)
    assert fa._HEADS2.pack(P, 1 << 40, 2, 3, 4, 0, P, 1 << 40, 2, 3, 4, 0) == bytes(one) * 2


def cache(fa, **kw):
    f = dict(k=P, v=P + MB, k_scale=None, v_scale=None, block_table=P + 2 * MB, lens=P + 3 * MB, seen=None,
             weight=P + 4 * MB, order=P + 5 * MB, B=2, Hkv=2, d=64, page_size=16, num_pages=8, max_pages=4, dtype=fa.FA_BF16)
    f.update(kw)
    return fa._KVCache(**f)


def spec(fa, d=64, rot=64, axes=1):
    return fa.RopeSpec(d, [1.0] * (rot // 2), [a % axes for a in range(rot // 2)])


# ---------------------------------------------------------------- frequencies
def test_phases_are_exact(fa):
    """turns = f / 2 pi in units of 2^-64 turns, to one unit (2^-53 f would be 2^11 of them)."""
    two_pi = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62) * 2
    freqs = [1.0, 10000.0 ** (-2 / 128), 1e-4, 12345.678, 2.0 ** 30 + 0.125, -0.75, -3.0, 0.0] * 4
    s = fa.RopeSpec(64, freqs)
    for f, t in zip(freqs, list(s._c.turns)):
        exact = Fraction(f) / two_pi * 2 ** 64
        room = 1 + abs(Fraction(f)) / 2 ** 36      # the two-part product: 2^-100 of f / 2 pi
        off = (t - exact) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= room, (f, float(min(off, 2 ** 64 - off)))


def test_spec_refusals(fa):
    init = fa.lib().fa_rope_spec_init
    s = fa._RopeSpec()
    f = (ctypes.c_double * 128)(*([1.0] * 128))
    ax = (ctypes.c_ubyte * 128)()
    r = ctypes.byref(s)
    assert init(r, 64, 64, 1, f, None, 0) == 0
    assert init(r, 64, 64, 1, f, ax, 0) == 0
    assert init(None, 64, 64, 1, f, ax, 0) == INVALID
    assert init(r, 64, 64, 1, None, ax, 0) == INVALID
    assert init(r, 96, 64, 1, f, ax, 0) == UNSUPPORTED
    for rot in (0, 8, 24, 80, -16):
        assert init(r, 64, rot, 1, f, ax, 0) == INVALID
    for axes in (0, 9):
        assert init(r, 64, 64, axes, f, ax, 0) == INVALID
    assert init(r, 64, 64, 1, f, ax, 2) == INVALID
    ax[31] = 3
    assert init(r, 64, 64, 3, f, ax, 0) == INVALID
    assert init(r, 64, 64, 4, f, ax, 0) == 0
    for bad in (math.nan, math.inf, 2.0 ** 31):
        f[5] = bad
        assert init(r, 64, 64, 4, f, ax, 0) == INVALID
    with pytest.raises(ValueError):
        fa.rope_spec(64, (8, 8, 8))
    with pytest.raises(ValueError):
        fa.RopeSpec(64, [1.0] * 32, [0] * 31)
    with pytest.raises(fa.FAError):
        fa.RopeSpec(64, [1.0] * 40)


# ---------------------------------------------------------------- rotation
def test_rope_refusals(fa):
    f = fa.lib().fa_rope
    x, y = (Heads * 2)(heads(fa, 0), heads(fa, 1)), (Heads * 2)(heads(fa, 2), heads(fa, 3))
    pos, sp = P + 5 * MB, spec(fa)

    def call(x=x, y=y, n=2, pos=pos, sp=sp, B=2, T=4, dtype=fa.FA_BF16, inverse=0):
        return f(x, y, n, pos, sp if isinstance(sp, int) or sp is None else sp._ref, B, T, dtype, inverse, None)

    def with_(arr, at, **kw):
        out = (Heads * 2)(*arr)
        for name, val in kw.items():
            setattr(out[at], name, val)
        return out

    assert call() in NO_GPU
    assert call(n=1) in NO_GPU
    assert call(n=0) == INVALID and call(n=3) == INVALID
    assert call(B=-1) == INVALID and call(T=-1) == INVALID
    assert call(B=0) == 0 and call(T=0) == 0
    assert call(inverse=2) == INVALID
    assert call(dtype=fa.FA_E4M3) == INVALID and call(dtype=7) == INVALID
    assert call(sp=None) == INVALID
    assert call(pos=None) == INVALID and call(pos=pos + 2) == INVALID
    assert call(x=with_(x, 0, data=None)) == INVALID
    assert call(y=with_(y, 1, data=P + 3 * MB + 8)) == INVALID
    assert call(x=with_(x, 0, stride_t=68)) == INVALID       # rows off 16 bytes
    assert call(x=with_(x, 0, stride_h=-256)) == INVALID
    assert call(x=with_(x, 0, H=3)) == INVALID               # another number of heads than y
    assert call(y=with_(y, 0, stride_t=0)) == INVALID        # rows of y on one another
    assert call(y=with_(y, 0, stride_h=64)) == INVALID
    assert call(x=with_(x, 0, stride_t=0)) in NO_GPU         # rows of x may be (a broadcast view)
    assert call(y=with_(y, 0, data=P)) in NO_GPU             # in place
    assert call(y=with_(y, 0, data=P + 16)) == INVALID       # half over its input
    assert call(y=with_(y, 0, data=P + MB)) == INVALID       # over the other input
    assert call(y=with_(y, 1, data=P + 2 * MB)) == INVALID   # over the other output
    assert call(pos=P + 2 * MB) == INVALID                   # positions inside an output
    bad = spec(fa)
    bad._c.axis[3] = 1
    assert call(sp=bad) == INVALID


# ---------------------------------------------------------------- the cache
BAD_CACHES = [
    (dict(B=-1), INVALID), (dict(Hkv=0), INVALID), (dict(num_pages=-1), INVALID), (dict(max_pages=-1), INVALID),
    (dict(dtype=1), INVALID), (dict(dtype=9), INVALID), (dict(d=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(num_pages=1 << 30, Hkv=4), INVALID),
    (dict(max_pages=1 << 28, page_size=16), INVALID), (dict(max_pages=(1 << 22) + 1, page_size=256), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(lens=None), INVALID), (dict(block_table=None), INVALID), (dict(k=P + 64), INVALID), (dict(weight=P + 4 * MB + 4), INVALID), (dict(order=P + 5 * MB + 8), INVALID), (dict(lens=P + 3 * MB + 2), INVALID),
    (dict(k_scale=P + 6 * MB, v_scale=P + 6 * MB), INVALID), (dict(dtype=2), INVALID), (dict(dtype=2, k_scale=P + 6 * MB), INVALID),
]


@pytest.mark.parametrize("kw,want", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(fa, kw, want):
    lib, c = fa.lib(), cache(fa, **kw)
    r = ctypes.byref(c)
    H = max(c.Hkv, 1)
    k, v = heads(fa, 8, H=H), heads(fa, 9, H=H)
    assert lib.fa_cache_append(r, ctypes.byref(k), ctypes.byref(v), None, None, None, None, None, 4, None) == want
    assert lib.fa_decode_paged(r, P + 8 * MB, P + 9 * MB, P + 10 * MB, 2 * H, 1, 1, 0.1, 0, P + 16 * MB, 1 << 30, None) == want
    assert lib.fa_cache_evict(r, 8, 0, 0, c.weight, c.order, P + 9 * MB, P + 10 * MB, None) == want


def test_append_refusals(fa):
    f = fa.lib().fa_cache_append
    sp = spec(fa)

    def call(c=None, k=None, v=None, q=None, qo=None, pos=None, sp=None, new=None, T=4, **kw):
        c = c or cache(fa, **kw)
        ref = lambda x: None if x is None else ctypes.byref(x)   # noqa: E731
        return f(ctypes.byref(c), ref(k or heads(fa, 8)), ref(v or heads(fa, 9)), ref(q), ref(qo), pos,
                 None if sp is None else sp._ref, new, T, None)

    pos, q, qo = P + 10 * MB, heads(fa, 11), heads(fa, 12)
    assert call() in NO_GPU
    assert call(q=q, qo=qo, pos=pos, sp=sp) in NO_GPU
    assert call(q=q, qo=q, pos=pos, sp=sp) in NO_GPU             # q in place
    assert f(None, None, None, None, None, None, None, None, 4, None) == INVALID
    assert call(T=-1) == INVALID and call(T=0) == 0
    assert call(B=0) == 0
    assert call(pos=pos) == INVALID                               # positions without a spec
    assert call(q=q, qo=qo) == INVALID                            # q without a rotation
    assert call(sp=sp) == INVALID                                 # a spec without positions
    assert call(q=q, pos=pos, sp=sp) == INVALID
    assert call(q=q, qo=heads(fa, 12, H=3), pos=pos, sp=sp) == INVALID
    assert call(pos=pos, sp=spec(fa, d=128, rot=64)) == INVALID   # another head width
    assert call(k=heads(fa, 8, H=3)) == INVALID
    assert call(k=heads(fa, 8, data=None)) == INVALID
    assert call(v=heads(fa, 9, stride_t=63)) == INVALID
    assert call(new=P + 7 * MB + 1) == INVALID
    assert call(k=heads(fa, 0)) == INVALID                        # k inside the pages
    assert call(v=heads(fa, 4)) == INVALID                        # v inside the weights
    assert call(c=cache(fa, v=P)) == INVALID                      # K and V on the same pages
    assert call(c=cache(fa, order=P + 4 * MB)) == INVALID
    assert call(q=q, qo=heads(fa, 0), pos=pos, sp=sp) == INVALID
    assert call(q=q, qo=heads(fa, 8), pos=pos, sp=sp) == INVALID  # q_out over k
    assert call(q=q, qo=heads(fa, 12, stride_h=64), pos=pos, sp=sp) == INVALID


def test_decode_paged_refusals(fa):
    lib = fa.lib()
    f, size = lib.fa_decode_paged, lib.fa_decode_paged_workspace_bytes
    assert size(2, 4, 2, 1, 4, 16, 64, 0) > 0
    assert size(2, 4, 2, 1, 4, 16, 64, 1) > size(2, 4, 2, 1, 4, 16, 64, 0)
    for bad in ((-1, 4, 2, 1, 4, 16, 64, 0), (2, 5, 2, 1, 4, 16, 64, 0), (2, 0, 2, 1, 4, 16, 64, 0), (2, 4, 0, 1, 4, 16, 64, 0),
                (2, 4, 2, 0, 4, 16, 64, 0), (2, 4, 2, 17, 4, 16, 64, 0), (2, 4, 2, 1, -1, 16, 64, 0), (2, 4, 2, 1, 4, 16, 96, 0),
                (2, 4, 2, 1, 4, 16, 64, 2), (2, 4, 2, 1, 1 << 28, 16, 64, 0), (1 << 28, 16, 1, 1, 4, 16, 64, 0)):
        assert size(*bad) == 0, bad

    def call(c=None, q=P + 8 * MB, o=P + 9 * MB, lse=P + 10 * MB, Hq=4, Tq=1, causal=1, scale=0.1, acc=0, ws=P + 16 * MB,
             n=64 * MB, **kw):
        c = c or cache(fa, **kw)
        return f(ctypes.byref(c), q, o, lse, Hq, Tq, causal, scale, acc, ws, n, None)

    assert call() in NO_GPU and call(acc=1) in NO_GPU
    assert call(B=0) == 0
    assert call(Tq=17) == UNSUPPORTED
    assert call(Tq=0) == INVALID and call(Hq=3) == INVALID and call(Hq=0) == INVALID
    assert call(causal=2) == INVALID and call(acc=2) == INVALID
    for s in (0.0, -1.0, math.nan, math.inf):
        assert call(scale=s) == INVALID
    assert call(acc=1, weight=None) == INVALID
    for name in ("q", "o", "lse"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: P + 12 * MB + 8}) == INVALID
    assert call(ws=None) == INVALID and call(n=16) == INVALID and call(ws=P + 16 * MB + 128) == INVALID
    assert call(o=P + 8 * MB) == INVALID                         # o over q
    assert call(o=P + 16) == INVALID                             # o inside the pages
    assert call(lse=P + 3 * MB) == INVALID                       # lse over lens
    assert call(ws=P + 4 * MB) == INVALID                        # workspace over the weights
    assert call(lse=P + 16 * MB) == INVALID                      # lse inside the workspace


def test_evict_refusals(fa):
    f = fa.lib().fa_cache_evict

    def call(c=None, budget=8, first=0, recent=0, w=P + 8 * MB, o=P + 9 * MB, n=P + 10 * MB, kept=P + 11 * MB, **kw):
        c = c or cache(fa, **kw)
        return f(ctypes.byref(c), budget, first, recent, w, o, n, kept, None)

    assert call() in NO_GPU
    assert call(w=P + 4 * MB, o=P + 5 * MB, n=P + 3 * MB) in NO_GPU     # in place
    assert call(B=0) == 0
    assert call(budget=0) == INVALID and call(first=-1) == INVALID and call(recent=-1) == INVALID
    assert call(first=5, recent=4) == INVALID and call(first=2 ** 31 - 1, recent=2 ** 31 - 1) == INVALID
    assert call(weight=None) == INVALID
    assert call(order=None) == INVALID                                  # an order_out without an order
    assert call(order=None, o=None) in NO_GPU
    assert call(order=None, o=None, recent=1) == INVALID                # recent needs the order
    assert call(o=None) == INVALID
    for name in ("w", "n", "kept"):
        assert call(**{name: None}) == INVALID
        assert call(**{name: P + 12 * MB + 1}) == INVALID
    assert call(kept=P + 4 * MB) == INVALID                             # kept over the weights
    assert call(w=P + 4 * MB + 4) == INVALID                            # half over its input
    assert call(o=P + 4 * MB) == INVALID
    assert call(n=P + 2 * MB) == INVALID                                # lens_out over the table
    assert call(kept=P) == INVALID


# ---------------------------------------------------------------- the binding
def test_binding_refusals(fa):
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)   # noqa: E731
    i32 = torch.int32
    args = (z(4, 2, 16, 64), z(4, 2, 16, 64), z(2, 3, dt=i32), z(2, dt=i32))
    c = fa.KVCache(*args)
    with pytest.raises(ValueError):
        fa.KVCache(args[0], z(4, 2, 16, 128), *args[2:])
    with pytest.raises(TypeError):
        fa.KVCache(args[0].float(), args[1].float(), *args[2:])
    with pytest.raises(TypeError):
        fa.KVCache(*args[:2], z(2, 3, dt=torch.int64), args[3])
    with pytest.raises(ValueError):
        fa.KVCache(*args, k_scale=z(2, dt=torch.float32), v_scale=z(2, dt=torch.float32))
    with pytest.raises(ValueError):
        fa.KVCache(z(4, 2, 16, 64, dt=torch.uint8), z(4, 2, 16, 64, dt=torch.uint8), *args[2:])
    with pytest.raises(ValueError):
        fa.KVCache(*args, weight=z(2, 2, 47, dt=torch.float32))
    with pytest.raises(ValueError):
        fa.KVCache(args[0].transpose(1, 2).contiguous().transpose(1, 2), *args[1:])
    q = z(2, 4, 1, 64)
    o, lse, ws = torch.empty_like(q), z(2, 4, 1, dt=torch.float32), z(4096, dt=torch.uint8)
    with pytest.raises(ValueError):
        fa.fa_decode_paged(c, q, o, lse, 0.1, ws)              # CPU tensors
    with pytest.raises(ValueError):
        fa.fa_decode_paged(c, z(2, 4, 1, 128), o, lse, 0.1, ws)
    with pytest.raises(TypeError):
        fa.fa_decode_paged(c, q.float(), o, lse, 0.1, ws)
    with pytest.raises(ValueError):
        fa.fa_cache_evict(c, 8)                                 # no weight
    sp = fa.rope_spec(64)
    with pytest.raises(ValueError):
        fa.fa_rope(q, o, z(1, 2, 2, dt=i32), sp)
    with pytest.raises(ValueError):
        fa.fa_rope(z(2, 4, 1, 128), z(2, 4, 1, 128), z(1, 2, 1, dt=i32), sp)
    with pytest.raises(TypeError):
        fa.fa_rope(q.half(), o.half(), z(1, 2, 1, dt=i32), sp)
    with pytest.raises(ValueError):
        fa.fa_rope(z(2, 4, 64, 1).transpose(2, 3), o, z(1, 2, 1, dt=i32), sp)   # rows not contiguous
    with pytest.raises(ValueError):
        fa.fa_rope(q, o, z(1, 2, 1, dt=i32), sp, k=q)           # k without k_out
    with pytest.raises(ValueError):
        fa.fa_cache_append(c, z(2, 2, 1, 64), z(2, 2, 1, 64), q=q, q_out=o)
    with pytest.raises(ValueError):
        fa.fa_cache_append(c, z(2, 2, 1, 64), z(2, 2, 1, 64), spec=sp)
    with pytest.raises(ValueError):
        fa.fa_cache_append(c, z(2, 2, 1, 64), z(2, 2, 2, 64))
