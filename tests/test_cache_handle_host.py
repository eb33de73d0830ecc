"""The handles KVCache and RopeSpec on the host: what the structure that the C calls read holds after
their attributes change.  Tensors are on the CPU and nothing is launched."""
import copy
import ctypes
import pickle

import pytest
import torch

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module")
def fa():
    from exact_io_aware_05_gb300 import build
    build.build()
    from exact_io_aware_05_gb300 import fa as _fa
    return _fa


def tensors(codes=False):
    dt = torch.uint8 if codes else BF16
    t = dict(k=torch.zeros((4, 2, 16, 64), dtype=dt), v=torch.zeros((4, 2, 16, 64), dtype=dt),
             block_table=torch.zeros((3, 2), dtype=I32), lens=torch.zeros(3, dtype=I32), seen=torch.zeros(3, dtype=I32),
             weight=torch.zeros((3, 2, 32)), order=torch.zeros((3, 2, 32), dtype=I32))
    if codes:
        t.update(k_scale=torch.ones(2), v_scale=torch.ones(2))
    return t


def held(cache):
    """Every tensor of the handle is at the address that the structure holds."""
    for n in ("k", "v", "block_table", "lens", "seen", "weight", "order", "k_scale", "v_scale"):
        t = getattr(cache, n)
        if getattr(cache._c, n) != (None if t is None else t.data_ptr()):
            return False
    return True


@pytest.mark.parametrize("codes", [False, True])
def test_an_assigned_tensor_is_the_one_that_is_read(fa, codes):
    cache = fa.KVCache(**tensors(codes))
    assert held(cache)
    ref = cache._ref
    cache.lens = cache.lens + 1
    assert held(cache)
    cache.lens += 1                                     # in place, and assigned again
    assert held(cache) and cache.lens.tolist() == [2, 2, 2]
    for name, t in tensors(codes).items():
        setattr(cache, name, t)
        assert getattr(cache, name) is t and held(cache)
    for name in ("seen", "weight", "order"):
        setattr(cache, name, None)
        assert held(cache)
        setattr(cache, name, tensors()[name])
        assert held(cache)
    assert cache._ref == ref


def test_what_does_not_fit_is_refused_and_changes_nothing(fa):
    cache = fa.KVCache(**tensors())
    before = {n: getattr(cache, n) for n in ("k", "v", "block_table", "lens", "seen", "weight", "order", "k_scale", "v_scale")}
    for name, bad, error in (
            ("lens", torch.zeros(4, dtype=I32), ValueError), ("lens", torch.zeros(3), TypeError),
            ("lens", torch.zeros(3, dtype=torch.int64), TypeError), ("lens", torch.zeros(6, dtype=I32)[::2], ValueError),
            ("lens", None, ValueError), ("k", None, ValueError), ("block_table", None, ValueError),
            ("lens", [1, 2, 3], TypeError),
            ("k", torch.zeros((5, 2, 16, 64), dtype=BF16), ValueError), ("v", torch.zeros((4, 2, 16, 64)), TypeError),
            ("weight", torch.zeros((3, 2, 31)), ValueError), ("order", torch.zeros((3, 2, 32)), TypeError),
            ("block_table", torch.zeros((3, 3), dtype=I32), ValueError), ("k_scale", torch.ones(2), ValueError)):
        with pytest.raises(error):
            setattr(cache, name, bad)
        assert held(cache) and all(getattr(cache, n) is t for n, t in before.items()), name
    codes = fa.KVCache(**tensors(True))
    with pytest.raises(ValueError):
        codes.k_scale = None
    with pytest.raises(ValueError):
        codes.v_scale = torch.ones(3)
    for name in ("B", "Hkv", "d", "page_size", "num_pages", "max_pages", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
        with pytest.raises(AttributeError):
            delattr(cache, name)
    with pytest.raises(AttributeError):
        del cache.lens
    cache.note = "a name of the caller's own"
    assert held(cache)


def test_copies_of_a_spec_have_their_own_table(fa):
    """A copy (deep, or from a pickle) reads its own structure, which lives as long as it does."""
    spec = fa.rope_spec(64, (8, 12, 12), interleaved=True)
    for copied in (copy.deepcopy(spec), copy.copy(spec), pickle.loads(pickle.dumps(spec))):
        assert copied._ref == ctypes.addressof(copied._c)
        assert bytes(copied._c) == bytes(spec._c)
        assert (copied.d, copied.rot, copied.n_axes, copied.interleaved) == (64, 64, 3, True)
    assert copy.deepcopy(spec)._ref != spec._ref


@pytest.mark.parametrize("codes", [False, True])
def test_copies_of_a_cache_are_handles_of_their_own(fa, codes):
    """A shallow copy shares the tensors, not the structure; a deep copy or a pickle has tensors of its own."""
    cache = fa.KVCache(**tensors(codes))
    cache.order = None
    shallow = copy.copy(cache)
    assert held(shallow) and shallow._ref != cache._ref and shallow._ref == ctypes.addressof(shallow._c)
    assert all(getattr(shallow, n) is getattr(cache, n) for n in cache._TENSORS)
    shallow.lens = shallow.lens + 5
    assert held(shallow) and held(cache) and cache.lens.tolist() == [0, 0, 0]
    for own in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert held(own) and own._ref == ctypes.addressof(own._c)
        for n in cache._TENSORS:
            a, b = getattr(own, n), getattr(cache, n)
            assert (a is None) == (b is None) and (a is None or (a.data_ptr() != b.data_ptr() and torch.equal(a, b)))
