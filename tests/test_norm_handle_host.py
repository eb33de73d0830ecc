"""A HeadNorm's weight whose memory was given back and has come again, at the same address, for another type or layout
(`weight.data = ...`): checked again, as one at another address is.  On the host, with views of one block of memory."""
import pytest
import torch

from test_cache_host import fa  # noqa: F401  (a fixture)


@pytest.fixture(params=["q_weight", "k_weight"])
def handle(fa, request):
    block = torch.ones(256)
    w = torch.nn.Parameter(block[:64])
    return fa.HeadNorm(64, **{request.param: w}), w, block, request.param


def test_another_type(fa, handle):
    n, w, block, name = handle
    assert n._ref and n._c.dtype == fa.FA_F32
    w.data = block.view(torch.bfloat16)[:64]
    assert w.data_ptr() == block.data_ptr()
    assert n._ref and n._c.dtype == fa.FA_BF16 and getattr(n._c, name) == block.data_ptr()
    w.data = block[:64]
    assert n._ref and n._c.dtype == fa.FA_F32
    w.data = block.view(torch.float16)[:64]
    with pytest.raises(TypeError):
        n._ref
    w.data = block[:64]
    assert n._ref


def test_another_layout(fa, handle):
    n, w, block, _ = handle
    for bad in (block[:32], block[:128], block[::2][:64]):
        w.data = bad
        assert w.data_ptr() == block.data_ptr()
        with pytest.raises(ValueError):
            n._ref
    w.data = block[:64]
    assert n._ref


def test_both_of_one_type(fa):
    block = torch.ones(256)
    q, k = torch.nn.Parameter(block[:64]), torch.nn.Parameter(torch.ones(64))
    n = fa.HeadNorm(64, q, k)
    q.data = block.view(torch.bfloat16)[:64]
    with pytest.raises(TypeError):
        n._ref
    k.data = k.data.bfloat16()
    assert n._ref and n._c.dtype == fa.FA_BF16 and n._c.k_weight == k.data_ptr()
