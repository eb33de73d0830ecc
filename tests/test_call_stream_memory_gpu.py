"""What a convenience allocates for a call on another stream is of that stream's memory: a block that was freed on the
current stream may still be in use there."""
import pytest
import torch

from test_sinks_gpu import data, fa  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
B, H, T, d = 2, 3, 640, 128


def results(fa, name, x, o, lse, stream):
    q, k, v, do = x
    if name == "forward":
        return fa.attention_forward(q, k, v, True, 0.1, stream)
    if name == "decode":
        return fa.attention_decode(q[:, :, :2].contiguous(), k, v, False, 0.1, stream=stream)
    if name == "fp8":
        o8, l8, ops = fa.attention_forward_fp8(q, k, v, True, 0.1, stream=stream)
        return o8, l8, *ops.values()
    kw = dict(backward=dict(causal=True), deterministic=dict(causal=True, deterministic=True), window=dict(causal=False, window=(100, 0)),
              sinks=dict(causal=False, window=(100, 0), sinks=4))[name]
    return fa.attention_backward(q, k, v, o, lse, do, scale=0.1, stream=stream, **kw)


@pytest.mark.parametrize("name", ["forward", "decode", "fp8", "backward", "deterministic", "window", "sinks"])
def test_memory_of_the_calls_stream(fa, name):
    x = data(B, H, T, T, d, 61)
    o, lse = fa.attention_forward(*x[:3], True, 0.1)
    want = results(fa, name, x, o, lse, None)
    sizes = [(t.shape, t.dtype) for t in want] + [((fa.fa_bwd_workspace_bytes(B, H, T, T, d),), torch.uint8)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    freed = [torch.empty(s, dtype=t, device=DEV) for s, t in sizes]        # blocks that fit, on the current stream
    places = [(t.data_ptr(), t.data_ptr() + t.nbytes) for t in freed]
    del freed
    got = results(fa, name, x, o, lse, side)
    torch.cuda.current_stream().wait_stream(side)
    for t in got:
        assert not any(a <= t.data_ptr() < b for a, b in places), name
    if name not in ("backward", "window", "sinks"):    # dq of those is a sum in any order
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    else:
        assert all(torch.equal(a, b) for a, b in zip(want[1:], got[1:]))
    assert fa.fa_sync_status() == fa.FA_OK
