"""Left bounds that hide no key (a window as long as the keys, or one that begins among the sinks) give the bits of the call
without one; the narrowest that hides a key does not."""
import pytest
import torch

from test_sinks_gpu import data, fa  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.gpu
SIZES = [(2, 3, 700, 700, 128), (1, 2, 300, 901, 64), (1, 2, 900, 300, 128), (1, 2, 520, 520, 256), (1, 1, 1, 1, 64), (4, 11, 1500, 1500, 64)]


def run(fa, x, deterministic=True, **kw):
    q, k, v, do = x
    kw = {"causal": False, **kw}
    causal = kw.pop("causal")
    o, lse = fa.attention_forward(q, k, v, causal, 0.1, **kw)
    out = [o, lse]
    if q.shape[3] < 256:
        out += fa.attention_backward(q, k, v, o, lse, do, causal, 0.1, deterministic=deterministic, **kw)
    assert fa.fa_sync_status() == fa.FA_OK
    return out


@pytest.mark.parametrize("B,H,Tq,Tk,d", SIZES)
def test_the_same_bits(fa, B, H, Tq, Tk, d):
    x = data(B, H, Tq, Tk, d, 51)
    want = run(fa, x, causal=True)
    for kw in (dict(window=(Tk - 1, 0)), dict(window=(2 ** 31 - 1, 0)), dict(window=(Tk - 1, 0), sinks=4), dict(window=(Tk + 500, 0), sinks=Tk),
               dict(window=(7, 0), sinks=Tk), dict(window=(1, 0), sinks=max(Tk - 2, 1)), dict(window=(0, 0), sinks=2 ** 31 - 1)):
        got = run(fa, x, **kw)
        assert all(torch.equal(a, b) for a, b in zip(want, got)), kw
    for right in (-1, 5):      # other right bounds, and a block mask
        assert all(torch.equal(a, b) for a, b in zip(run(fa, x, window=(-1, right)), run(fa, x, window=(Tk - 1, right)))), right
    mask = (torch.rand((-(-Tq // 128), -(-Tk // 128)), device="cuda") < 0.6).to(torch.uint8)
    assert all(torch.equal(a, b) for a, b in zip(run(fa, x, window=(-1, 0), block_mask=mask), run(fa, x, window=(Tk, 0), block_mask=mask)))
    if Tk > 1:                 # the last row no longer sees the first key
        for kw in (dict(window=(Tk - 2, 0)), dict(window=(0, 0), sinks=Tk - 2)):
            got = run(fa, x, **kw)
            assert not torch.equal(got[1][:, :, -1], want[1][:, :, -1])
