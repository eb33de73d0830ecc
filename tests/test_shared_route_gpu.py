"""Which way a long prefix in e4m3 goes: read by every sequence where there are few of them, and by itself where there are
many; results as in tests/test_shared_gpu.py either way."""
import pytest

from test_shared_gpu import check, fa, shared_cache  # noqa: F401  (fa: a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,n,Hq,Hkv,d,Tq,joined", [
    (49152, 3, 16, 4, 64, 4, False), (98304, 2, 8, 8, 64, 1, False), (98304, 2, 8, 8, 128, 1, False),
    (49152, 16, 16, 4, 64, 4, True), (65536, 6, 8, 8, 128, 1, True),
])
def test_long_prefixes_in_e4m3(fa, P, n, Hq, Hkv, d, Tq, joined):
    cache, pages = shared_cache(fa, 71, P, [7 + i for i in range(n)], Hkv, d, 64, True)
    check(fa, None, cache, pages, P, Hq, Tq, sequences=[0, n - 1], joined=joined)
