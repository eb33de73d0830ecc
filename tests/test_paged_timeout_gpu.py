"""The paged decode's timeout path, run on the GPU without a fault: a test-only build of the library
leaves out one mbarrier arrive of one launch, with a 250 ms limit (see test_timeout_gpu.py).

The math warps wait for a tile whose phase never completes, raise the abort flag and record the wait;
the loader, which may have issued its last copy before, waits until its copies have landed.  The call
returns, the status names one of the two waits and is then clear, and the same call made normally right
after, on the same memory, is right.
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
FA_ERR_TIMEOUT = 4
FULL, EMPTY = 1, 2      # wait sites of the kernel


@pytest.fixture(scope="module")
def results():
    from exact_io_aware_05_gb300 import build
    build.build(test_variant=True)
    env = dict(os.environ, FA_WAIT_TIMEOUT_MS="250")
    r = subprocess.run([sys.executable, os.path.join(HERE, "paged_timeout_child.py")], env=env, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


# in a unit that fits the ring the loader waits for no stage
@pytest.mark.parametrize("name,sites", [("fits_the_ring", {FULL}), ("last_tiles", {FULL}),
                                        ("longer_than_the_ring", {FULL, EMPTY}), ("in_shares_e4m3", {FULL, EMPTY})])
def test_tile_never_signalled(results, name, sites):
    res = results[name]
    assert res["launch"] == 0 and res["word"] & 0xFF == FA_ERR_TIMEOUT and (res["word"] >> 8) in sites, res
    assert res["again_launch"] == 0 and res["again_status"] == 0
    assert res["again_excess"] <= 0


def test_timeout_beside_a_bad_length(results):
    """A length out of range is reported first, and its sequence alone is left out; the timeout, after which
    no output of the call is valid, is what the caller has to hear of."""
    res = results["beside_a_bad_length"]
    assert res["launch"] == 0 and res["status"] == FA_ERR_TIMEOUT
    assert res["again_launch"] == 0 and res["again_status"] == 0
    assert res["again_excess"] <= 0


def test_status_words_are_read_once_they_are_in_use(results):
    """fa_sync_status reads the words of the cache kernels only after one of them was launched."""
    assert results["reads_before_any_cache_call"] == 0
    assert results["reads_after_decodes"] == 1      # the paged decode's, not append's and evict's
