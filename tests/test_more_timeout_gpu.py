"""The timeout path of the paged decode under a window and of the shared prefix's attention, run on the GPU without a
fault (see test_paged_timeout_gpu.py): one arrive is left out, every wait runs out within its limit, the status says so
and is then clear, and the same call made normally right after is right."""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))
FA_ERR_TIMEOUT = 4


@pytest.fixture(scope="module")
def results():
    from exact_io_aware_05_gb300 import build
    build.build(test_variant=True)
    env = dict(os.environ, FA_WAIT_TIMEOUT_MS="250")
    r = subprocess.run([sys.executable, os.path.join(HERE, "more_timeout_child.py")], env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("name", ["window", "long_window_e4m3", "prefix", "prefix_d256", "prefix_e4m3", "prefix_one_tile"])
def test_tile_never_signalled(results, name):
    res = results[name]
    assert res["launch"] == 0 and res["word"] & 0xFF == FA_ERR_TIMEOUT, res
    assert res["again_launch"] == 0 and res["again_status"] == 0 and res["repeats"], res
    assert res["off"] <= 0.05 and res["off_lse"] <= 1e-3, res
