"""The CPython module of the binding's checks: its name is the running interpreter's, and without it the
package imports and the calls go through ctypes."""
import os
import subprocess
import sys
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def build():
    from exact_io_aware_05_gb300 import build as b
    b.build()
    return b


def test_the_file_is_this_interpreters(build):
    """Another interpreter does not find it (and makes its own): the C API that it uses is this version's."""
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.basename(build.PY_SO) == "_fa_py" + suffix and os.path.exists(build.PY_SO)
    assert not os.path.exists(os.path.join(build.PKG, "_fa_py.so"))
    from exact_io_aware_05_gb300 import _fa_py
    assert os.path.samefile(_fa_py.__file__, build.PY_SO)


def test_an_untagged_file_of_before_goes(build):
    """A build takes away the name that every interpreter would load."""
    stale = os.path.join(build.PKG, "_fa_py.so")
    with open(stale, "wb") as f:
        f.write(b"of another interpreter")
    build.build()
    assert not os.path.exists(stale)


def test_without_the_module_the_calls_go_through_ctypes(build):
    """In a child process that cannot import it: the package imports, and refusals are those of the checks."""
    code = r"""
import sys
class No:
    def find_spec(self, name, path=None, target=None):
        if name.endswith("._fa_py"):
            raise ImportError("not built for this Python")
sys.meta_path.insert(0, No())
import torch
from exact_io_aware_05_gb300 import fa
assert fa._fa_py is None
q = torch.zeros((2, 4, 1, 64), dtype=torch.bfloat16)
pos = torch.zeros((1, 2, 1), dtype=torch.int32)
spec = fa.rope_spec(64)
cache = fa.alloc_kv_cache(2, 2, 64, 32, 16, weight=True, device="cpu")
o, lse, ws = torch.empty_like(q), torch.zeros((2, 4, 1)), torch.zeros(4096, dtype=torch.uint8)
for call in (lambda: fa.fa_rope(q, o, pos, spec), lambda: fa.fa_rope_bwd(q, o, pos, spec),
             lambda: fa.fa_cache_append(cache, q[:, :2], q[:, :2]), lambda: fa.fa_decode_paged(cache, q, o, lse, 0.1, ws),
             lambda: fa.fa_cache_evict(cache, 4)):
    try:
        call()
    except ValueError as e:
        assert "expected CUDA tensors" in str(e) or "same device" in str(e), e
    else:
        raise AssertionError("CPU tensors were taken")
try:
    fa.fa_rope(q.half(), o, pos, spec)
except TypeError:
    print("fine")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]
