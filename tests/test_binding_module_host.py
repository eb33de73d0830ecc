"""The CPython module of the binding's checks: its name is the running interpreter's."""
import os
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
