"""The binding's C module: built for the interpreter that builds it."""
import os
import sysconfig

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture()
def build():
    import __graft_entry__
    return __graft_entry__._build_module()


def test_the_module_carries_the_interpreter_in_its_name(build):
    if build.python_header() is None:
        pytest.skip("no Python.h")
    try:
        build.build()
    except RuntimeError as e:
        pytest.skip(f"no CUDA toolkit to build with: {e}")
    import fp8_mixed_precision_saturating_gb300 as g
    name = "_fastcall" + sysconfig.get_config_var("EXT_SUFFIX")
    assert "cpython" in name and os.path.basename(g._fastcall.__file__) == name
    assert not os.path.exists(os.path.join(build.PKG, "_fastcall.so"))
