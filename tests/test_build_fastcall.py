"""The binding's C module: built for the interpreter that builds it, and left out where it does not compile."""
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


def test_a_module_that_does_not_compile_is_left_out(build, tmp_path, monkeypatch):
    if build.python_header() is None:
        pytest.skip("no Python.h")
    source, target = tmp_path / "fastcall.c", tmp_path / "_fastcall.so"
    source.write_text("#error not here\n")
    target.write_text("an older one")
    os.utime(target, (0, 0))
    monkeypatch.setattr(build, "FASTCALL_SOURCE", str(source))
    monkeypatch.setattr(build, "FASTCALL", str(target))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="not here"):
        assert build.build_fastcall() is False
    assert not target.exists()


def test_a_module_that_is_up_to_date_is_kept(build, tmp_path, monkeypatch):
    if build.python_header() is None:
        pytest.skip("no Python.h")
    source, target = tmp_path / "fastcall.c", tmp_path / "_fastcall.so"
    source.write_text("int fp8gb_nothing;\n")
    for name, path in (("FASTCALL_SOURCE", source), ("FASTCALL", target), ("PKG", tmp_path)):
        monkeypatch.setattr(build, name, str(path))
    assert build.build_fastcall() and target.exists()
    before = target.stat().st_mtime_ns
    assert build.build_fastcall() and target.stat().st_mtime_ns == before
    os.utime(target, (0, 0))
    assert build.build_fastcall() and target.stat().st_mtime_ns > 0
