"""What build() makes of a machine without the Python headers or a C compiler, and which built
files it takes for current (CPU only)."""
import os
import sysconfig

import pytest

from shared_prefix_fan_gb300 import binding, build


@pytest.fixture
def module(tmp_path, monkeypatch):
    """A place for the extension module where there is none yet; the library is current, and
    must not be compiled again."""
    build.build()
    path = str(tmp_path / os.path.basename(build.HOST))
    monkeypatch.setattr(build, "HOST", path)

    def compiled(*a):
        raise AssertionError("the library is compiled again")
    monkeypatch.setattr(build, "_compile", compiled)
    return path


@pytest.mark.parametrize("lacks", ["headers", "gcc"])
def test_without_headers_or_compiler_the_library_is_there(module, tmp_path, monkeypatch, lacks):
    if lacks == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    for _ in range(2):
        with pytest.warns(UserWarning, match="not built"):
            assert build.build() == build.LIB
    assert not os.path.exists(module)
    monkeypatch.setattr(binding, "_host", None)
    monkeypatch.setattr(binding, "HOST_PATH", module)
    with pytest.raises(RuntimeError, match="not built"):
        binding.kv_append_q8(None, None, None, None, None)
    assert binding.load().fanout_version()


def test_a_module_of_other_sources_is_not_left(module, tmp_path, monkeypatch):
    for age, left in ((0, False), (None, True)):
        open(module, "w").close()
        if age is not None:
            os.utime(module, (age, age))
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
        build._host_calls([os.path.join(build.CSRC, "host_calls.c")])
        assert os.path.exists(module) == left


def test_a_source_that_does_not_compile_raises(module, tmp_path, monkeypatch):
    (tmp_path / "Python.h").write_text("#error no\n")
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    with pytest.raises(RuntimeError, match="host_calls.c"):
        build.build()


def test_only_the_missing_module_is_built(module):
    assert build.build() == build.LIB and os.path.exists(module)
    made = os.path.getmtime(module)
    build.build()
    assert os.path.getmtime(module) == made


def test_the_module_is_named_after_its_interpreter():
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert "cpython" in suffix
    assert binding.HOST_PATH.endswith("_host_calls" + suffix) and binding.HOST_PATH == build.HOST
