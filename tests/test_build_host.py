"""libda.so is built where the serving calls' binding cannot be: its users and
those of the other operators need neither Python's headers nor torch's."""
import ctypes
import os
import sysconfig
import types

import pytest

import deformable_view_feature_gb300 as da
from deformable_view_feature_gb300 import build

SOURCE = 'extern "C" int answer() { return 42; }\n'


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one small source into a folder of its own."""
    csrc, out = tmp_path / "csrc", tmp_path / "out"
    csrc.mkdir()
    (csrc / "a.cu").write_text(SOURCE)
    for name, value in dict(CSRC=str(csrc), OUT_DIR=str(out), LIB=str(out / "libda.so"), DEBUG_DIR=str(out / "debug"),
                            DEBUG_LIB=str(out / "debug" / "libda_debug.so"), BINDING_SRC=str(csrc / "binding.cpp"),
                            BINDING=str(out / os.path.basename(build.BINDING))).items():
        monkeypatch.setattr(build, name, value)
    (csrc / "binding.cpp").write_text('#include <there/is/no/such/header.h>\n')
    return tmp_path


def test_a_binding_that_does_not_compile_leaves_the_library(small):
    with pytest.warns(UserWarning, match="no/such/header"):
        lib = build.build()
    assert ctypes.CDLL(lib).answer() == 42 and not os.path.exists(build.BINDING)
    with pytest.warns(UserWarning, match="binding.cpp"):  # the library is up to date, the binding is tried again
        assert build.build() == lib


def test_no_host_compiler(small, monkeypatch):
    monkeypatch.setenv("CXX", str(small / "no-such-compiler"))
    with pytest.warns(UserWarning, match="binding.cpp"):
        lib = build.build()
    assert ctypes.CDLL(lib).answer() == 42


def test_serving_calls_raise_without_the_binding(small, monkeypatch):
    monkeypatch.setattr(da, "_binding_module", None)
    monkeypatch.setattr(da, "load_library", lambda: types.SimpleNamespace(_handle=0))
    with pytest.raises(RuntimeError, match="not built"):
        da.qkr_forward(None)


def test_a_binding_of_older_sources_does_not_stay(small):
    out = small / "out"
    out.mkdir()
    (out / os.path.basename(build.BINDING)).write_text("of older sources")
    os.utime(build.BINDING, (1, 1))
    with pytest.warns(UserWarning, match="binding.cpp"):
        build.build()
    assert not os.path.exists(build.BINDING)


def test_a_library_that_does_not_compile_is_an_error(small):
    (small / "csrc" / "a.cu").write_text("no such type;\n")
    with pytest.warns(UserWarning, match="binding.cpp"), pytest.raises(RuntimeError, match="nvcc failed on a.cu"):
        build.build()


def test_the_bindings_name_says_for_which_python_it_is():
    assert build.BINDING.endswith(sysconfig.get_config_var("EXT_SUFFIX")) and "_binding-" in build.BINDING
