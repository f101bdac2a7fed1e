"""The compiled calls are optional: a torch for which they do not compile, do not link or do not load leaves a whole
library and the calls through ctypes.  No GPU; nvcc only for one empty source."""
import importlib.metadata
import os
import sysconfig

import pytest

import swiglu_mlp_group_gb300 as ck
from swiglu_mlp_group_gb300 import _build


@pytest.fixture
def folder(monkeypatch, tmp_path):
    """A build of one empty source, in a folder of its own."""
    if _build._calls_dirs() is None:
        pytest.skip("torch's, Python's or CUDA's headers are not there")
    empty = tmp_path / "empty.cu"
    empty.write_text("extern \"C\" int empty() { return 0; }\n")
    monkeypatch.setattr(_build, "BUILD_DIR", str(tmp_path))
    monkeypatch.setattr(_build, "LIB_PATH", str(tmp_path / _build.LIB_NAME))
    monkeypatch.setattr(_build, "sources", lambda: [str(empty)])
    return tmp_path


@pytest.fixture
def unloaded(monkeypatch):
    monkeypatch.setattr(ck, "_quick_module", False)
    monkeypatch.setattr(ck, "lib", lambda: None)


def test_named_after_torch_and_python():
    name = os.path.basename(_build.calls_path())
    assert importlib.metadata.version("torch") in name and name.endswith(sysconfig.get_config_var("EXT_SUFFIX"))


def test_a_source_that_does_not_compile(folder, unloaded, monkeypatch):
    bad = folder / "torch_calls.cpp"
    bad.write_text("#error no such torch\n")
    monkeypatch.setattr(_build, "CALLS_SOURCE", str(bad))
    with open(_build.calls_path(), "w") as f:
        f.write("of an older library")
    with pytest.warns(RuntimeWarning, match="no such torch"):
        assert _build.build(force=True) == _build.LIB_PATH
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.calls_path())
    assert _build.up_to_date()
    assert ck._quick() is None
    # put right, it is built again
    bad.write_text("int calls() { return 0; }\n")
    os.utime(bad, (os.path.getmtime(_build.LIB_PATH) + 5,) * 2)
    assert not _build.up_to_date()
    _build.build()
    os.utime(_build.LIB_PATH, (os.path.getmtime(bad) + 5,) * 2)
    os.utime(_build.calls_path(), (os.path.getmtime(bad) + 5,) * 2)
    assert _build.up_to_date() and not os.path.exists(_build._calls_failed())


def test_libraries_that_do_not_link(folder, unloaded, monkeypatch):
    good = folder / "torch_calls.cpp"
    good.write_text("int calls() { return 0; }\n")
    monkeypatch.setattr(_build, "CALLS_SOURCE", str(good))
    torch_dir, python_inc, cuda_inc = _build._calls_dirs()
    monkeypatch.setattr(_build, "_calls_dirs", lambda: (str(folder / "no_torch"), python_inc, cuda_inc))
    with pytest.warns(RuntimeWarning, match="link failed"):
        _build.build(force=True)
    assert os.path.exists(_build.LIB_PATH) and not os.path.exists(_build.calls_path()) and _build.up_to_date()
    assert ck._quick() is None


def test_a_file_that_does_not_load(folder, unloaded):
    with open(_build.calls_path(), "w") as f:
        f.write("of another machine")
    with pytest.warns(RuntimeWarning, match="do not load"):
        assert ck._quick() is None
    assert ck._quick() is None  # and is not tried again
