"""The build on machines that lack what only the 8-bit operators' binding needs."""
import os
import sysconfig

import pytest


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build module with its results in a folder of the test's, and one source file."""
    from top_routing_grouped_gb300 import build as b
    monkeypatch.setattr(b, "OUT", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_fp8.so"))
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "sources", lambda: [os.path.join(b.CSRC, "ep_scan.cu")])
    return b


def test_library_is_built_without_what_the_binding_needs(build, monkeypatch, tmp_path):
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    (tmp_path / "_fp8.so").write_bytes(b"of another library")
    with pytest.warns(UserWarning, match="Python.h is missing"):
        assert build.build(build.OUT) == build.OUT
    assert os.path.exists(build.OUT) and not os.path.exists(build.BINDING)
    assert build.up_to_date(build.OUT)


def test_this_machine_has_what_the_binding_needs_or_says_what_not(build, monkeypatch):
    assert build.binding_lacks() is None
    monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.binding_lacks() == "g++"
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.binding_lacks() == "torch"
    assert not build.up_to_date(build.OUT)


def test_a_binding_that_does_not_compile_is_an_error(build, monkeypatch, tmp_path):
    bad = tmp_path / "binding.cpp"
    bad.write_text("#error no\n")
    monkeypatch.setattr(build, "binding_source", lambda: str(bad))
    with pytest.raises(RuntimeError, match="binding.cpp"):
        build.build(build.OUT)
