"""What the build needs for which of its two results: the library of C entry points
(nvcc alone), and the compiled part of the Python binding (g++, torch, Python's headers)."""
import importlib.util
import os

import pytest

from conftest import ROOT


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module, linking the objects that are there into a folder of the test's."""
    spec = importlib.util.spec_from_file_location("gbf_build", os.path.join(ROOT, "fusion_add_rmsnorm_gb300", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    try:
        mod.nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "libgbfuse.so"))
    monkeypatch.setattr(mod, "BINDING", str(tmp_path / os.path.basename(mod.BINDING)))
    return mod


def fails(*_):
    raise RuntimeError("g++ on decode_binding.cpp failed: no headers")


def test_the_library_is_linked_before_the_binding_fails(build, monkeypatch):
    monkeypatch.setattr(build, "compile_binding", fails)
    with pytest.raises(RuntimeError, match="no headers"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_the_library_alone(build, monkeypatch):
    monkeypatch.setattr(build, "compile_binding", fails)
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert build.build(binding=False) == build.LIB and os.path.exists(build.LIB)


def test_without_torch_the_binding_says_so(build, monkeypatch):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="needs torch"):
        build.build()
    assert os.path.exists(build.LIB)


def test_another_torch_builds_the_binding_anew(build, monkeypatch, tmp_path):
    ran = []

    def run(cmd, what):
        ran.append((what, cmd))
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    (tmp_path / "decode_binding.so").touch()               # an untagged one of an older build
    open(build.LIB, "w").close()
    version = build._torch_version()
    for v, compiles in ((version, True), (version, False), ("9.9.9", True), ("9.9.9", False), (version, True)):
        monkeypatch.setattr(build, "_torch_version", lambda: v)
        ran.clear()
        obj = build.compile_binding(0)
        assert [w for w, _ in ran] == (["g++ on decode_binding.cpp"] if compiles else [])
        assert not compiles or f'-DGBF_BUILT_FOR_TORCH="{v}"' in ran[0][1]
    build.link_binding(obj)
    assert not (tmp_path / "decode_binding.so").exists()
    assert build.BINDING.endswith(build.TAG) and "cpython" in build.TAG
