"""CPU checks of the build: the C library does not depend on the torch binding."""

import importlib
import os
import shutil

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module with one small source and its outputs in a folder of the test's own."""
    b = importlib.import_module("mxfp4_expert_layer_gb300.build")
    if not os.path.exists(b.nvcc_path()) and not shutil.which(b.nvcc_path()):
        pytest.skip("no nvcc")
    for name, value in (("SOURCES", ["moe_peak.cu"]), ("BUILD_DIR", str(tmp_path / "_build")),
                        ("LIB_PATH", str(tmp_path / b.LIB_NAME)), ("EXT_PATH", str(tmp_path / "_dense_ext.so"))):
        monkeypatch.setattr(b, name, value)
    return b


def torch_folder(tmp_path, cuda):
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    if cuda:
        (tmp_path / "torch" / "lib" / "libtorch_cuda.so").touch()
    return str(tmp_path / "torch")


def test_a_torch_without_cuda_gets_the_library_alone(build, tmp_path, monkeypatch):
    folder = torch_folder(tmp_path, False)
    monkeypatch.setattr(build, "_torch_dir", lambda: folder)
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.EXT_PATH)
    assert not build.is_stale()


def test_a_binding_that_fails_leaves_the_library(build, tmp_path, monkeypatch):
    folder = torch_folder(tmp_path, True)  # (without headers)
    monkeypatch.setattr(build, "_torch_dir", lambda: folder)
    with pytest.raises(RuntimeError, match="dense_binding"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.EXT_PATH)
    assert build.is_stale()


def test_a_binding_of_another_torch_or_python_is_built_anew(build, tmp_path, monkeypatch):
    folder = torch_folder(tmp_path, True)
    version = tmp_path / "torch" / "version.py"
    version.write_text("__version__ = '1'\n")
    monkeypatch.setattr(build, "_torch_dir", lambda: folder)
    built = []

    def link(obj):
        built.append(obj)
        (tmp_path / "_dense_ext.so").touch()
    monkeypatch.setattr(build, "_compile_ext", lambda: "binding.o")
    monkeypatch.setattr(build, "_link_ext", link)
    build.build()
    assert len(built) == 1 and not build.is_stale()
    build.build()
    assert len(built) == 1
    version.write_text("__version__ = '2'\n")
    assert build.is_stale()
    build.build()
    assert len(built) == 2 and not build.is_stale()
    monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    assert build.is_stale()
