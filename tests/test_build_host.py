"""Host tests of the build: the C library does not depend on torch or on the binding's extension module."""
import importlib.metadata
import importlib.util
import os
import shutil

import pytest

from structured_sparse_long_gb300 import build as pbuild
from structured_sparse_long_gb300 import paged


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A build folder of its own with the current objects (nothing is compiled again), and no library yet."""
    pbuild.build()
    shutil.copytree(pbuild.BUILD_DIR, tmp_path / "_build")
    monkeypatch.setattr(pbuild, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(pbuild, "LIB_DIR", str(tmp_path / "_lib"))
    monkeypatch.setattr(pbuild, "LIB_PATH", str(tmp_path / "_lib" / "libpi_attn.so"))
    monkeypatch.setattr(pbuild, "NATIVE_PATH", str(tmp_path / "_lib" / os.path.basename(pbuild.NATIVE_PATH)))
    return tmp_path


def test_the_library_is_linked_when_the_binding_does_not_compile(place, monkeypatch, capfd):
    """The library is there and loads; what needs the binding says that it is missing, an older one is not kept, and the
    next build tries again."""
    os.makedirs(pbuild.LIB_DIR)
    with open(pbuild.NATIVE_PATH, "w") as fh:
        fh.write("an older module")
    os.utime(pbuild.NATIVE_PATH, (0, 0))
    with monkeypatch.context() as m:
        m.setattr(pbuild, "_native_command", lambda target: ["g++", "-c", os.path.join(pbuild.CSRC, "not_there.cpp"), "-o", target])
        assert pbuild.build() == pbuild.LIB_PATH
    assert os.path.exists(pbuild.LIB_PATH) and not os.path.exists(pbuild.NATIVE_PATH)
    assert "binding" in capfd.readouterr().err
    monkeypatch.setattr(paged, "_native", None)
    with pytest.raises(RuntimeError, match="native binding not built"):
        paged._load_native()
    pbuild.build()
    assert os.path.exists(pbuild.NATIVE_PATH)


def test_the_library_is_linked_without_torch(place, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert pbuild.build() == pbuild.LIB_PATH
    assert os.path.exists(pbuild.LIB_PATH) and not os.path.exists(pbuild.NATIVE_PATH)


def test_torch_needs_no_package_metadata(place, monkeypatch):
    def version(name):
        raise importlib.metadata.PackageNotFoundError(name)
    monkeypatch.setattr(importlib.metadata, "version", version)
    pbuild.build()
    assert os.path.exists(pbuild.LIB_PATH) and os.path.exists(pbuild.NATIVE_PATH)


def test_a_kernel_that_does_not_compile_is_an_error(place, monkeypatch):
    monkeypatch.setattr(pbuild, "NVCC_FLAGS", pbuild.NVCC_FLAGS + ["--no-such-flag"])
    os.remove(os.path.join(pbuild.BUILD_DIR, "api.o"))
    with pytest.raises(RuntimeError, match="nvcc failed for .*api.cu"):
        pbuild.build()
