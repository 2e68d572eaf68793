"""The build: the CUDA library does not depend on the extension module of fp8.py, and that is built anew for another
torch."""
import importlib.util
import os
import types

import pytest

from dense_fp32_matrix_10_gb300 import build


def test_library_is_linked_without_the_extension(monkeypatch, tmp_path):
    build.build()
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib.so"))
    ext = tmp_path / "ext.so"
    ext.write_text("of another torch")
    os.utime(ext, (0, 0))
    monkeypatch.setattr(build, "TORCH_EXT", str(ext))
    for compiler in ("/bin/false", str(tmp_path / "no such compiler")):
        monkeypatch.setenv("CXX", compiler)
        with pytest.warns(UserWarning, match="not built"):
            assert build.build() == str(tmp_path / "lib.so")
        assert (tmp_path / "lib.so").stat().st_size > 100000
        assert not ext.exists()


def test_extension_is_built_anew_for_another_torch(monkeypatch, tmp_path):
    compiler = tmp_path / "cxx"
    compiler.write_text('#!/bin/sh\necho x >> "%s"\nwhile [ "$1" != -o ]; do shift; done\ntouch "$2"\n'
                        % (tmp_path / "runs"))
    compiler.chmod(0o755)
    monkeypatch.setenv("CXX", str(compiler))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "TORCH_EXT", str(tmp_path / "ext.so"))
    version = tmp_path / "version.py"
    monkeypatch.setattr(importlib.util, "find_spec", lambda name: types.SimpleNamespace(origin=str(tmp_path / "__init__.py")))

    def runs(torch_version):
        version.write_text(f"__version__ = '{torch_version}'\n")
        os.utime(version, (0, 0))   # unpacked from an archive: older than the module
        assert build._torch_extension(False) == str(tmp_path / "ext.so")
        return len((tmp_path / "runs").read_text().split())

    assert runs("2.9.1") == 1
    assert runs("2.9.1") == 1
    assert runs("2.11.0") == 2
