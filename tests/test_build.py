"""The build: what each of the two shared objects needs, and when it is made anew."""
import os

import pytest

from gemv_w4a16_gemm_gb300 import build as libbuild


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """The build of one small source into a folder of its own."""
    monkeypatch.setattr(libbuild, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(libbuild, "LIB", str(tmp_path / "libw4q.so"))
    monkeypatch.setattr(libbuild, "BINDING", str(tmp_path / "_w4q_binding.so"))
    monkeypatch.setattr(libbuild, "SOURCES", ("selftest.cu",))
    return tmp_path


def test_the_library_is_built_without_the_python_module(elsewhere, monkeypatch):
    """libw4q.so needs nvcc alone; torch's headers or g++ may be missing."""
    def missing(force):
        raise RuntimeError("no torch headers")
    monkeypatch.setattr(libbuild, "_compile_binding", missing)
    with pytest.raises(RuntimeError, match="no torch headers"):
        libbuild.build()
    assert os.path.exists(libbuild.LIB)
