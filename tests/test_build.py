"""The build: what each of the two shared objects needs, and when it is made anew."""
import os
import shutil
import subprocess
import sys

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


def test_a_copy_of_the_package_loads_its_own_library(tmp_path):
    """The Python module takes the library beside it, wherever the package lies."""
    libbuild.build()
    copy = tmp_path / os.path.basename(libbuild.PKG)
    shutil.copytree(libbuild.PKG, copy, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__"))
    code = ("from gemv_w4a16_gemm_gb300 import w4q; w4q._native(); "
            "print('\\n'.join({l.split()[-1] for l in open('/proc/self/maps') if 'w4q' in l}))")
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert sorted(r.stdout.split()) == [str(copy / "_w4q_binding.so"), str(copy / "libw4q.so")]


def test_another_torch_makes_the_python_module_anew(elsewhere, monkeypatch):
    runs = []
    def run(cmd):  # a compiler that writes an empty output
        runs.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(libbuild, "_run", run)
    libbuild.build()
    assert len(runs) == 2          # compiled and linked
    libbuild.build()
    assert len(runs) == 2
    monkeypatch.setattr(libbuild, "_torch_id", lambda: "another torch")
    libbuild.build()
    assert len(runs) == 4
    libbuild.build()
    assert len(runs) == 4
