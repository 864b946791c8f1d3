"""The build: the library alone where there is no torch, the binding made again for another torch or
Python, and nothing left running or lying about when a compiler fails."""
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_cache_147_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _tool(path, text):
    path.write_text("#!/bin/sh\n" + text)
    path.chmod(0o755)


@pytest.fixture()
def elsewhere(tmp_path, monkeypatch):
    """Compilers of the test's own, and outputs in a folder of its own."""
    (tmp_path / "bin").mkdir()
    monkeypatch.setenv("PATH", f"{tmp_path / 'bin'}:{os.environ['PATH']}")
    for name, at in (("LIB", "libpkv.so"), ("TORCH_LIB", "_pkv_torch.so"), ("BUILD", "b"),
                     ("TORCH_STAMP", "b/version")):
        monkeypatch.setattr(build, name, str(tmp_path / at))
    return tmp_path


def test_the_library_builds_without_torch(tmp_path):
    # a fresh process in which torch cannot be imported, and a compiler that only makes the file
    _tool(tmp_path / "nvcc", 'while [ "$1" != -o ]; do shift; done; touch "$2"\n')
    code = ("import sys; sys.modules['torch'] = None\n"
            "from paged_kv_cache_147_gb300 import build\n"
            f"build.LIB, build.BUILD = {str(tmp_path / 'libpkv.so')!r}, {str(tmp_path / 'b')!r}\n"
            f"build.TORCH_LIB = {str(tmp_path / '_pkv_torch.so')!r}\n"
            "print(build.build())\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                       env=dict(os.environ, PATH=f"{tmp_path}:{os.environ['PATH']}"))
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip() == str(tmp_path / "libpkv.so") and (tmp_path / "libpkv.so").exists()
    assert not (tmp_path / "_pkv_torch.so").exists()


def test_a_failed_library_build_leaves_no_compiler_and_no_file_behind(elsewhere):
    pid = elsewhere / "pid"
    _tool(elsewhere / "bin" / "nvcc", f"while [ ! -s {pid} ]; do sleep 0.05; done; exit 1\n")
    _tool(elsewhere / "bin" / "g++", 'while [ "$1" != -o ]; do shift; done; touch "$2"\n'
                                     f"echo $$ > {pid}; sleep 30\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.build()
    with pytest.raises(ProcessLookupError):
        os.kill(int(pid.read_text()), 0)
    assert sorted(os.listdir(elsewhere)) == ["b", "bin", "pid"] and not os.listdir(elsewhere / "b")


def test_a_failed_binding_is_said_and_leaves_the_library(elsewhere):
    make = 'while [ "$1" != -o ]; do shift; done; touch "$2"\n'
    _tool(elsewhere / "bin" / "nvcc", make)
    _tool(elsewhere / "bin" / "g++", make + "exit 1\n")
    with pytest.raises(RuntimeError, match="pkv_torch.cpp"):
        build.build()
    assert sorted(os.listdir(elsewhere)) == ["b", "bin", "libpkv.so"]


def test_the_binding_is_made_again_for_another_torch_or_python(elsewhere):
    make = 'while [ "$1" != -o ]; do shift; done; echo "$2" >> {log}; touch "$2"\n'
    log = elsewhere / "log"
    for name in ("nvcc", "g++"):
        _tool(elsewhere / "bin" / name, make.format(log=log))
    build.build()
    first = log.read_text().count("_pkv_torch")
    build.build()
    assert first == 1 and log.read_text().count("_pkv_torch") == 1
    stamp = (elsewhere / "b" / "version").read_text()
    assert torch.__version__ in stamp and sys.implementation.cache_tag in stamp
    for other in (stamp.replace(sys.implementation.cache_tag, "cpython-39"),
                  stamp.replace(torch.__version__, "1.0")):
        (elsewhere / "b" / "version").write_text(other)
        build.build()
    assert log.read_text().count("_pkv_torch") == 3 and log.read_text().count("libpkv.so") == 1
