"""The library builds without torch and without g++: the native marshalling of
the torch binding is an option, and no error of it stops a build."""
import os
import shutil
import subprocess
import sys

import pytest

from tiled_fp32_gemm_gb300 import build

SRC = os.path.join(build.CSRC, "torch_binding.cpp")


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """A build folder of its own with the library already built, so that
    build() has the binding alone to make."""
    for name in ("LIB", "CHECKED_LIB"):
        monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))

    def compiled(src, obj, verbose, defines=()):
        open(obj, "w").close()
        return ""

    monkeypatch.setattr(build, "_compile", compiled)
    real = subprocess.run

    def run(cmd, **kw):
        if "-shared" in cmd and SRC not in cmd:     # the library's link
            open(cmd[cmd.index("-o") + 1], "w").close()
            return subprocess.CompletedProcess(cmd, 0, "", "")
        return real(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path


def built(folder):
    return (folder / "libmtsgemm.so").exists()


def bindings(folder):
    return [f for _, _, files in os.walk(folder) for f in files if "mt_torch_binding" in f]


def old_binding():
    path = build.binding_path()
    os.makedirs(os.path.dirname(path))
    open(path, "w").close()
    os.utime(path, (0, 0))                             # older than its sources


def test_without_torch(monkeypatch, elsewhere):
    monkeypatch.setitem(sys.modules, "torch", None)    # import torch raises ImportError
    build.build()
    assert built(elsewhere) and not bindings(elsewhere)


def test_without_a_host_compiler(monkeypatch, elsewhere):
    which = shutil.which
    monkeypatch.setattr(build.shutil, "which", lambda n: None if n == "g++" else which(n))
    old_binding()
    build.build()
    assert built(elsewhere) and not bindings(elsewhere)


def test_binding_that_does_not_compile_warns_and_leaves_no_old_one(monkeypatch, elsewhere):
    old_binding()
    run = build.subprocess.run

    def failing(cmd, **kw):
        if SRC in cmd:
            return subprocess.CompletedProcess(cmd, 1, "", "error: no such header")
        return run(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", failing)
    with pytest.warns(RuntimeWarning, match="no such header"):
        build.build()
    assert built(elsewhere) and not bindings(elsewhere)
