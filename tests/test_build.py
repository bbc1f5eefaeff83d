"""The build of the library and of the module beside it, on stand-ins for the compilers."""

import os
import subprocess
import sysconfig

import pytest
import torch

import memory_bandwidth_amd as q4
from memory_bandwidth_amd import build


@pytest.fixture
def places(tmp_path, monkeypatch):
    """A build into tmp_path whose compiles and link only write their output file."""
    monkeypatch.setattr(build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libq4gemv.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / os.path.basename(build.BIND)))
    failing = set()

    def run(cmd, **kw):
        if cmd[0] in failing:
            return subprocess.CompletedProcess(cmd, 1, "", "no header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    return failing


def test_builds_both(places):
    assert build.build() == build.LIB
    assert open(build.LIB).read() == "new" and open(build.BIND).read() == "new"
    assert sorted(os.listdir(os.path.dirname(build.LIB))) == sorted(
        ["_build", os.path.basename(build.BIND), os.path.basename(build.LIB)])


def test_a_module_that_does_not_build_leaves_the_library(places):
    """The library is there, an older module is not, and the failure is told."""
    with open(build.BIND, "w") as f:
        f.write("old")
    places.add("g++")
    with pytest.raises(RuntimeError, match="bind_i8.cpp"):
        build.build()
    assert open(build.LIB).read() == "new" and not os.path.exists(build.BIND)


def test_no_host_compiler_leaves_the_library(places, monkeypatch):
    stand_in = build.subprocess.run

    def run(cmd, **kw):
        if cmd[0] == "g++":
            raise FileNotFoundError("g++")
        return stand_in(cmd, **kw)

    monkeypatch.setattr(build.subprocess, "run", run)
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build.build()
    assert open(build.LIB).read() == "new"


def test_a_library_that_does_not_build_leaves_both_as_they_were(places):
    for path in (build.LIB, build.BIND):
        with open(path, "w") as f:
            f.write("old")
    places.add(build.hipcc())
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build.build()
    assert open(build.LIB).read() == "old" and open(build.BIND).read() == "old"


def test_the_module_is_for_one_python_and_one_torch(monkeypatch):
    """Another Python does not find it, and another torch is refused."""
    assert build.BIND.endswith("_bind_i8" + sysconfig.get_config_var("EXT_SUFFIX"))
    if not os.path.exists(q4.LIB_PATH) or not os.path.exists(build.BIND):
        build.build()
    module = q4._load_bind()
    assert module.__file__ == build.BIND and module.torch == torch.__version__
    monkeypatch.setattr(q4, "_bind", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="torch"):
        q4.quant_i8(torch.zeros(1, 16))
