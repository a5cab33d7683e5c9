"""What is built when: the C library by nvcc alone, the binding where its tools are, each when it is out of date."""

import os
import sys
import sysconfig

import pytest

from speculative_decoding_draft_stream_gb300 import build as b


@pytest.fixture
def steps(monkeypatch, tmp_path):
    """build() in an empty folder, its commands written down; a command only makes its output."""
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB_PATH", str(tmp_path / b.LIB_NAME))
    monkeypatch.setattr(b, "BINDING_PATH", str(tmp_path / "_serving.so"))
    ran = []

    def run(cmd, what, verbose):
        ran.append((os.path.basename(cmd[0]), os.path.basename(cmd[cmd.index("-o") + 1])))
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(b, "_run", run)
    return ran


LIBRARY = {("nvcc", os.path.splitext(s)[0] + ".o") for s in b.SOURCES} | {("nvcc", b.LIB_NAME + ".tmp")}
BINDING = {("g++", "ns_binding.o"), ("g++", "_serving.so.tmp")}


def test_everything_once(steps):
    assert not b.up_to_date()
    assert b.build() == b.LIB_PATH and set(steps) == LIBRARY | BINDING
    assert os.path.exists(b.LIB_PATH) and os.path.exists(b.BINDING_PATH) and b.up_to_date()
    steps.clear()
    b.build()
    assert steps == []
    b.build(force=True)
    assert set(steps) == LIBRARY | BINDING


@pytest.mark.parametrize("without", ["torch", "g++", "Python.h"])
def test_the_library_needs_nvcc_alone(steps, monkeypatch, tmp_path, capsys, without):
    open(b.BINDING_PATH, "w").close()  # one of other tools
    if without == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)  # import torch fails
    elif without == "g++":
        which = b.shutil.which
        monkeypatch.setattr(b.shutil, "which", lambda x: None if x == "g++" else which(x))
    else:
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(b.sysconfig, "get_paths", lambda: paths)
    assert b.build() == b.LIB_PATH and set(steps) == LIBRARY
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)
    assert f"no {without}" in capsys.readouterr().err
    assert b.library_up_to_date() and not b.up_to_date()
    steps.clear()
    b.build()
    assert steps == []


def test_a_binding_that_fails_leaves_the_library(steps, monkeypatch):
    run = b._run

    def fail(cmd, what, verbose):
        if "g++" in cmd[0]:
            raise RuntimeError(what)
        run(cmd, what, verbose)

    monkeypatch.setattr(b, "_run", fail)
    with pytest.raises(RuntimeError, match="ns_binding.cpp"):
        b.build()
    assert set(steps) == LIBRARY and b.library_up_to_date() and not os.path.exists(b.BINDING_PATH)


def test_another_torch_or_python_rebuilds_the_binding(steps, monkeypatch):
    import torch

    b.build()
    for obj, name in ((torch, "__version__"), (sys, "version")):
        steps.clear()
        with monkeypatch.context() as m:
            m.setattr(obj, name, getattr(obj, name) + ".other")
            assert b.library_up_to_date() and not b.up_to_date()
            b.build()
            assert set(steps) == BINDING and b.up_to_date()
        assert not b.up_to_date()
        b.build()


def test_each_follows_its_own_sources(steps, monkeypatch, tmp_path):
    b.build()
    later = os.path.getmtime(b.LIB_PATH) + 100

    def newer(match):
        real = os.path.getmtime
        return lambda f: later if f.endswith(match) else real(f)

    for match, rebuilt in (("ns_pages.cu", LIBRARY), ("ns_ptx.cuh", LIBRARY), (b.BINDING, BINDING),
                           ("nanospec_ops.h", LIBRARY | BINDING)):
        steps.clear()
        with monkeypatch.context() as m:
            m.setattr(b.os.path, "getmtime", newer(match))
            b.build()
        assert set(steps) == rebuilt
