"""What the build makes, of what, and when it makes it again.  A shell script
stands in for nvcc: it writes the file that it is asked for."""
import importlib.metadata
import importlib.util
import os
import stat
import sys
import sysconfig

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py as a module of its own, with outputs in a folder of the test's."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "gradient_sync_rcc_gb300", "build.py")
    spec = importlib.util.spec_from_file_location("build_under_test", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\necho "$@" >> %s\nwhile [ "$1" != -o ]; do shift; done\n: > "$2"\n'
                    % (tmp_path / "calls"))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    m.NVCC = str(nvcc)
    m.OBJDIR = str(tmp_path / "_build")
    m.LIB = str(tmp_path / "librcc.so")
    m.BINDING = str(tmp_path / "_lm.so")

    def run():
        calls = tmp_path / "calls"
        if calls.exists():
            calls.unlink()
        assert m.build(lib=m.LIB, objdir=m.OBJDIR) == m.LIB
        return len(calls.read_text().splitlines()) if calls.exists() else 0
    m.run = run
    m.compiles_binding = lambda works: setattr(m, "binding_command", lambda out: [
        sys.executable, "-c", "import sys; open(sys.argv[1], 'w') if %r else sys.exit('no header')"
        % works, out])
    return m


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))


def test_without_torch_the_library_is_built(build, monkeypatch):
    without_torch(monkeypatch)
    assert build.run() > 0
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert build.up_to_date() and build.run() == 0


def test_a_binding_that_does_not_compile_leaves_the_library(build, capfd):
    build.compiles_binding(False)
    assert build.run() > 0
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "no header" in capfd.readouterr().err
    assert not build.up_to_date()
    build.compiles_binding(True)      # the next build makes what is missing alone
    assert build.run() == 0 and os.path.exists(build.BINDING) and build.up_to_date()


def test_a_binding_that_fails_takes_the_old_one_away(build, monkeypatch):
    build.compiles_binding(True)
    build.run()
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0")
    build.compiles_binding(False)
    build.run()
    assert not os.path.exists(build.BINDING)


def test_a_binding_of_another_torch_or_python_is_built_again(build, monkeypatch):
    build.compiles_binding(True)
    build.run()
    assert build.up_to_date() and build.run() == 0
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0")
    assert not build.up_to_date()
    build.run()
    assert build.up_to_date()
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "another")
    assert not build.up_to_date()
