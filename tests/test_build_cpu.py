"""What the build makes, with a stand-in for the compilers: the library needs no
torch, only the native half of the Python binding does."""
import importlib.util
import os
import subprocess

import pytest

from speculative_decoding_verify_pass_gb300 import _build


class Toolchain:
    """Stands in for nvcc and g++: writes the output file and keeps the command."""

    def __init__(self, fails=""):
        self.fails, self.commands = fails, []

    def run(self, cmd, **_):
        self.commands.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        if self.fails and any(self.fails in a for a in cmd):
            return subprocess.CompletedProcess(cmd, 1, b"no such header")
        with open(out, "w") as f:
            f.write("made")
        return subprocess.CompletedProcess(cmd, 0, b"")

    def start(self, cmd, **kw):
        done = self.run(cmd, **kw)
        done.communicate = lambda: (done.stdout, None)
        return done


@pytest.fixture
def tools(monkeypatch, tmp_path):
    t = Toolchain()
    for name in ("LIB", "BINDING"):
        monkeypatch.setattr(_build, name, str(tmp_path / os.path.basename(getattr(_build, name))))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(_build.subprocess, "Popen", t.start)
    monkeypatch.setattr(_build.subprocess, "run", t.run)
    return t


def without_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))


def made(cmds, path):
    return [c for c in cmds if c[c.index("-o") + 1].startswith(path)]


def test_the_library_is_built_without_torch(tools, monkeypatch):
    without_torch(monkeypatch)
    assert _build.build() == _build.LIB
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)
    assert not any("binding" in a for c in tools.commands for a in c)
    assert len(made(tools.commands, _build.LIB)) == 1
    n = len(tools.commands)
    _build.build()                                     # built: nothing to do
    assert len(tools.commands) == n


def test_a_torch_that_appears_later_gets_its_binding(tools, monkeypatch):
    pytest.importorskip("torch")
    with monkeypatch.context() as m:
        without_torch(m)
        _build.build()
    _build.build()
    assert os.path.exists(_build.BINDING)
    n = len(tools.commands)
    _build.build()
    assert len(tools.commands) == n


def test_a_binding_that_fails_leaves_the_library(tools):
    """Headers of torch or Python that do not compile are reported, after the library is in place."""
    pytest.importorskip("torch")
    tools.fails = "binding.cpp"
    with pytest.raises(RuntimeError, match="no such header"):
        _build.build()
    assert os.path.exists(_build.LIB) and not os.path.exists(_build.BINDING)


def test_a_source_that_fails_is_reported(tools):
    tools.fails = "pages.cu"
    with pytest.raises(RuntimeError, match="pages.cu"):
        _build.build()
    assert not os.path.exists(_build.LIB)


@pytest.mark.parametrize("what", ["torch", "python", "place"])
def test_a_binding_of_another_torch_or_python_is_rebuilt(tools, monkeypatch, tmp_path, what):
    """No source changes, but the ABI that _paged.so was compiled for does."""
    root = tmp_path / "site" / "torch"
    (root / "lib").mkdir(parents=True)
    (root / "lib" / "libc10_cuda.so").write_text("")
    (root / "version.py").write_text("__version__ = '2.9.1'\n")
    (root / "__init__.py").write_text("")
    place = [root]
    find = importlib.util.find_spec

    class Spec:
        @property
        def origin(self):
            return str(place[0] / "__init__.py")
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name, *a: Spec() if name == "torch" else find(name, *a))
    _build.build()
    n = len(tools.commands)
    _build.build()
    assert len(tools.commands) == n and os.path.exists(_build.BINDING)
    if what == "torch":
        (root / "version.py").write_text("__version__ = '2.11.0'\n")
    elif what == "python":
        monkeypatch.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-313-other")
    else:
        place[0] = root.rename(tmp_path / "site" / "torch2")
    _build.build()
    assert made(tools.commands[n:], _build.BINDING)
    n = len(tools.commands)
    _build.build()
    assert len(tools.commands) == n
