"""When the compiled Python binding is built again, and when it is left out."""
import os

import pytest

from state_space_model_gb300 import build


@pytest.fixture
def own_binding(monkeypatch, tmp_path):
    """build.build() with a binding and a stamp of the test's own."""
    build.build()
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_attn_ext.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "stamp"), raising=False)


def test_binding_is_built_once(own_binding):
    assert not build._binding_up_to_date()
    build.build()
    assert build._binding_up_to_date()
    first = os.stat(build.BINDING).st_mtime_ns
    build.build()
    assert os.stat(build.BINDING).st_mtime_ns == first


@pytest.mark.parametrize("change", ["python", "torch"])
def test_binding_is_built_again_for_another_python_or_torch(own_binding, monkeypatch, change):
    build.build()
    if change == "python":
        monkeypatch.setattr(build.sys, "version", "3.99.0")
    else:
        real = os.stat
        monkeypatch.setattr(build.os, "stat", lambda p, *a, **k: Later(real(p, *a, **k))
                            if str(p).endswith("libtorch_python.so") else real(p, *a, **k))
    assert not build._binding_up_to_date()


class Later:
    """A file's status, an hour on."""

    def __init__(self, st):
        self.st = st

    def __getattr__(self, name):
        return getattr(self.st, name)

    @property
    def st_mtime_ns(self):
        return self.st.st_mtime_ns + 3600 * 10 ** 9


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_library_is_built_without_torch_or_host_compiler(own_binding, monkeypatch, capfd, missing):
    if missing == "torch":
        import importlib.util
        real = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
        monkeypatch.setitem(build.sys.modules, "torch", None)      # importing it fails
    else:
        real = build.shutil.which
        monkeypatch.setattr(build.shutil, "which", lambda n, *a, **k: None if n == "g++" else real(n, *a, **k))
        run = build.subprocess.run

        def no_compiler(cmd, *a, **k):
            if cmd[0] == "g++":
                raise FileNotFoundError(2, "No such file or directory", "g++")
            return run(cmd, *a, **k)

        monkeypatch.setattr(build.subprocess, "run", no_compiler)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not os.path.exists(build.BINDING)
    assert missing in capfd.readouterr().err


def test_compiler_that_fails_to_start_is_tried_again(monkeypatch):
    """Starting a process can fail with EFAULT while other threads start theirs."""
    real, left = build.subprocess.run, [2]

    def run(cmd, *a, **k):
        if left[0]:
            left[0] -= 1
            raise OSError(14, "Bad address", cmd[0])
        return real(cmd, *a, **k)

    monkeypatch.setattr(build.subprocess, "run", run)
    assert build._run(["true"]).returncode == 0
    left[0] = 3
    with pytest.raises(OSError):
        build._run(["true"])
    left[0] = 0
    with pytest.raises(FileNotFoundError):
        build._run(["no-such-compiler"])
