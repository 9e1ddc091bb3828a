"""What the build needs, and when it builds anew.  Compilers and linkers are faked: no
GPU, and no compilation."""
import importlib.util
import os
import shutil

import pytest

from exact_attention_82_gb300 import build as b


@pytest.fixture
def commands(tmp_path, monkeypatch):
    """The build in a folder of its own, its commands recorded and their outputs written empty."""
    made = []

    class Done:
        returncode, stdout, stderr = 0, "", ""

    def run(cmd, **kw):
        made.append(list(cmd))
        open(cmd[cmd.index("-o") + 1], "w").close()
        return Done

    out = tmp_path / "out"
    monkeypatch.setattr(b, "OUT_DIR", str(out))
    monkeypatch.setattr(b, "LIB_PATH", str(out / b.LIB_NAME))
    monkeypatch.setattr(b, "BINDING_PATH", str(out / "fa_binding.so"))
    monkeypatch.setattr(b, "nvcc", lambda: "/nowhere/bin/nvcc")
    monkeypatch.setattr(b.subprocess, "run", run)
    return made


def without(monkeypatch, what):
    if what == "torch":
        find = importlib.util.find_spec
        monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    else:
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == what else which(name, *a, **k))


@pytest.mark.parametrize("what", ["torch", "g++"])
def test_the_library_is_built_without(what, commands, monkeypatch):
    without(monkeypatch, what)
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert {os.path.basename(c[0]) for c in commands} == {"nvcc"}
    n = len(commands)
    assert b.build() == b.LIB_PATH and len(commands) == n, "built again"


@pytest.mark.parametrize("what", ["torch", "g++"])
def test_the_binding_says_what_is_missing_and_leaves_the_library(what, commands, monkeypatch):
    without(monkeypatch, what)
    with pytest.raises(RuntimeError, match=what.replace("+", "[+]")):
        b.build_binding(force=True)
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)


def test_a_binding_that_does_not_compile_leaves_the_library(commands, monkeypatch):
    run = b.subprocess.run

    def fails(cmd, **kw):
        done = run(cmd, **kw)
        if b.BINDING_SOURCE in " ".join(cmd):
            class Failed(done):
                returncode, stderr = 1, "no such header"
            return Failed
        return done

    monkeypatch.setattr(b.subprocess, "run", fails)
    with pytest.raises(RuntimeError, match="no such header"):
        b.build_binding()
    assert os.path.exists(b.LIB_PATH) and not os.path.exists(b.BINDING_PATH)


@pytest.mark.parametrize("changed", ["torch", "python", "build.py"])
def test_the_binding_is_built_anew_after_a_change_of(changed, commands, monkeypatch, tmp_path):
    """It holds torch's and Python's binary interfaces, whose change leaves the sources' times alone."""
    torch_dir = tmp_path / "torch"
    torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1.0'")
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: type("Spec", (), {"origin": str(torch_dir / "__init__.py")})
                        if name == "torch" else find(name, *a))
    b.build_binding()
    n = len(commands)
    b.build_binding()
    assert len(commands) == n, "built again without a change"
    if changed == "torch":
        (torch_dir / "version.py").write_text("__version__ = '1.1'")
    elif changed == "python":
        get = b.sysconfig.get_config_var
        monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: ".cpython-999.so" if name == "EXT_SUFFIX" else get(name))
    else:
        later = os.path.getmtime(b.LIB_PATH) + 100
        mtime = os.path.getmtime
        monkeypatch.setattr(os.path, "getmtime", lambda p: later if os.path.basename(p) == "build.py" else mtime(p))
    assert not b.binding_up_to_date()
    assert b.up_to_date() == (changed != "build.py")
    b.build_binding()
    assert len(commands) > n


def test_builds_at_the_same_time_write_files_of_their_own(commands):
    """Nothing that one build compiles lies where another one compiles the same source."""
    written = []
    for _ in range(2):
        b.build_binding(force=True)
        written.append({c[c.index("-o") + 1] for c in commands})
        commands.clear()
    assert len(written[0]) == len(b.SOURCES) + 3 and not written[0] & written[1]
    assert sorted(os.listdir(b.OUT_DIR)) == ["fa_binding.so", "fa_binding.so.key", b.LIB_NAME]
