"""What build.py builds and when, with compilers that only write their output files."""
import importlib.metadata
import os
import shutil
import subprocess
import sys
import types

import pytest

from quantized_hybrid_layer_b200 import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """build.py on a copy of the sources, with the commands it runs recorded; g++ fails where `fail` says so."""
    f = types.SimpleNamespace(ran=[], fail=False, src=str(tmp_path / "pkg" / "csrc"), lib=str(tmp_path / "pkg" / "lib.so"),
                              marshal=str(tmp_path / "pkg" / "_marshal.so"))
    shutil.copytree(b.CSRC, f.src)
    os.makedirs(tmp_path / "include")
    shutil.copy(os.path.join(os.path.dirname(b.HERE), "include", "qhl_stage.h"), tmp_path / "include")
    for name, value in (("HERE", str(tmp_path / "pkg")), ("CSRC", f.src), ("BUILD", str(tmp_path / "_build")), ("LIB", f.lib),
                        ("MARSHAL", f.marshal)):
        monkeypatch.setattr(b, name, value)

    def run(cmd, **kw):
        f.ran.append("g++" if "g++" in cmd[0] else "link" if "-shared" in cmd else os.path.basename(cmd[cmd.index("-c") + 1]))
        if f.ran[-1] == "g++" and f.fail:
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as out:
            out.write(" ".join(cmd))
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return f


def built(f):
    f.ran.clear()
    assert b.build() == f.lib
    return sorted(f.ran)


ALL = sorted(b.SOURCES + ["g++", "link"])


def test_everything_once(fake):
    assert built(fake) == ALL
    assert os.path.exists(fake.lib) and os.path.exists(fake.marshal)
    assert built(fake) == []


def test_the_library_is_built_where_the_marshalling_module_is_not(fake, monkeypatch):
    """A user of the C library needs nvcc alone."""
    fake.fail = True
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        b.build()
    assert os.path.exists(fake.lib) and not os.path.exists(fake.marshal)


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_library_is_built_without_pytorch_or_a_host_compiler(fake, monkeypatch, capsys, missing):
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
    else:
        which = shutil.which
        monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    assert built(fake) == sorted(b.SOURCES + ["link"])
    assert os.path.exists(fake.lib) and not os.path.exists(fake.marshal)
    assert missing in capsys.readouterr().err.lower().replace("pytorch", "torch")


def test_each_is_rebuilt_for_its_own_sources(fake):
    built(fake)
    later = os.path.getmtime(fake.lib) + 100
    os.utime(os.path.join(fake.src, "marshal.cpp"), (later, later))
    assert built(fake) == ["g++"]
    os.utime(fake.marshal, (later, later))
    os.utime(os.path.join(fake.src, "pages.cu"), (later, later))
    assert built(fake) == sorted(b.SOURCES + ["link"])


def test_the_marshalling_module_is_rebuilt_for_another_pytorch(fake, monkeypatch):
    built(fake)
    assert built(fake) == []
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "99.1" if name == "torch" else version(name))
    assert built(fake) == ["g++"]
    assert built(fake) == []
