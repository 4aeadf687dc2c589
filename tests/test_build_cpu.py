"""The build of the paged-cache calls' binding: with torch or Python upgraded, and without them."""
import importlib.util
import os

import pytest

from bit_quantised_gemm_b200 import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """The commands of a build whose outputs lie elsewhere; each leaves its output behind."""
    ran = []

    def run(cmd, check):
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()

    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(build, "BIND_RECORD", str(tmp_path / "bind.txt"))
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran


def test_the_binding_is_built_once(commands):
    assert build.build_binding() and len(commands) == 1
    assert build.build_binding() and len(commands) == 1
    assert build.build_binding(force=True) and len(commands) == 2


def test_another_torch(commands):
    build.build_binding()
    text = open(build.BIND_RECORD).read()
    with open(build.BIND_RECORD, "w") as f:
        f.write(text.replace("__version__ = '", "__version__ = '1."))
    assert text != open(build.BIND_RECORD).read()
    build.build_binding()
    assert len(commands) == 2 and open(build.BIND_RECORD).read() == text


def test_another_python(commands, monkeypatch):
    build.build_binding()
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": os.path.dirname(__file__)})
    assert not build.build_binding()  # no headers there
    assert len(commands) == 1
    assert build.sysconfig.get_config_var("SOABI") in importlib.util.find_spec("bit_quantised_gemm_b200._bind").origin


def test_without_torch(commands, monkeypatch, capsys):
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    assert not build.build_binding()
    assert not commands and "no torch" in capsys.readouterr().err
