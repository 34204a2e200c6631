"""When the native module for torch tensors is built again (no compiler runs here)."""
import importlib.util
import os
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def b(tmp_path, monkeypatch):
    spec = importlib.util.spec_from_file_location("_h3blk_build_test", os.path.join(ROOT, "joint_video_audio_b200", "build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.OBJDIR, m.MODULE = str(tmp_path / "obj"), str(tmp_path / "_fp4_torch.so")
    os.makedirs(m.OBJDIR)
    m.runs = 0

    def run(cmd, **kw):
        m.runs += 1
        open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(m.subprocess, "run", run)
    return m


def _torch_at(b, monkeypatch, path, version):
    os.makedirs(path, exist_ok=True)
    f = os.path.join(path, "version.py")
    with open(f, "w") as h:
        h.write(f"__version__ = '{version}'\n")
    os.utime(f, (1e9, 1e9))  # installed long before the module was built
    monkeypatch.setattr(b, "find_spec", lambda name: types.SimpleNamespace(origin=os.path.join(path, "__init__.py")))


def test_built_once(b):
    for _ in range(3):
        b._build_module(False)
    assert b.runs == 1
    b._build_module(True)
    assert b.runs == 2


def test_another_torch(b, monkeypatch, tmp_path):
    """Of another version or in another place, however old its files are."""
    _torch_at(b, monkeypatch, str(tmp_path / "a"), "1")
    b._build_module(False)
    b._build_module(False)
    assert b.runs == 1
    _torch_at(b, monkeypatch, str(tmp_path / "a"), "2")
    b._build_module(False)
    assert b.runs == 2
    _torch_at(b, monkeypatch, str(tmp_path / "b"), "2")
    b._build_module(False)
    b._build_module(False)
    assert b.runs == 3


def test_another_python(b, monkeypatch):
    b._build_module(False)
    monkeypatch.setattr(b.sysconfig, "get_config_var", lambda name: "cpython-399-other")
    b._build_module(False)
    assert b.runs == 2


def test_a_module_of_unknown_origin(b):
    b._build_module(False)
    os.remove(os.path.join(b.OBJDIR, "_fp4_torch.stamp"))
    b._build_module(False)
    assert b.runs == 2


def test_a_failed_build_leaves_the_old_one(b, monkeypatch):
    b._build_module(False)
    ok = b.subprocess.run
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, **kw: types.SimpleNamespace(returncode=1, stdout="", stderr="no"))
    with pytest.raises(RuntimeError):
        b._build_module(True)
    monkeypatch.setattr(b.subprocess, "run", ok)
    b._build_module(False)
    assert b.runs == 1


def test_every_header_counts(b):
    names = {os.path.basename(h) for h in b._headers()}
    assert {"h3blk.h", "ptx.cuh", "kernels.cuh", "api_internal.h"} <= names
