"""What build() leaves behind when a step of it cannot run.  The compilers are replaced by
writers of empty files, so that only the order and the handling of failures is tested."""
import os
import sys

import pytest

from two_compressed_kv_gb300 import build_lib


@pytest.fixture
def box(monkeypatch, tmp_path):
    """build_lib with its outputs under tmp_path, an old marshalling module there, no compilers."""
    monkeypatch.setattr(build_lib, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(build_lib, "LIB", str(tmp_path / "libmkv.so"))
    monkeypatch.setattr(build_lib, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build_lib, "nvcc", lambda: "/opt/cuda/bin/nvcc")
    (tmp_path / "_marshal.so").write_text("old")

    def run(cmd):
        if cmd[0] == "g++" and run.gxx_fails:
            raise RuntimeError("g++: no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("new")
        return ""
    run.gxx_fails = False
    monkeypatch.setattr(build_lib, "_run", run)
    return run


def test_build_makes_both(box):
    assert build_lib.build() == build_lib.LIB
    assert open(build_lib.LIB).read() == open(build_lib.MARSHAL).read() == "new"


def test_library_builds_without_torch(box, monkeypatch, capsys):
    """The C library needs nvcc alone; a marshalling module of an older build, whose argument
    structs may not be this library's, does not stay."""
    monkeypatch.setitem(sys.modules, "torch", None)
    assert build_lib.build() == build_lib.LIB
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.MARSHAL)
    assert "torch" in capsys.readouterr().err


def test_library_survives_a_failing_marshal_step(box):
    box.gxx_fails = True
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        build_lib.build()
    assert os.path.exists(build_lib.LIB) and not os.path.exists(build_lib.MARSHAL)


def test_nothing_half_made_stays(box, monkeypatch):
    """A failing nvcc step leaves the library and the module of the last build, and no other file."""
    build_lib.build()
    here = os.path.dirname(build_lib.LIB)
    was = sorted(os.listdir(here))

    def run(cmd):
        if "-c" in cmd:
            raise RuntimeError("nvcc: no such header")
        return box(cmd)
    monkeypatch.setattr(build_lib, "_run", run)
    with pytest.raises(RuntimeError, match="nvcc"):
        build_lib.build()
    assert sorted(os.listdir(here)) == was
