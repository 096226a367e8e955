"""build_library without the marshalling module: the library stands by itself."""

import os

import pytest

from ring_allreduce_reduction_virtual_amd import build


def fail(*_):
    raise RuntimeError("no such header")


def test_library_is_built_without_the_marshalling_module(monkeypatch, tmp_path, capsys):
    """A torch that ar_marshal.cpp does not fit costs the native checks of tensors only; an older module goes too."""
    old = tmp_path / "_armarshal.so"
    old.write_bytes(b"of another torch")
    monkeypatch.setattr(build, "MARSHAL_PATH", str(old))
    monkeypatch.setattr(build, "_build_main", lambda verbose=False: "libar.so")
    monkeypatch.setattr(build, "build_probe", lambda verbose=False: "libarprobe.so")
    monkeypatch.setattr(build, "build_marshal", fail)
    assert build.build_library() == "libar.so"
    assert "no such header" in capsys.readouterr().err and not os.path.exists(old)
    assert build.build_library() == "libar.so"


@pytest.mark.parametrize("part", ["_build_main", "build_probe"])
def test_other_parts_fail_the_build(monkeypatch, tmp_path, part):
    monkeypatch.setattr(build, "MARSHAL_PATH", str(tmp_path / "_armarshal.so"))
    for name in ("_build_main", "build_probe", "build_marshal"):
        monkeypatch.setattr(build, name, lambda verbose=False: "built")
    monkeypatch.setattr(build, part, fail)
    with pytest.raises(RuntimeError, match="header"):
        build.build_library()


def test_marshalling_module_fails_by_itself(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "MARSHAL_PATH", str(tmp_path / "_armarshal.so"))
    monkeypatch.setattr(build, "MARSHAL_SOURCE", "no_such_source.cpp")
    with pytest.raises(RuntimeError, match="build failed"):
        build.build_marshal()
