"""CPU tests of the build of the attention binding: the library does not depend
on it, and a new one takes the old one's place whole."""
import os
import stat

import pytest

from expert_layer_gb300 import _build


def compiler(path, body):
    path.write_text("#!/bin/sh\n" + body)
    path.chmod(path.stat().st_mode | stat.S_IXUSR)
    return str(path)


@pytest.fixture
def apart(tmp_path, monkeypatch):
    """A binding in a folder of its own; the library's objects as they are."""
    _build.build()
    at = tmp_path / "_attn_binding.so"
    monkeypatch.setattr(_build, "BINDING", str(at))
    return at


@pytest.mark.parametrize("why", ["no compiler", "it fails", "no PyTorch"])
def test_library_is_built_without_the_binding(apart, tmp_path, monkeypatch, why):
    apart.write_bytes(b"for other sources")
    os.utime(apart, (1, 1))
    if why == "no compiler":
        monkeypatch.setattr(_build, "CXX", str(tmp_path / "missing"))
    elif why == "it fails":
        monkeypatch.setattr(_build, "CXX", compiler(tmp_path / "cxx", "echo no header >&2; exit 1\n"))
    else:
        def missing(verbose=False):
            raise ImportError("no module torch")
        monkeypatch.setattr(_build, "build_binding", missing)
    with pytest.warns(UserWarning, match="attention functions are not available"):
        lib = _build.build()
    assert os.path.exists(lib) and lib == _build.LIB
    if why != "no PyTorch":
        assert not apart.exists()                    # the one that does not fit is gone
    assert not list(tmp_path.glob("*.so.*")), "parts left behind"


def test_library_is_linked_before_the_binding_fails(tmp_path, monkeypatch):
    linked = tmp_path / "libmoe_gb300.so"
    _build.build()
    monkeypatch.setattr(_build, "LIB", str(linked))
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "_attn_binding.so"))
    monkeypatch.setattr(_build, "CXX", str(tmp_path / "missing"))
    with pytest.warns(UserWarning):
        assert _build.build() == str(linked)
    assert linked.exists()


def test_new_binding_takes_the_place_of_a_mapped_one(apart, tmp_path, monkeypatch):
    apart.write_bytes(b"old")
    os.utime(apart, (1, 1))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path))          # where it is noted what the binding is for
    monkeypatch.setattr(_build, "CXX", compiler(
        tmp_path / "cxx", 'while [ "$1" != "-o" ]; do shift; done\nprintf new > "$2"\n'))
    with open(apart, "rb") as old:
        assert _build.build_binding() == str(apart)
        assert old.read() == b"old"
    assert apart.read_bytes() == b"new"
