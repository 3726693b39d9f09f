"""What the build makes of what is installed, without compiling anything."""
import os
import types

import pytest

import compressed_sparse_kv_04_b200
from compressed_sparse_kv_04_b200 import binding
from compressed_sparse_kv_04_b200 import build as csa_build


@pytest.fixture
def built(monkeypatch, tmp_path):
    """The build in an empty folder, with compilers that only leave their file."""
    for name, file in (("BUILD", "_build"), ("LIB", "libcsa.so"), ("CALLS", "_calls.so"),
                       ("CALLS_TAG", "calls.tag")):
        monkeypatch.setattr(csa_build, name, str(tmp_path / file))
    monkeypatch.setattr(csa_build, "_compile", lambda src: (src + ".o", ""))

    def link(cmd):
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(csa_build.subprocess, "check_call", link)
    return tmp_path


def test_the_library_is_linked_where_the_native_calls_fail(built, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")
    monkeypatch.setattr(csa_build, "_compile_calls", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        csa_build.build()
    assert os.path.exists(csa_build.LIB)
    assert not csa_build.up_to_date()


@pytest.mark.parametrize("missing", ["torch", "headers"])
def test_the_library_needs_neither_torch_nor_python_headers(built, monkeypatch, missing, capsys):
    def never():
        raise AssertionError("_calls.so has nothing to compile against")
    monkeypatch.setattr(csa_build, "_compile_calls", never)
    if missing == "torch":
        find = csa_build.importlib.util.find_spec
        monkeypatch.setattr(csa_build.importlib.util, "find_spec",
                            lambda name, *a: None if name == "torch" else find(name, *a))
    else:
        monkeypatch.setattr(csa_build.sysconfig, "get_paths", lambda: {"include": str(built)})
    assert csa_build.build() == csa_build.LIB
    assert os.path.exists(csa_build.LIB) and "_calls.so is not built" in capsys.readouterr().err
    assert csa_build.up_to_date()
    csa_build.build()


def test_each_target_follows_its_own_sources(built, monkeypatch):
    made = []

    def calls():
        made.append("calls")
        open(csa_build.CALLS, "w").close()
        open(csa_build.CALLS_TAG, "w").write(csa_build.calls_tag())
    monkeypatch.setattr(csa_build, "_compile_calls", calls)
    monkeypatch.setattr(csa_build, "_compile", lambda src: (made.append("lib"), "")[::-1])
    csa_build.build()
    assert csa_build.up_to_date() and set(made) == {"calls", "lib"}
    made.clear()
    os.utime(csa_build.CALLS, (0, 0))
    assert not csa_build.up_to_date()
    csa_build.build()
    assert made == ["calls"]
    made.clear()
    os.utime(csa_build.LIB, (0, 0))
    csa_build.build()
    assert set(made) == {"lib"}


def test_native_calls_of_another_torch_or_python_are_rebuilt(built, monkeypatch):
    monkeypatch.setattr(csa_build, "_compile_calls", lambda: None)
    csa_build.build()
    open(csa_build.CALLS, "w").close()
    assert not csa_build.calls_up_to_date()  # built by nobody knows what
    open(csa_build.CALLS_TAG, "w").write(csa_build.calls_tag())
    assert csa_build.up_to_date()
    for other in ("torch 2.99, C++11 ABI 1, Python cpython-312-x86_64-linux-gnu",
                  csa_build.calls_tag().replace("cpython-3", "cpython-4")):
        monkeypatch.setattr(csa_build, "calls_tag", lambda: other)
        assert not csa_build.up_to_date()


def test_the_binding_refuses_native_calls_of_another_torch(monkeypatch):
    csa_build.build()
    monkeypatch.setattr(binding, "_calls", None)
    assert binding._native().built_for == csa_build.calls_tag()
    monkeypatch.setattr(binding, "_calls", None)
    monkeypatch.setattr(csa_build, "calls_tag", lambda: "torch 2.99")
    with pytest.raises(RuntimeError, match="built for .* this is torch 2.99"):
        binding._native()
    # A module from before modules said what they were built for.
    monkeypatch.setattr(compressed_sparse_kv_04_b200, "_calls", types.SimpleNamespace())
    with pytest.raises(RuntimeError, match="built for an unknown torch"):
        binding._native()
