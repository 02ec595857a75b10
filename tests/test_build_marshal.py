"""The marshalling module's build: skipped where its prerequisites are missing, repeated for another
torch, loud when the compiler fails, and a module of another torch is refused."""
import os
import subprocess
import types

import pytest

import tree_speculative_decoding_07_b200 as tv
from tree_speculative_decoding_07_b200 import build_lib


@pytest.fixture
def place(tmp_path, monkeypatch):
    """Builds go to a folder of their own, by a compiler that only notes that it was called."""
    monkeypatch.setattr(build_lib, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build_lib, "MARSHAL_STAMP", str(tmp_path / "_marshal.built_for"))
    calls = []

    def compiler(cmd):
        calls.append(cmd)
        open(build_lib.MARSHAL, "w").close()

    monkeypatch.setattr(build_lib, "subprocess", types.SimpleNamespace(check_call=compiler))
    return calls


def test_without_a_compiler_or_headers_it_says_so_and_goes_on(place, monkeypatch, tmp_path, capsys):
    monkeypatch.setenv("CXX", "a-compiler-that-is-not-there")
    assert build_lib.build_marshal() is None
    assert "a-compiler-that-is-not-there" in capsys.readouterr().err
    monkeypatch.delenv("CXX")
    import torch
    monkeypatch.setattr(torch, "__file__", str(tmp_path / "torch" / "__init__.py"))
    assert build_lib.build_marshal() is None
    assert "Tensor.h" in capsys.readouterr().err
    assert place == [] and not os.path.exists(build_lib.MARSHAL)


def test_it_is_built_again_for_another_torch_only(place, monkeypatch):
    assert build_lib.build_marshal() == build_lib.MARSHAL and len(place) == 1
    build_lib.build_marshal()
    assert len(place) == 1
    import torch
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    build_lib.build_marshal()
    build_lib.build_marshal()
    assert len(place) == 2 and any("0.0.other" in x for x in place[1])
    os.remove(build_lib.MARSHAL_STAMP)  # nobody knows what that module was built for
    build_lib.build_marshal()
    build_lib.build_marshal(force=True)
    assert len(place) == 4


def test_a_failed_build_raises_and_leaves_nothing_that_passes_for_one(place, monkeypatch):
    build_lib.build_marshal()

    def fails(cmd):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(build_lib.subprocess, "check_call", fails)
    with pytest.raises(subprocess.CalledProcessError):
        build_lib.build_marshal(force=True)
    with pytest.raises(subprocess.CalledProcessError):
        build_lib.build_marshal()


def test_a_module_of_another_torch_is_refused(monkeypatch):
    import torch
    assert tv._native().built_for == build_lib.marshal_target()
    monkeypatch.setattr(tv, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.other")
    with pytest.raises(ImportError, match="0.0.other"):
        tv._native()
