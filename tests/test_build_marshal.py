"""The marshalling module's build is skipped where its prerequisites are missing."""
import os
import types

import pytest

from tree_speculative_decoding_07_b200 import build_lib


@pytest.fixture
def place(tmp_path, monkeypatch):
    """Builds go to a folder of their own, by a compiler that only notes that it was called."""
    monkeypatch.setattr(build_lib, "MARSHAL", str(tmp_path / "_marshal.so"))
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
