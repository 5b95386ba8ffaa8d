"""libpsa.so needs nvcc alone: where the binding's native module cannot be
built, the library is, and the binding does without the module.  Host-only."""

import os

import pytest

from block_sparse_attention_psa_b200 import build


@pytest.mark.parametrize("error", [ModuleNotFoundError("No module named 'torch'"), FileNotFoundError("g++"),
                                   RuntimeError("g++ failed: Python.h: No such file or directory")], ids=repr)
def test_the_library_is_built_without_the_native_module(monkeypatch, tmp_path, capsys, error):
    def fails():
        raise error

    old = tmp_path / "_call.so"
    old.write_text("built from other sources")
    monkeypatch.setattr(build, "CALL", str(old))
    monkeypatch.setattr(build, "_build_call", fails)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not old.exists()
    assert "_call.so is not built" in capsys.readouterr().err
