"""CPU tests of the build and of the CPython module between the library and torch."""

import importlib.util
import os

import pytest
import torch

from paged_kv_decode_splitk_gb300 import api, build, pd


def test_library_builds_without_torch(monkeypatch):
    """The C library needs no PyTorch: nothing but the module over torch's tensors is left out."""
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    before = os.path.getmtime(build.BINDING)
    assert build.build() == build.LIB
    assert os.path.getmtime(build.BINDING) == before


def _rope_declined_then_checked():
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    rotation = type("Rotation", (), {"head_dim": 64, "handle": 1})
    with pytest.raises(ValueError, match="x: BF16"):  # by the checked way, which says what is wrong
        api._check_rope(rotation, x, torch.zeros(2, dtype=torch.int32), None, 0)
    assert pd.quick().rope(1, 64, x, x, None, 0) is NotImplemented


def test_module_missing(monkeypatch, tmp_path):
    monkeypatch.setattr(pd, "_quick", None)
    monkeypatch.setattr(pd, "PKG", str(tmp_path))
    with pytest.warns(RuntimeWarning, match="is missing"):
        pd.quick()
    _rope_declined_then_checked()


def test_module_that_does_not_load(monkeypatch, tmp_path):
    monkeypatch.setattr(pd, "_quick", None)
    monkeypatch.setattr(pd, "PKG", str(tmp_path))
    os.mkdir(tmp_path / "_build")
    (tmp_path / "_build" / "pd_binding.so").write_bytes(b"no library")
    with pytest.warns(RuntimeWarning, match="does not load"):
        pd.quick()
    _rope_declined_then_checked()


def test_module_of_another_torch(monkeypatch):
    assert pd.quick().built_for == torch.__version__
    monkeypatch.setattr(pd, "_quick", None)
    monkeypatch.setattr(torch, "__version__", "1.0")
    with pytest.warns(RuntimeWarning, match="was built for torch"):
        pd.quick()
    _rope_declined_then_checked()


def test_module_in_use(recwarn):
    """Nothing stands in for it where it is as built."""
    assert type(pd.quick()).__name__ == "module" and not [w for w in recwarn if w.category is RuntimeWarning]
