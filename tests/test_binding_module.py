"""The native part of the Python binding is used only with the torch and Python that it was built for."""
import types

import pytest

import submanifold_sparse_conv_amd as sc
from submanifold_sparse_conv_amd import _lib, build
from tests.test_build import small  # noqa: F401


def test_built_for_this_torch_and_python():
    import sys

    import torch

    said = _lib.binding().built_for
    assert torch.__version__ in said and "%d.%d" % sys.version_info[:2] in said


@pytest.mark.parametrize("more", [{}, dict(built_for="torch 1.0, Python 3.4"), dict(built_for="")])
def test_binding_of_another_torch_or_python_is_refused(monkeypatch, more):
    bound = []
    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(sc, "_binding", types.SimpleNamespace(bind=lambda *a: bound.append(a), **more), raising=False)
    with pytest.raises(ImportError, match="build"):
        _lib.binding()
    assert not bound and _lib._binding is None


def test_no_binding_of_older_sources_beside_a_new_library(small, monkeypatch):  # noqa: F811
    (small / "_binding.so").write_bytes(b"of an earlier build")
    monkeypatch.setenv("CXX", "false")
    with pytest.raises(RuntimeError):
        build.build()
    assert (small / "lib.so").exists() and not (small / "_binding.so").exists()
