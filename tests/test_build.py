"""The build of the library and of the native part of the Python binding, one without the other."""
import ctypes

import pytest

from submanifold_sparse_conv_amd import build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one small source in a folder of its own."""
    src = tmp_path / "one.hip"
    src.write_text('extern "C" int one() { return 1; }\n')
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    for name, at in (("LIB", "lib.so"), ("BINDING", "_binding.so"), ("BUILD_DIR", "objects")):
        monkeypatch.setattr(build, name, str(tmp_path / at))
    return tmp_path


@pytest.mark.parametrize("cxx", ["false", "/no/such/compiler"])
def test_library_without_the_binding(small, monkeypatch, cxx):
    """A user of the C ABI gets the library where the binding does not compile (no Python or torch headers); the build
    says that it failed all the same."""
    monkeypatch.setenv("CXX", cxx)
    with pytest.raises((RuntimeError, OSError)):
        build.build()
    assert ctypes.CDLL(str(small / "lib.so")).one() == 1
    assert not (small / "_binding.so").exists()
