"""What building the library needs: hipcc, and torch for the binding's native
module alone.  A stand-in for the compiler records its calls."""

import importlib.util
import os
import stat
import sys

import pytest

from conftest import ROOT

PACKAGE = os.path.join(ROOT, "quantized_linear_layers_awq_amd")


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module over an empty folder, with a compiler that writes empty outputs and no other on the path."""
    spec = importlib.util.spec_from_file_location("build_under_test", os.path.join(PACKAGE, "build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    fake = tmp_path / "hipcc"
    fake.write_text(f"#!{sys.executable}\nimport sys\nopen(sys.argv[sys.argv.index('-o') + 1], 'w').close()\n")
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("HIPCC", str(fake))
    monkeypatch.setenv("PATH", str(tmp_path))
    for name, path in (("HERE", ""), ("BUILD_DIR", "objects"), ("LIB_PATH", "libtilefuse.so"), ("CALLS_PATH", "_calls.so")):
        monkeypatch.setattr(module, name, str(tmp_path / path))
    return module


def test_hipcc_builds_everything(build, tmp_path):
    assert build.build() == str(tmp_path / "libtilefuse.so")
    assert (tmp_path / "libtilefuse.so").exists() and (tmp_path / "_calls.so").exists()


def test_the_library_builds_without_torch(build, tmp_path, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # as if it were not installed
    assert build.build() == str(tmp_path / "libtilefuse.so")
    assert (tmp_path / "libtilefuse.so").exists() and not (tmp_path / "_calls.so").exists()
