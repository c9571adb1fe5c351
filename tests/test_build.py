"""The build, on a small source folder of its own."""
import importlib.util
import os

import pytest

FILE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_deterministic_bf16_gb300", "build.py")


@pytest.fixture
def build(tmp_path, monkeypatch):
    """build.py run as a script runs it (the package is not imported), pointed at tmp_path."""
    spec = importlib.util.spec_from_file_location("build_alone", FILE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    pkg = tmp_path / "pkg"
    (pkg / "csrc").mkdir(parents=True)
    (pkg / "csrc" / "one.cu").write_text('extern "C" __attribute__((visibility("default"))) int one() { return 1; }\n')
    (pkg / "csrc" / "bind.cpp").write_text("#include <torch/extension.h>\n")
    for name, path in (("PKG", pkg), ("CSRC", pkg / "csrc"), ("OUT", pkg / "libdetffn.so"), ("NATIVE", pkg / "_native.so"),
                       ("BUILD", tmp_path / "_build")):
        monkeypatch.setattr(m, name, str(path))
    return m


def test_the_library_builds_without_pytorch(build, monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    for _ in range(2):   # from nothing, and with nothing left to do
        assert build.build() == build.OUT and os.path.exists(build.OUT)
        assert not os.path.exists(build.NATIVE)
    assert build.build(force=True) == build.OUT
