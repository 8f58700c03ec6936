"""The library builds without torch, and the compiled binding follows torch and Python. No GPU
needed."""
import os
import subprocess
import sys

import pytest

import paged_kv_cache_442_b200 as pa
from paged_kv_cache_442_b200 import build as pa_build

WITHOUT_TORCH = """
import glob, os, sys
sys.modules["torch"] = None            # import torch raises ImportError
sys.path.insert(0, {root!r})
from paged_kv_cache_442_b200 import build
tmp = {tmp!r}
build.BUILD_DIR = os.path.join(tmp, "objects")
build.LIB, build.BINDING = os.path.join(tmp, "libpa.so"), os.path.join(tmp, "_pa_torch.so")
build._sources = lambda: [os.path.join(tmp, "one.cpp")]
assert build.build() == build.LIB and os.path.exists(build.LIB)
assert not glob.glob(os.path.join(tmp, "_pa_torch*"))
assert build.up_to_date()
import paged_kv_cache_442_b200          # the package itself needs no torch either
"""


def test_the_library_builds_without_torch(tmp_path):
    (tmp_path / "one.cpp").write_text('extern "C" int one() { return 1; }\n')
    code = WITHOUT_TORCH.format(root=pa_build.ROOT, tmp=str(tmp_path))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_a_binding_of_another_torch_is_not_up_to_date(tmp_path, monkeypatch):
    pa_build.build()
    assert pa_build.up_to_date()
    monkeypatch.setattr(pa_build, "binding_target", lambda: "torch 99.0, Python 3.12")
    assert not pa_build.up_to_date()


@pytest.mark.parametrize("held", [b"", b"\x7fELF pa_built_for{torch 99.0, Python 3.12}"])
def test_a_binding_of_another_or_an_unknown_torch_is_not_loaded(held, tmp_path, monkeypatch):
    pa_build.build()
    other = tmp_path / "_pa_torch.so"
    other.write_bytes(held)
    monkeypatch.setattr(pa_build, "BINDING", str(other))
    monkeypatch.setattr(pa, "BINDING_PATH", str(other))
    monkeypatch.setattr(pa, "_native_module", None)
    with pytest.raises(ImportError, match="built for"):
        pa._native()


def test_the_binding_that_is_built_names_its_torch():
    pa_build.build()
    assert os.path.exists(pa_build.BINDING)
    assert pa_build.built_for() == pa_build.binding_target()
