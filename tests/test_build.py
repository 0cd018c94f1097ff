"""What the package's build needs and leaves, with stand-ins for the compilers
(no GPU, nothing of the package's own build is touched)."""
import os
import stat
import sysconfig

import pytest
import torch

import mla_attention_nvfp4_gb300 as mla
from mla_attention_nvfp4_gb300 import build as b


@pytest.fixture
def sandbox(tmp_path, monkeypatch):
    """An empty build folder, one source, and an nvcc that writes its output file."""
    fake = tmp_path / "nvcc"
    fake.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do if [ "$1" = -o ]; then echo built > "$2"; fi; shift; done\n')
    fake.chmod(fake.stat().st_mode | stat.S_IEXEC)
    monkeypatch.setenv("NVCC", str(fake))
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmla_nvfp4.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "binding.so"))
    return tmp_path


def test_the_library_is_built_where_the_binding_cannot_be(sandbox, monkeypatch):
    monkeypatch.setenv("CXX", str(sandbox / "no-such-compiler"))
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_the_library_is_not_built_again_for_the_binding(sandbox, monkeypatch):
    cxx = sandbox / "nvcc"  # writes its output as well
    monkeypatch.setenv("CXX", str(cxx))
    b.build()
    before = os.stat(b.LIB).st_mtime_ns
    os.remove(b.BINDING)
    b.build()
    assert os.path.exists(b.BINDING) and os.stat(b.LIB).st_mtime_ns == before


def test_calls_without_the_binding_load_the_library(tmp_path, monkeypatch):
    mla.load_library()
    monkeypatch.setattr(mla, "_LIB", None)
    monkeypatch.setattr(mla, "_FP8", None)
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "missing.so"))
    monkeypatch.setenv("CXX", str(tmp_path / "no-such-compiler"))
    assert mla.load_library().mla_nvfp4_status_string(0)
    with pytest.raises(RuntimeError, match="8-bit"):
        mla.mla_nvfp4_fp8_quantize(torch.zeros(2, 128).bfloat16())


def test_the_binding_is_of_this_interpreter_and_this_pytorch(tmp_path, monkeypatch):
    # a tree built beside another PyTorch or Python is not taken for current
    suffix = sysconfig.get_config_var("EXT_SUFFIX")
    assert torch.__version__ in os.path.basename(b.BINDING) and b.BINDING.endswith(suffix)
    assert b.binding_name() == os.path.basename(b.BINDING)
    other = tmp_path / "torch"
    other.mkdir()
    (other / "__init__.py").write_text("")
    (other / "version.py").write_text("__version__ = '9.9.0'\n")

    class Spec:
        origin = str(other / "__init__.py")

    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: Spec)
    assert b.binding_name() == f"_mla_fp8.torch-9.9.0{suffix}"
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    assert "torch-none" in b.binding_name()
