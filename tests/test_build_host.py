"""What the library's build needs: nvcc alone. The module for torch tensors is built on its own, when it is needed."""
import os
import subprocess
import sys
import sysconfig

import pytest

from exact_io_aware_32_gb300 import build, fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def empty(tmp_path, monkeypatch):
    """A build folder that holds the objects but neither the library nor the module, and a host compiler that fails."""
    build.build()
    for src in build.SOURCES:
        os.symlink(os.path.join(build.BUILD, src.replace(".cu", ".o")), tmp_path / src.replace(".cu", ".o"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libfa.so"))
    monkeypatch.setattr(build, "_torch_module_cmd", lambda out: ["sh", "-c", "echo no headers; exit 1"])
    monkeypatch.setattr(fa, "_lib", None)
    monkeypatch.setattr(fa, "_torch_module", None)
    return tmp_path


def test_library_builds_and_loads_where_the_module_does_not(empty):
    assert build.build() == str(empty / "libfa.so") and os.path.exists(empty / "libfa.so")
    assert fa.fa_fwd_paged_workspace_bytes(4, 2, 8, 2, 128, 1) > 0
    with pytest.raises(RuntimeError, match="no headers"):
        fa._paged()
    assert fa.fa_paged_plan(0, 0, 1, 16, 0, 0, 0, 0, 1, 0, 0, 0, 1, 0, stream=0) == fa.FA_ERR_INVALID_ARG


def test_addresses_need_no_torch():
    """The calls that take raw addresses work in an interpreter without torch."""
    build.build()
    code = """
import sys
sys.modules["torch"] = None
sys.path.insert(0, %r)
from exact_io_aware_32_gb300 import build, fa
build.build()
assert fa.fa_fwd(0, 0, 0, 0, 0, 1, 1, 1, 64, 1.0, False, stream=0) == fa.FA_ERR_INVALID_ARG
assert fa.fa_fwd_paged_workspace_bytes(4, 2, 8, 2, 128, 1) > 0
""" % ROOT
    subprocess.check_call([sys.executable, "-c", code])


def test_module_is_named_after_torch_and_the_interpreter(monkeypatch):
    import torch

    name = os.path.basename(build.torch_module())
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    other = os.path.basename(build.torch_module())
    monkeypatch.undo()
    real = sysconfig.get_config_var
    monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-399-z80" if n == "SOABI" else real(n))
    assert len({name, other, os.path.basename(build.torch_module())}) == 3
