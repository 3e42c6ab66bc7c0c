"""How the attention layer's marshalling module is built, on the CPU: it is
tied to one torch and one Python, the library to neither."""
import os
import subprocess
import sys

import pytest
import torch

from nvfp4_w4a4_quantized_act_b200 import build as nbuild
from nvfp4_w4a4_quantized_act_b200 import ops


def test_the_module_of_another_torch_or_python_is_not_found():
    here = nbuild.binding_path(torch.__version__)
    assert ops.BINDING_PATH == here and here.endswith(".so") and os.path.dirname(here) == nbuild.PKG
    assert here != nbuild.binding_path("2.0.0") and here != nbuild.binding_path(torch.__version__, "cpython-39")
    assert nbuild.binding_path("2.0.0") != nbuild.binding_path("2.0.1")


def test_another_torch_means_another_build(monkeypatch, tmp_path):
    """A module that is newer than its source, but was built for another torch,
    does not pass for this one's."""
    made = []

    def compile(cmd):
        made.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
    monkeypatch.setattr(nbuild, "PKG", str(tmp_path))
    monkeypatch.setattr(nbuild.subprocess, "check_call", compile)
    first = nbuild.build_binding()
    assert len(made) == 1 and os.path.exists(first) and nbuild.build_binding() == first and len(made) == 1
    monkeypatch.setattr(torch, "__version__", "99.0")
    assert nbuild.build_binding() != first and len(made) == 2


def test_the_library_does_not_wait_for_the_module(monkeypatch):
    """Without g++ or torch's headers the library is built all the same, first;
    --library-only asks for nothing else."""
    order = []
    monkeypatch.setattr(nbuild, "build_library", lambda *a: order.append("library"))

    def fails(*a):
        order.append("module")
        raise FileNotFoundError("g++")
    monkeypatch.setattr(nbuild, "build_binding", fails)
    assert nbuild.build(binding=False) == nbuild.LIB and order == ["library"]
    with pytest.raises(FileNotFoundError):
        nbuild.build()
    assert order == ["library", "library", "module"]


def test_library_alone_needs_no_torch():
    code = ("import sys; sys.modules['torch'] = None; "
            "from nvfp4_w4a4_quantized_act_b200 import build; build.up_to_date = lambda: True; print(build.build(binding=False))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=nbuild.ROOT, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == nbuild.LIB, r.stderr[-1000:]
