"""What the build needs: the C library nvcc alone, its torch module torch and g++."""
import os
import subprocess
import sys

import pytest

from memory_bound_transformer_decode_gb300 import build


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """The build in a directory of its own, with compilers that only write their outputs; the commands run."""
    for name, file in (("BUILD", ""), ("LIB", "libddl.so"), ("TORCH_LIB", "_ddl_torch.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file) if file else str(tmp_path))
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        fail = os.path.basename(cmd[0]) in failing
        if not fail:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, int(fail), "", "")

    failing = set()
    monkeypatch.setattr(build.subprocess, "run", run)
    return ran, failing, tmp_path


def test_the_library_is_built_without_torch(tools, monkeypatch):
    ran, _, where = tools
    monkeypatch.setitem(sys.modules, "torch", None)  # (import torch raises ImportError)
    assert build.build() == build.LIB
    assert (where / "libddl.so").exists() and not (where / "_ddl_torch.so").exists()
    assert ran and all(os.path.basename(c[0]) == "nvcc" for c in ran)
    n = len(ran)
    assert build.build() == build.LIB and len(ran) == n  # nothing is stale


def test_a_module_that_does_not_compile_fails_loudly_and_leaves_the_library(tools):
    ran, failing, where = tools
    failing.add("g++")
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert (where / "libddl.so").exists() and not (where / "_ddl_torch.so").exists()


def test_library_and_module_are_built_and_only_when_stale(tools):
    ran, _, where = tools
    build.build()
    assert (where / "libddl.so").exists() and (where / "_ddl_torch.so").exists()
    n = len(ran)
    build.build()
    assert len(ran) == n
    os.utime(where / "_ddl_torch.so", (0, 0))
    build.build()
    assert [os.path.basename(c[0]) for c in ran[n:]] == ["g++", "g++"]
