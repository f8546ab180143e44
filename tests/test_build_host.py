"""What the build makes, when, and what a failing half leaves behind: on a copy of the build script with stand-ins
for the compilers, which write the file they are asked for, or fail."""

import importlib.util
import os
import shutil
import subprocess
import sys
import time

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

COMPILER = """#!/bin/sh
echo "$0 $*" >> "{log}"
[ -e "{fail}" ] && exit 1
while [ $# -gt 0 ]; do
    if [ "$1" = -o ]; then echo built > "$2"; fi
    shift
done
"""


class Tree:
    """A package of two kernels' sources and the binding, with its own compilers."""

    def __init__(self, tmp, monkeypatch):
        self.pkg = tmp / "pkg"
        (self.pkg / "csrc").mkdir(parents=True)
        (tmp / "include").mkdir()
        (tmp / "bin").mkdir()
        for p in (self.pkg / "csrc" / "a.cu", self.pkg / "csrc" / "b.cu", self.pkg / "csrc" / "binding.cpp",
                  tmp / "include" / "ssm_scan.h"):
            p.write_text("")
            os.utime(p, (1, 1))
        shutil.copy(os.path.join(ROOT, "selective_state_space_bwd_b200", "build.py"), self.pkg / "build.py")
        self.log, self.lib, self.binding = tmp / "log", self.pkg / "libssm_scan.so", self.pkg / "_ssm_torch.so"
        for name, var in (("nvcc", "NVCC"), ("cxx", "CXX")):
            tool = tmp / "bin" / name
            tool.write_text(COMPILER.format(log=self.log, fail=tmp / ("fail_" + name)))
            tool.chmod(0o755)
            monkeypatch.setenv(var, str(tool))
        self.tmp = tmp

    def fail(self, name, on=True):
        p = self.tmp / ("fail_" + name)
        p.write_text("") if on else p.unlink()

    def load(self):
        spec = importlib.util.spec_from_file_location("build_copy", self.pkg / "build.py")
        mod = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(mod)
        return mod

    def runs(self, name):
        """Command lines of a compiler so far."""
        lines = self.log.read_text().splitlines() if self.log.exists() else []
        return [s for s in lines if s.split()[0].endswith("/" + name)]


@pytest.fixture
def tree(tmp_path, monkeypatch):
    return Tree(tmp_path, monkeypatch)


def test_a_build_makes_both_and_a_second_one_nothing(tree):
    b = tree.load()
    assert not b.up_to_date()
    assert b.build() == str(tree.lib) and tree.lib.exists() and tree.binding.exists()
    assert len(tree.runs("nvcc")) == 3 and len(tree.runs("cxx")) == 2 and b.up_to_date()
    b.build()
    assert len(tree.runs("nvcc")) == 3 and len(tree.runs("cxx")) == 2
    now = time.time() + 10
    os.utime(tree.pkg / "csrc" / "a.cu", (now, now))
    b.build()
    assert len(tree.runs("nvcc")) == 5 and len(tree.runs("cxx")) == 2  # one object and the library


def test_the_library_does_not_wait_for_the_binding(tree):
    """The C ABI needs nvcc alone: where the binding cannot be compiled the library is there, and the error after it."""
    tree.fail("cxx")
    b = tree.load()
    with pytest.raises(subprocess.CalledProcessError) as e:
        b.build()
    assert "binding.cpp" in " ".join(e.value.cmd)
    assert tree.lib.exists() and not tree.binding.exists() and not b.up_to_date()
    tree.fail("cxx", False)
    b.build()
    assert tree.binding.exists() and len(tree.runs("nvcc")) == 3  # the library was not built again


def test_a_failing_kernel_source_makes_nothing(tree):
    tree.fail("nvcc")
    with pytest.raises(subprocess.CalledProcessError):
        tree.load().build()
    assert not tree.lib.exists() and not tree.binding.exists()


def test_without_torch_the_library_alone_is_built(tree, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    b = tree.load()
    assert b.build() == str(tree.lib) and tree.lib.exists() and b.up_to_date()
    assert not tree.runs("cxx") and not tree.binding.exists()


def test_the_library_alone_on_demand(tree):
    b = tree.load()
    b.build(binding=False)
    assert tree.lib.exists() and not tree.runs("cxx") and not b.up_to_date()
    b.build(binding=False)
    assert len(tree.runs("nvcc")) == 3


def test_another_torch_or_python_makes_the_binding_anew(tree, monkeypatch):
    """The binding is compiled against one torch, C++ ABI and Python: under another it is not up to date."""
    import sysconfig

    import torch
    b = tree.load()
    b.build()
    assert b.up_to_date() and len(tree.runs("cxx")) == 2
    real = sysconfig.get_config_var
    for n, change in enumerate((lambda m: m.setattr(torch, "__version__", "0.0.1"),
                                lambda m: m.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI",
                                                    not torch._C._GLIBCXX_USE_CXX11_ABI),
                                lambda m: m.setattr(sysconfig, "get_config_var",
                                                    lambda k: "other" if k == "SOABI" else real(k)))):
        with monkeypatch.context() as m:
            change(m)
            assert not b.up_to_date()
            b.build()
            assert b.up_to_date() and len(tree.runs("cxx")) == 2 * (2 * n + 2)
        assert not b.up_to_date()
        b.build()
        assert len(tree.runs("cxx")) == 2 * (2 * n + 3) and len(tree.runs("nvcc")) == 3


def test_a_binding_of_another_torch_is_not_used(monkeypatch):
    if not os.path.exists(os.path.join(ROOT, "selective_state_space_bwd_b200", "_ssm_torch.so")):
        pytest.skip("needs the built binding")
    import torch

    from selective_state_space_bwd_b200 import build, ssm_scan
    build.build()
    monkeypatch.setattr(ssm_scan, "_torch_binding", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        with pytest.raises(RuntimeError, match="was built against"):
            ssm_scan._native()
    assert ssm_scan._native() is not None
