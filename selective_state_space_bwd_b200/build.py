"""Build libssm_scan.so (all CUDA sources under csrc/) for sm_100a with nvcc, and the compiled binding
_ssm_torch.so (csrc/binding.cpp) with the host compiler, in-tree.  The library needs nvcc alone; the binding, which
only Python programs with torch use, is left out where torch is not installed, or with ``--library``."""

from __future__ import annotations

import glob
import importlib.util
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "libssm_scan.so")
BINDING = os.path.join(HERE, "_ssm_torch.so")
BINDING_KEY = os.path.join(HERE, "_build", "binding.key")  # binding_key() of the binding that is there
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources():
    return sorted(glob.glob(os.path.join(HERE, "csrc", "*.cu")))


def deps():
    return sources() + sorted(glob.glob(os.path.join(HERE, "csrc", "*.h*"))) + [
        os.path.join(ROOT, "include", "ssm_scan.h")]


def binding_deps():
    return [os.path.join(HERE, "csrc", "binding.cpp"), os.path.join(ROOT, "include", "ssm_scan.h")]


def _newer(out, ins) -> bool:
    return os.path.exists(out) and all(os.path.getmtime(p) <= os.path.getmtime(out) for p in ins)


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def binding_key() -> str:
    """What a compiled binding belongs to: torch's version and C++ ABI, and the Python's ABI."""
    import sysconfig

    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {sysconfig.get_config_var('SOABI')}")


def _binding_up_to_date() -> bool:
    if not _newer(BINDING, binding_deps()) or not os.path.exists(BINDING_KEY):
        return False
    try:
        with open(BINDING_KEY) as f:
            return f.read() == binding_key()
    except Exception:  # a torch that does not import: the build says so, behind the library
        return False


def up_to_date(binding: bool = True) -> bool:
    return _newer(LIB, deps()) and not (binding and _has_torch() and not _binding_up_to_date())


def _binding_commands(obj):
    """The host compiler's commands for the binding (compile, link), against the installed torch."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension as ext
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(shutil.which(os.environ.get("NVCC", "nvcc")))))
    inc = [sysconfig.get_paths()["include"], *ext.include_paths(), os.path.join(cuda, "include")]
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cxx = os.environ.get("CXX", "g++")
    return ([cxx, "-std=c++17", "-O2", "-fPIC", "-fvisibility=hidden",
             f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
             "-DTORCH_EXTENSION_NAME=_ssm_torch", f'-DSSM_BUILT_AGAINST="{binding_key()}"', *[f"-isystem{p}" for p in inc], "-c", binding_deps()[0], "-o", obj],
            [cxx, "-shared", obj, "-o", BINDING + ".tmp", f"-L{lib}", "-ltorch_python", "-ltorch", "-ltorch_cpu",
             "-lc10", "-lc10_cuda", "-L" + HERE, "-l:libssm_scan.so", "-Wl,-rpath,$ORIGIN"])


def build(force: bool = False, verbose: bool = False, binding: bool = True) -> str:
    """Compile every source whose object is stale to an object, in parallel (one nvcc process
    each; no device code crosses files), then link the shared library and, against it, the binding.
    An error of the binding's is raised once the library is in place."""
    if not force and up_to_date(binding):
        return LIB
    nvcc = os.environ.get("NVCC", "nvcc")
    obj_dir = os.path.join(HERE, "_build")
    os.makedirs(obj_dir, exist_ok=True)
    flags = [*ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
             "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags.append("-Xptxas=-v")
    objs = [os.path.join(obj_dir, os.path.basename(src)[:-3] + ".o") for src in sources()]
    headers = [p for p in deps() if not p.endswith(".cu")]

    def stale(src, obj):
        return force or not os.path.exists(obj) or any(
            os.path.getmtime(p) > os.path.getmtime(obj) for p in [src, *headers])

    procs = [subprocess.Popen([nvcc, *flags, "-c", src, "-o", obj])
             for src, obj in zip(sources(), objs) if stale(src, obj)]
    link = compiling = error = None
    if binding and _has_torch() and (force or not _binding_up_to_date()):
        try:
            compile_, link = _binding_commands(os.path.join(obj_dir, "binding.o"))
            compiling = subprocess.Popen(compile_)
        except Exception as e:  # a torch that does not import, no compiler: the library comes first
            error = e
    failed = [p.args for p in procs if p.wait() != 0]
    if compiling and compiling.wait() != 0:
        error = subprocess.CalledProcessError(1, compiling.args)
    if failed:
        raise subprocess.CalledProcessError(1, failed[0])
    if force or not _newer(LIB, [*deps(), *objs]):
        subprocess.run([nvcc, *ARCH, "-shared", "-Xlinker", "-soname=libssm_scan.so", "-o", LIB + ".tmp", *objs],
                       check=True)
        os.replace(LIB + ".tmp", LIB)
    if error:
        raise error
    if link:
        subprocess.run(link, check=True)
        os.replace(BINDING + ".tmp", BINDING)
        with open(BINDING_KEY, "w") as f:
            f.write(binding_key())
    return LIB


if __name__ == "__main__":
    build(force=True, verbose="-v" in sys.argv, binding="--library" not in sys.argv)
    print(LIB)
