"""Build the sm_100a C-ABI library in-tree with nvcc (no GPU needed to build)."""
from __future__ import annotations

import os
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libnvfp4_b200.so")
# test-only variant: same sources built with NVFP4_WAIT_TEST, whose kernels' wait
# limit and a forced stall can be set, so that tests can make a bounded wait expire
WAIT_TEST_LIB = os.path.join(HERE, "libnvfp4_b200_waittest.so")
ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]


def sources() -> list[str]:
    out = [os.path.join(ROOT, "include", "nvfp4.h")]
    for name in sorted(os.listdir(CSRC)):
        if name.endswith((".cu", ".cuh", ".h")):
            out.append(os.path.join(CSRC, name))
    return out


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _compile(out: str, defines: list[str], force: bool, verbose: bool) -> str:
    newest = max(os.path.getmtime(p) for p in sources())
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    tmp = out + ".tmp%d" % os.getpid()
    cmd = [nvcc(), *ARCH_FLAGS, "-O3", "-lineinfo", "-std=c++17", "-shared",
           "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
           "--cudart", "static", *defines, "-I", os.path.join(ROOT, "include"),
           "-o", tmp, os.path.join(CSRC, "nvfp4_api.cu")]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
        print(" ".join(cmd), file=sys.stderr)
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile csrc/nvfp4_api.cu (the library's single translation unit) into LIB."""
    return _compile(LIB, [], force, verbose)


def build_wait_test(force: bool = False) -> str:
    """The test-only variant (NVFP4_WAIT_TEST) into WAIT_TEST_LIB."""
    return _compile(WAIT_TEST_LIB, ["-DNVFP4_WAIT_TEST"], force, False)


def host_calls_path() -> str:
    """The INT8 path's marshalling as a CPython module (host code over torch's C++ headers).
    It depends on the layouts of the interpreter and the torch it was built with, so its name
    carries both: another one does not find it, and builds its own."""
    import re
    import sysconfig
    import torch
    key = "-".join((sysconfig.get_config_var("SOABI") or "", "torch", torch.__version__,
                    (torch.version.git_version or "")[:12],
                    "abi%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)))
    return os.path.join(HERE, "_host_calls.%s.so" % re.sub(r"[^0-9A-Za-z+_-]", "_", key))


def build_host_calls(force: bool = False) -> str:
    """Compile csrc/host_calls.cpp (with g++, against the installed torch) into host_calls_path()."""
    src, out = os.path.join(CSRC, "host_calls.cpp"), host_calls_path()
    newest = max(os.path.getmtime(p) for p in (src, os.path.join(ROOT, "include", "nvfp4.h")))
    if not force and os.path.exists(out) and os.path.getmtime(out) >= newest:
        return out
    import sysconfig
    import torch
    base = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    inc = [os.path.join(base, "include"),
           os.path.join(base, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    tmp = out + ".tmp%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for path in inc:
        cmd += ["-isystem", path]
    cmd += ["-o", tmp, src, "-L", os.path.join(base, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_cuda", "-ltorch_python"]
    subprocess.check_call(cmd)
    os.replace(tmp, out)
    return out


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
    print(build_wait_test(force="--force" in sys.argv))
    print(build_host_calls(force="--force" in sys.argv))
