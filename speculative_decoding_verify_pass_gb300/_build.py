"""Builds libspecverify.so (sm_103a) in-tree with nvcc, and beside it _paged.so,
the native half of the Python binding of the paged-cache calls, with g++.
Without torch the library is built alone: users of the C ABI need no torch.

Each translation unit compiles in parallel; the shared library links against
the shared CUDA runtime so it uses the same runtime instance as the process's
PyTorch, and the binding against both.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libspecverify.so")
BINDING = os.path.join(HERE, "_paged.so")
SOURCES = ["gemm.cu", "attention.cu", "misc.cu", "api.cu", "noalloc.cu", "sampling.cu", "pages.cu",
           "paged_attn.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    path = shutil.which("nvcc")
    if path:
        return path
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the library")


def _torch_dir():
    """Where a torch with CUDA is installed (it is not imported); None without one."""
    spec = importlib.util.find_spec("torch")
    path = os.path.dirname(spec.origin) if spec and spec.origin else None
    return path if path and os.path.exists(os.path.join(path, "lib", "libc10_cuda.so")) else None


def _stamp() -> str:
    return os.path.join(BUILD, "paged.abi")


def _abi(torch_dir) -> str:
    """What _paged.so is compiled against and its sources' times do not show (kept in
    _stamp()): the interpreter's ABI and the torch that is installed."""
    with open(os.path.join(torch_dir, "version.py")) as f:
        return "%s %s\n%s" % (sysconfig.get_config_var("SOABI"), torch_dir, f.read())


def _stale() -> bool:
    torch_dir = _torch_dir()
    built = [LIB, BINDING, _stamp()] if torch_dir else [LIB]
    if not all(os.path.exists(p) for p in built):
        return True
    if torch_dir:
        with open(_stamp()) as f:
            if f.read() != _abi(torch_dir):
                return True
    t = min(os.path.getmtime(p) for p in built)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(ROOT, "include", "spec.h"),
                                                                os.path.abspath(__file__)]
    return any(os.path.getmtime(p) > t for p in deps if os.path.exists(p))


def build(force: bool = False, verbose: bool = False, extra_flags=None) -> str:
    if not force and not _stale():
        return LIB
    # objects in a directory of this process: ranks that build at the same
    # time never write one another's files; the library is replaced atomically
    objdir = os.path.join(BUILD, "pid%d" % os.getpid())
    os.makedirs(objdir, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", CSRC,
                    "-I", os.path.join(ROOT, "include"), "--expt-relaxed-constexpr"] + list(extra_flags or [])
    def start(cmd):
        return cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)

    def finish(procs):
        failed = []
        for cmd, p in procs:
            out, _ = p.communicate()
            text = out.decode(errors="replace")
            if verbose and text.strip():
                sys.stdout.write(text)
            if p.returncode != 0:
                failed.append((cmd, text))
        if failed:
            raise RuntimeError("compilation failed:\n" + "\n".join("$ %s\n%s" % (" ".join(c), t) for c, t in failed))

    procs = []
    objs = []
    for src in SOURCES:
        obj = os.path.join(objdir, src.replace(".cu", ".o"))
        objs.append(obj)
        cmd = [cc] + flags + ["-c", os.path.join(CSRC, src), "-o", obj]
        procs.append(start(cmd))
    torch_dir = _torch_dir()
    bobj = os.path.join(objdir, "binding.o")
    if torch_dir:
        cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I", os.path.join(torch_dir, "include"),
               "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               "-I", sysconfig.get_paths()["include"], "-I", os.path.join(os.path.dirname(os.path.dirname(cc)), "include"),
               "-I", os.path.join(ROOT, "include"), "-c", os.path.join(CSRC, "binding.cpp"), "-o", bobj]
        binding = start(cmd)
    finish(procs)
    tmp = LIB + ".tmp%d" % os.getpid()
    link = [cc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + ["-Xlinker", "-rpath,/usr/local/cuda/lib64"]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
    os.replace(tmp, LIB)
    if torch_dir:                               # after the library, which stands without it
        finish([binding])
        tmp = BINDING + ".tmp%d" % os.getpid()
        torch_lib = os.path.join(torch_dir, "lib")
        link = ["g++", "-shared", "-o", tmp, bobj, "-L" + HERE, "-l:libspecverify.so", "-L" + torch_lib, "-ltorch_python", "-ltorch_cpu",
                "-ltorch", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + torch_lib]
        r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout.decode(errors="replace"))
        os.replace(tmp, BINDING)
        tmp = os.path.join(objdir, "paged.abi")
        with open(tmp, "w") as f:
            f.write(_abi(torch_dir))
        os.replace(tmp, _stamp())
    shutil.rmtree(objdir, ignore_errors=True)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True,
          extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else None)
    print(LIB)
