"""Build libattn.so (CUDA for sm_103a) in-tree with nvcc, and the native part of
the Python binding with g++.

Every translation unit is compiled in parallel, then linked into
``transformer_attention_fwd_gb300/_build/libattn.so`` and, against it and the
installed torch (where there is one), ``_build/_attn_binding.so``, which is built
again for another torch or Python.  ptxas statistics (registers, spills, shared
memory) are written to ``_build/ptxas.log``.
"""
from __future__ import annotations

import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libattn.so")
BINDING = os.path.join(BUILD, "_attn_binding.so")

SOURCES = ["attn_api.cu", "prefill_bf16.cu", "prefill_d64.cu", "decode_bf16.cu", "simt_f32.cu",
           "varlen_sched.cu", "rope.cu", "append.cu", "append_e4m3.cu", "decode_e4m3.cu",
           "decode_e4m3_short.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
              "--expt-relaxed-constexpr", "-I", INCLUDE]


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _torch() -> str | None:
    """The installed torch's folder; None without one for CUDA."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.origin:
        return None
    folder = os.path.dirname(spec.origin)
    return folder if os.path.exists(os.path.join(folder, "lib", "libtorch_cuda.so")) else None


def _binding_compile(obj: str) -> list[str]:
    t = _torch()
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D_GLIBCXX_USE_CXX11_ABI=1",
            "-isystem", sysconfig.get_paths()["include"], "-isystem", os.path.join(t, "include"),
            "-isystem", os.path.join(cuda, "include"), "-I", INCLUDE,
            "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj]


def _binding_link(obj: str, out: str) -> list[str]:
    lib = os.path.join(_torch(), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L", BUILD, "-l:libattn.so", "-L", lib, "-lc10", "-lc10_cuda",
            "-ltorch_cpu", "-ltorch_cuda", "-ltorch_python", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def _inputs():
    return glob.glob(os.path.join(CSRC, "*")) + glob.glob(os.path.join(INCLUDE, "*.h")) + [__file__]


def _older(target: str) -> bool:
    """The target is missing, or older than an input."""
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in _inputs())


def installed_torch() -> str:
    """The version in the installed torch's version.py ("" if it says none)."""
    try:
        with open(os.path.join(_torch() or "", "version.py")) as f:
            found = re.search(r"^__version__\s*=\s*['\"]([^'\"]+)", f.read(), re.M)
    except OSError:
        return ""
    return found.group(1) if found else ""


def binding_for(torch_version: str) -> str:
    """What a binding is good for: it holds the layouts of one torch's C++ classes, and of
    one Python's."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def binding_built_for() -> str:
    """The same of the binding that is there ("" if it does not say)."""
    try:
        with open(BINDING + ".for") as f:
            return f.read()
    except OSError:
        return ""


def _binding_stale() -> bool:
    return _torch() is not None and (_older(BINDING) or not os.path.exists(LIB) or
                                     binding_built_for() != binding_for(installed_torch()))


def is_stale() -> bool:
    return _older(LIB) or _binding_stale()


def _start(cmd: list[str]) -> subprocess.Popen:
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)


def _link(cmd, target: str) -> None:
    """Runs the link command cmd(output) and puts its output in the target's place."""
    tmp = target + f".tmp{os.getpid()}"
    r = subprocess.run(cmd(tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError(f"link of {os.path.basename(target)} failed")
    os.replace(tmp, target)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libattn.so, and the binding where torch with CUDA is installed, if any source
    changed (or ``force``); return libattn.so's path.  The library needs neither torch nor
    Python's headers, and is there even if the binding fails."""
    lib, binding = force or _older(LIB), _torch() is not None and (force or _binding_stale())
    if not lib and not binding:
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    procs, logs, objs, failed = [], [], [], []
    binding_obj = os.path.join(BUILD, "binding.o")
    if binding:
        procs.append(("binding.cpp", None, _start(_binding_compile(binding_obj))))
    if lib:
        cc = nvcc()
        for src in SOURCES:
            obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
            objs.append(obj)
            procs.append((src, obj, _start([cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj])))
    for src, _, p in procs:
        out, _ = p.communicate()
        logs.append(f"== {src}\n{out}")
        if p.returncode != 0:
            failed.append(src)
    if lib:
        with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
            f.write("\n".join(logs))
    if failed:
        sys.stderr.write("\n".join(logs))
    if set(failed) - {"binding.cpp"}:
        raise RuntimeError(f"nvcc failed for {failed}")
    if lib:
        _link(lambda out: [cc, *ARCH, "-shared", "-o", out, *objs], LIB)
    if failed:
        raise RuntimeError("g++ failed for binding.cpp")
    if binding:
        _link(lambda out: _binding_link(binding_obj, out), BINDING)
        # In place at once, and after the binding: other processes may load it meanwhile.
        tmp = BINDING + f".for.tmp{os.getpid()}"
        with open(tmp, "w") as f:
            f.write(binding_for(installed_torch()))
        os.replace(tmp, BINDING + ".for")
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
