"""Build libattn.so (CUDA for sm_103a) in-tree with nvcc, and the native part of
the Python binding with g++.

Every translation unit is compiled in parallel, then linked into
``transformer_attention_fwd_gb300/_build/libattn.so`` and, against it and the
installed torch, ``_build/_attn_binding.so``.  ptxas statistics (registers,
spills, shared memory) are written to ``_build/ptxas.log``.
"""
from __future__ import annotations

import glob
import os
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


def _torch() -> str:
    import importlib.util
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch not found")
    return os.path.dirname(spec.origin)


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


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(BINDING):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(BINDING))
    return any(os.path.getmtime(p) > t for p in _inputs())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile libattn.so if any source changed (or ``force``); return its path."""
    if not force and not is_stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    binding_obj = os.path.join(BUILD, "binding.o")
    binding_cmd = _binding_compile(binding_obj)
    procs = [("binding.cpp", None, binding_cmd,
              subprocess.Popen(binding_cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True))]
    for src in SOURCES:
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((src, obj, cmd, subprocess.Popen(cmd, stdout=subprocess.PIPE,
                                                        stderr=subprocess.STDOUT, text=True)))
    logs, objs, failed = [], [], []
    for src, obj, cmd, p in procs:
        out, _ = p.communicate()
        logs.append(f"== {src}\n{out}")
        if p.returncode != 0:
            failed.append(src)
        if obj is not None:
            objs.append(obj)
    with open(os.path.join(BUILD, "ptxas.log"), "w") as f:
        f.write("\n".join(logs))
    if failed:
        sys.stderr.write("\n".join(logs))
        raise RuntimeError(f"nvcc failed for {failed}")
    tmp = LIB + f".tmp{os.getpid()}"
    link = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(link, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError("link of libattn.so failed")
    os.replace(tmp, LIB)
    tmp = BINDING + f".tmp{os.getpid()}"
    r = subprocess.run(_binding_link(binding_obj, tmp), stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout)
        raise RuntimeError("link of _attn_binding.so failed")
    os.replace(tmp, BINDING)
    if verbose:
        print("\n".join(logs))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
