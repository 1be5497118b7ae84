"""Build of the in-tree CUDA library ``libhra.so`` for GB300 (sm_103a only).

Each translation unit under ``csrc/`` is compiled by nvcc in parallel into ``_build/`` at the
repository root, then linked into ``qwen3_prefill_delayed_gb300/libhra.so`` (cudart linked
statically, so the library loads on a machine without a GPU and its symbols can be listed there).
Beside it the host compiler builds ``_kv8_binding.so``, the compiled Python calls of the 8-bit cache.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libhra.so")
BINDING_SRC = os.path.join(CSRC, "kv8_binding.cpp")
BINDING = os.path.join(PKG, "_kv8_binding.so")
SOURCES = ["api.cu", "gemm_tc.cu", "attention.cu", "attention_tc.cu", "elementwise.cu", "codebook.cu", "fp8.cu",
           "noalloc.cu", "head.cu", "nvfp4.cu", "decode_pass.cu", "kv8_append.cu", "kv8_attention.cu", "kv8_prompt.cu", "kv8_shared.cu",
           "kv8_pages.cu",
           "kv8_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fno-strict-aliasing",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhra.so")


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_command(out: str):
    """g++ of the CPython module: it needs torch's headers and links its shared libraries, and no CUDA compiler."""
    import sysconfig

    import torch
    t = os.path.dirname(torch.__file__)
    nvcc_root = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(t, "include"), sysconfig.get_paths()["include"], os.path.join(nvcc_root, "include"),
           "/usr/local/cuda/include"]
    cxx = shutil.which("g++") or "g++"
    return [cxx, "-shared", "-fPIC", "-O2", "-std=c++17", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            *["-I" + d for d in inc], BINDING_SRC, "-o", out, "-L" + os.path.join(t, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + os.path.join(t, "lib")]


def _binding_needs() -> str:
    """What the binding is made with, as text."""
    import torch
    return "\n".join(_binding_command("") + [torch.__version__, sys.implementation.cache_tag or ""])


def _read(path: str) -> str:
    try:
        with open(path) as f:
            return f.read()
    except OSError:
        return ""


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "hra.h"))
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(o)
        if force or _stale(o, [s] + headers):
            jobs.append([nvcc, *ARCH, *FLAGS, *extra_flags, "-c", s, "-o", o])

    # the binding depends on torch and Python too: it is made anew when they, or the command, are others than last time
    binding_tmp = os.path.join(BUILD, f"{os.path.basename(BINDING)}.tmp{os.getpid()}")
    made_with = os.path.join(BUILD, os.path.basename(BINDING) + ".made_with")
    binding, binding_error, now = None, None, ""
    try:
        now = _binding_needs()
        if force or _stale(BINDING, [BINDING_SRC, os.path.join(ROOT, "include", "hra.h")]) or _read(made_with) != now:
            binding = _binding_command(binding_tmp)
            jobs.append(binding)
    except ImportError as e:
        binding_error = str(e)

    def run(cmd):
        try:
            return cmd, subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:
            return cmd, subprocess.CompletedProcess(cmd, 127, "", f"{e}\n")

    failed = []
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0 and cmd is binding:
                binding_error = f"{cmd[0]} failed for {BINDING_SRC}"
            elif r.returncode != 0:
                failed.append(next(a for a in cmd if a.startswith(CSRC)))
    if failed:
        raise RuntimeError("nvcc failed for: " + ", ".join(failed))
    if force or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("link failed:\n" + r.stdout + r.stderr)
        os.replace(tmp, LIB)
    if binding_error is not None:   # the library does not need it
        raise RuntimeError("libhra.so is built; the Python calls of the 8-bit cache are not: " + binding_error)
    if binding is not None:
        os.replace(binding_tmp, BINDING)
        with open(made_with, "w") as f:
            f.write(now)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
