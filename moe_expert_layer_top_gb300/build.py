"""In-tree build of the CUDA libraries for sm_103a.

``build()`` compiles:
* ``csrc/*.cu`` -> ``moe_expert_layer_top_gb300/_build/libmoe.so``, the C-ABI library;
* the same sources with ``-DMOE_DEBUG_BOUNDS`` -> ``_build/libmoe_debug.so``, the
  bounds-checked build (every kernel index checked; a miss is reported as
  MOE_ERR_DEVICE_BOUNDS and the access skipped), loaded instead of libmoe.so
  when the environment sets MOE_DEBUG_BOUNDS=1;
* ``csrc/attention_torch.cpp`` -> ``_build/attention_torch.so``, the Python module
  that passes PyTorch tensors to the attention calls (host code, g++; only where
  PyTorch is installed, anew for another one, and after the libraries, which need
  nvcc alone);
* ``synth/synth.cu`` -> ``synth/_build/libmoe_synth.so``, the device side of the
  seeded input generator.
The translation units are compiled in parallel, each with one ``-gencode``.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(LIB_DIR, "libmoe.so")
DEBUG_DIR = os.path.join(LIB_DIR, "debug")
DEBUG_LIB_PATH = os.path.join(LIB_DIR, "libmoe_debug.so")
TORCH_SRC = os.path.join(CSRC, "attention_torch.cpp")
TORCH_LIB_PATH = os.path.join(LIB_DIR, "attention_torch.so")
TORCH_STAMP_PATH = os.path.join(LIB_DIR, "attention_torch.stamp")
SYNTH_DIR = os.path.join(ROOT, "synth")
SYNTH_LIB_DIR = os.path.join(SYNTH_DIR, "_build")
SYNTH_LIB_PATH = os.path.join(SYNTH_LIB_DIR, "libmoe_synth.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("command failed: " + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def _compile(src: str, obj: str, extra=()):
    return _run([nvcc(), *ARCH, *FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj])


def _torch_home() -> str | None:
    """Directory of the installed PyTorch, without importing it; None where there is none."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def _torch_stamp(home: str) -> str:
    """What the module was built against: it fits no other interpreter or PyTorch."""
    with open(os.path.join(home, "version.py")) as f:
        return f"{sys.version}\n{home}\n{f.read()}"


def _torch_module_stale(home: str) -> bool:
    if _stale(TORCH_LIB_PATH, [TORCH_SRC, os.path.join(INCLUDE, "moe.h")]) or not os.path.exists(TORCH_STAMP_PATH):
        return True
    with open(TORCH_STAMP_PATH) as f:
        return f.read() != _torch_stamp(home)


def _build_torch_module(home: str):
    import sysconfig
    import torch
    lib = os.path.join(home, "lib")
    tmp = TORCH_LIB_PATH + ".tmp"
    _run([os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE,
          "-I", sysconfig.get_paths()["include"], "-isystem", os.path.join(home, "include"),
          "-isystem", os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include"), TORCH_SRC,
          "-o", tmp, "-L", lib, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-Wl,-rpath,{lib}"])
    os.replace(tmp, TORCH_LIB_PATH)
    with open(TORCH_STAMP_PATH, "w") as f:
        f.write(_torch_stamp(home))


def _stale(target: str, sources) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(s) > t for s in sources)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(LIB_DIR, exist_ok=True)
    os.makedirs(DEBUG_DIR, exist_ok=True)
    os.makedirs(SYNTH_LIB_DIR, exist_ok=True)
    cus = sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))
    deps = cus + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    deps.append(os.path.join(INCLUDE, "moe.h"))
    synth_src = os.path.join(SYNTH_DIR, "synth.cu")
    jobs = []
    if force or _stale(LIB_PATH, deps):
        objs = [os.path.join(LIB_DIR, os.path.basename(c)[:-3] + ".o") for c in cus]
        jobs.append(("moe", cus, objs, LIB_PATH, ()))
    if force or _stale(DEBUG_LIB_PATH, deps):
        objs = [os.path.join(DEBUG_DIR, os.path.basename(c)[:-3] + ".o") for c in cus]
        jobs.append(("moe_debug", cus, objs, DEBUG_LIB_PATH, ("-DMOE_DEBUG_BOUNDS",)))
    if force or _stale(SYNTH_LIB_PATH, [synth_src]):
        jobs.append(("synth", [synth_src], [os.path.join(SYNTH_LIB_DIR, "synth.o")], SYNTH_LIB_PATH, ()))
    work = [(s, o, tuple(flags) + (("-Xptxas", "-v") if verbose else ()))
            for _, srcs, objs, _, flags in jobs for s, o in zip(srcs, objs)]
    home = _torch_home()
    module = home is not None and (force or _torch_module_stale(home))
    with ThreadPoolExecutor(max_workers=max(1, min(len(work) + 1, os.cpu_count() or 4))) as ex:
        pending = [ex.submit(_build_torch_module, home)] if module else []
        logs = list(ex.map(lambda a: _compile(*a), work))
        if verbose:
            for log in logs:
                print(log)
        for _, _, objs, lib, _ in jobs:
            tmp = lib + ".tmp"
            _run([nvcc(), *ARCH, "-shared", "-o", tmp, *objs])
            os.replace(tmp, lib)
        for p in pending:  # last: the libraries are there whatever becomes of it
            p.result()
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
